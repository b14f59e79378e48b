// Plays the queue of a wave's loads as the e4m3 products send for them, with the counts they wait by.
// A line of input is one form; its answer is "ok" or what is read before it has landed.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <deque>

#include "waits.h"

namespace {

struct Load {
    int slab;
    char part;                                  // 'x', 'w', or 's' for scales, whose use waits for them
};

struct Queue {
    std::deque<Load> out;                       // sent for and maybe not here, oldest first
    void send(int slab, char part, int n) { out.insert(out.end(), n, Load{slab, part}); }
    void wait(int n) {
        while ((int)out.size() > n) out.pop_front();
    }
    void use_scales() {
        while (std::any_of(out.begin(), out.end(), [](Load l) { return l.part == 's'; })) out.pop_front();
    }
    bool here(int slab) const {
        return std::none_of(out.begin(), out.end(), [=](Load l) { return l.part != 's' && l.slab == slab; });
    }
};

// A wave of a tile of `full` whole slabs; scales: it fetches those of the workgroup.  The first slab that is
// read too soon, or -1.
int play_tile(const dmm::StageQueue& q, int begin, int full, bool scales) {
    const int n = q.stages, half = q.x - q.x / 2;
    Queue loads;
    if (full >= n) {
        for (int i = 0; i < n; ++i) loads.send(i, 'w', q.w);
        if (scales) loads.send(-1, 's', 2);
        for (int i = 0; i < n; ++i) loads.send(i, 'x', q.x);
        if (scales) loads.use_scales();
        loads.wait(begin);
    } else {
        for (int i = 0; i < full; ++i) loads.send(i, 'x', q.x + q.w);
        loads.wait(0);
    }
    for (int t = 0; t < full; ++t) {
        if (!loads.here(t)) return t;
        if (scales && t % n == 0) loads.send(-1, 's', 2);
        if (q.early && t + n < full) loads.send(t + n, 'x', half + q.w);
        if (scales && t % n == n - 1) loads.use_scales();
        loads.wait(t + n - (q.early ? 0 : 1) < full ? q.slab() : 0);
        if (t + n < full) loads.send(t + n, 'x', q.early ? q.x - half : q.x + q.w);
    }
    return -1;
}

// Wave `wave` of a streaming workgroup over nb blocks, `loads` a block.  The first block that is read too soon, or -1.
int play_stream(int nbuf, int W, int loads, int wave, int nb, bool old) {
    Queue q;
    for (int i = 0; i < nbuf; ++i) q.send(wave + i * W, 'w', loads);
    for (int c = wave; c < nb; c += W) {
        int behind = dmm::blocks_behind(c, W, nbuf, nb);
        if (old) behind = c < nbuf * W || c + (nbuf - 1) * W < nb ? nbuf - 1 : nbuf > 2 && c + W < nb ? 1 : 0;
        q.wait(behind * loads);
        if (!q.here(c)) return c;
        if (c + nbuf * W < nb) q.send(c + nbuf * W, 'w', loads);
    }
    return -1;
}

}  // namespace

int main() {
    char kind[16];
    while (std::scanf("%15s", kind) == 1) {
        if (!std::strcmp(kind, "tile")) {
            int early, begin;                   // begin < 0: the kernels' count
            dmm::StageQueue q;
            if (std::scanf("%d %d %d %d %d", &q.stages, &q.x, &q.w, &early, &begin) != 5) return 1;
            q.early = early != 0;
            int bad = -1, full = 0;
            for (; bad < 0 && full < 40; ++full)
                for (int scales = 0; bad < 0 && scales < 2; ++scales)
                    bad = play_tile(q, begin < 0 ? q.begin() : begin, full, scales != 0);
            if (bad < 0) std::puts("ok");
            else std::printf("slab %d of %d\n", bad, full - 1);
        } else if (!std::strcmp(kind, "stream")) {
            int nbuf, W, loads, old;            // old: all first blocks count as sent for behind each of them
            if (std::scanf("%d %d %d %d", &nbuf, &W, &loads, &old) != 4) return 1;
            int bad = -1, nb = 0;
            for (nb = 0; bad < 0 && nb < 8 * nbuf * W; ++nb)
                for (int wave = 0; bad < 0 && wave < W; ++wave) bad = play_stream(nbuf, W, loads, wave, nb, old != 0);
            if (bad < 0) std::puts("ok");
            else std::printf("block %d of %d\n", bad, nb - 1);
        } else {
            return 1;
        }
    }
    return 0;
}
