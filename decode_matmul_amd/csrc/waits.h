// How many of a wave's loads may be outstanding where the e4m3 products wait for what they read
// next.  Loads land in the order in which they were sent for, so a count is right where at least that many
// were sent for behind the last one that is needed.  Plain C++: a test plays the queues
// of all forms on the CPU.
#pragma once

namespace dmm {

// Tiles: x loads of x and w of W a slab, `stages` slabs under way.  A tile begins with W of all
// stages, then x of all stages; later a slab's x and W go together (early: W and the first half of x
// at the middle of the slab whose stage they take, the rest at its end).
struct StageQueue {
    int stages, x, w;
    bool early;
    // Before slab 0.  x of the last stage only: the counts behind the slabs suppose whole slabs one
    // behind the other, and would not wait for x of stages whose W came long before.
    constexpr int begin() const { return x; }
    // Behind slab t, when all up to slab t + stages - 1 (early: the first part of slab t + stages too)
    // were sent for: slab t + 1 has landed.
    constexpr int slab() const { return (stages - 2) * (x + w) + (early ? w + x - x / 2 : 0); }
};

// Streaming: a wave's blocks are c, c + W, ..; the first NBUF were sent for whether they are there (of nb) or
// not, and block c + NBUF W goes once block c is multiplied.  How many blocks were sent for behind
// block c when it is waited for.
constexpr int blocks_behind(int c, int W, int NBUF, int nb) {
    const int sent = nb > NBUF * W ? nb : NBUF * W;
    int n = 0;
    while (n < NBUF - 1 && c + (n + 1) * W < sent) ++n;
    return n;
}

}  // namespace dmm
