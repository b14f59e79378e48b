// Which tile of a product a workgroup takes: dense, or of the experts' lists.
#pragma once

#include "mx.h"

namespace dmm {

// The workgroup's tile: its tokens are positions [m0, m_end) of the batch or
// of the order list, its rows of W start at n0.
struct Place {
    int64_t m0, m_end, n0, expert;
};

// Tile t of mt tiles of rows by nt along N, in groups of GM tiles of rows that take the
// tiles along N in turn and share the rows of W (GM = 1: the tiles along N innermost).
template <int GM>
__device__ inline void in_groups(int64_t t, int64_t mt, int64_t nt, int64_t& m, int64_t& n) {
    const int64_t grp = t / (GM * nt), m8 = grp * GM, gm = mt - m8 < GM ? mt - m8 : GM;
    const int64_t in = t - m8 * nt;
    m = m8 + in % gm;
    n = in / gm;
}

// Tile b of the experts' tiles: experts in turn, an expert's tiles of BM
// positions and BN rows of W in groups of GM; each XCD gets a contiguous
// share of the tiles that there are.  False when there are fewer: then m0 is the
// workgroup's number among the m_end that have none.
template <int BM, int BN, int GM, int kThreads, class Args>
__device__ bool place_grouped(const Args& a, Place& p) {
    __shared__ int found[4];
    __shared__ int sums[kThreads / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slots = (int)(a.M * a.top_k);
    const int ntiles = (int)((a.N + BN - 1) / BN);
    // bounds of the list of expert e, kept in range whatever the offsets hold
    auto bound = [&](int e) {
        const int o = a.offsets[e];
        return o < 0 ? 0 : (o > slots ? slots : o);
    };
    if (tid == 0) found[2] = -1;
    // An expert's tiles and those before it: experts e0 .. e0 + kThreads - 1, one a thread.
    int first = 0, last = 0, n = 0, mine = 0;
    auto scan = [&](int e0, int before) {
        const int e = e0 + tid;
        n = 0;
        if (e < a.n_experts) {
            first = bound(e);
            last = bound(e + 1);
            n = last > first ? (last - first + BM - 1) / BM : 0;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 63) sums[wave] = inc;
        __syncthreads();
        int all = before;
        mine = before + inc - n;
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w < wave) mine += sums[w];
            all += sums[w];
        }
        return all;
    };
    int total = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += kThreads) {
        if (e0 > 0) __syncthreads();
        total = scan(e0, total);
    }
    total = readfirstlane(total);
    const int64_t all = (int64_t)total * ntiles;
    const int64_t b = blockIdx.x;
    // XCD b % 8 takes tiles all * (b % 8) / 8 .. all * (b % 8 + 1) / 8 - 1
    const int64_t x = b % 8, lo = all * x / 8, hi = all * (x + 1) / 8;
    const int64_t t = lo + b / 8;
    if (t >= hi) {
        const int64_t cap = gridDim.x / 8;      // of an XCD
        p.m0 = cap * x - lo + t - hi;
        p.m_end = cap * 8 - all;
        return false;
    }
    const int want = readfirstlane((int)(t / ntiles));
    int before = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += kThreads) {
        if (a.n_experts > kThreads) {           // otherwise the one scan is at hand
            __syncthreads();
            before = scan(e0, before);
        }
        if (want >= mine && want < mine + n) {
            int64_t m, nt;
            in_groups<GM>(t - (int64_t)mine * ntiles, n, ntiles, m, nt);
            found[0] = first + (int)m * BM;
            found[1] = last;
            found[3] = (int)nt;
            found[2] = e0 + tid;
        }
    }
    __syncthreads();
    p.m0 = readfirstlane(found[0]);
    const int64_t end = readfirstlane(found[1]);
    // (overlapping lists can have more tiles than an int counts: no thread or two may have the tile)
    if (readfirstlane(found[2]) < 0 || end <= p.m0) {
        p.m0 = p.m_end = a.M * a.top_k;
        return false;
    }
    p.m_end = end < p.m0 + BM ? end : p.m0 + BM;
    p.n0 = (int64_t)readfirstlane(found[3]) * BN;
    p.expert = readfirstlane(found[2]);
    return true;
}

// Rows of slots of no expert: NaN.  A workgroup without a tile takes every step-th
// from number `first` on; there are at least as many of them as those slots make tiles.
template <class Args>
__device__ void write_nan_rows(const Args& a, int64_t first, int64_t step, int threads) {
    const int64_t slots = a.M * a.top_k, begin = a.offsets[a.n_experts];
    for (int64_t i = (begin < 0 ? 0 : begin) + first; i < slots; i += step) {
        const int64_t slot = a.order[i];
        if (slot < 0 || slot >= slots) continue;
        for (int64_t n = threadIdx.x; n < a.N; n += threads) {
            if (a.y_dtype == TQ_F32) ((float*)a.y)[slot * a.N + n] = __builtin_nanf("");
            else ((uint16_t*)a.y)[slot * a.N + n] = 0x7fc0u;
        }
    }
}

// Dense: groups of 8 tiles along M share the rows of W; each XCD takes a contiguous range.
template <int BM, int BN, class Args>
__device__ Place place_dense(const Args& a) {
    const int64_t mt = (a.M + BM - 1) / BM, nt = (a.N + BN - 1) / BN;
    const int64_t t = xcd_block(blockIdx.x, mt * nt);
    int64_t m, n;
    in_groups<8>(t, mt, nt, m, n);
    Place p;
    p.m0 = m * BM;
    p.n0 = n * BN;
    p.m_end = p.m0 + BM < a.M ? p.m0 + BM : a.M;
    p.expert = 0;
    return p;
}

// Workgroups of the experts' tiles: whole shares of the 8 XCDs, the largest share has a tile
// more than an eighth.
template <int BM, class Args>
int64_t grouped_blocks(const Args& a, int64_t nt) {
    const int64_t slots = a.M * a.top_k;
    const int64_t tiles = (slots / BM + (a.n_experts < slots ? a.n_experts : slots)) * nt;
    return (tiles / 8 + 1) * 8;
}

}  // namespace dmm
