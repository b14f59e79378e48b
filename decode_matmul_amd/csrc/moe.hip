// The router's side of the grouped experts: moe_route (counts and lists of the
// slots of each expert) and moe_balance / moe_balance_grad.
#include <type_traits>

#include "lanes.h"

namespace dmm {

namespace {

// ------------------------------------------------------------------ route
//
// A stable counting sort of the slots by expert; ids of no expert count as
// expert E.  The slots are cut into chunks of kChunk consecutive ones, a
// workgroup each, and a slot's place is
//     offset of its expert + slots of that expert in earlier chunks
//     + slots of that expert earlier in its chunk.
// Within a chunk wave w holds the w-th quarter, in rows of 64 consecutive
// slots: lanes with the same expert find each other by one ballot for each
// bit of the id, and a count per (wave, expert) in LDS carries on from row to
// row.  No place depends on the order in which anything runs.
//
// Bound: latency.  One chunk takes one launch.  Up to kSumChunks take two, the
// counts of each chunk and the places, for which a workgroup sums the counts
// itself; more take three, the counts' running sums over the chunks in between.
// (16384 slots of 64 experts: 15.2 us with one launch of 4 workgroups that each
// count everything.)
constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRows = 4;                        // rows of 64 slots a wave
constexpr int kChunk = kRouteThreads * kRows;
constexpr int kSumChunks = 64;
constexpr int kScanThreads = 256;

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t slot, int64_t slots, int E) {
    if (slot >= slots) return -1;               // behind the last slot: counted nowhere
    const int id = ids[slot];
    return id >= 0 && id < E ? id : E;
}

// Exclusive sums of v over the workgroup's threads, and the sum of all; `sums`
// holds kRouteWaves words and is free again after the next barrier.
__device__ __forceinline__ int exclusive_sum(int v, int* sums, int& all) {
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    return before + inc - v;
}

enum RouteChunks { kOnly, kSummed, kScanned };

// kOnly: the only chunk.  kSummed: cc [chunks][E + 1] holds the chunks' counts.
// kScanned: cc [chunks + 1][E + 1] holds each chunk's running sums, the last row
// the totals.
template <RouteChunks MODE>
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const int32_t* ids, int64_t slots, int E,
                                                                    int bits, const int32_t* cc, int chunks,
                                                                    int32_t* counts, int32_t* offsets,
                                                                    int32_t* order) {
    extern __shared__ int lds[];                // [kRouteWaves][E + 1] counts, then places; kRouteWaves sums
    int* const sums = lds + kRouteWaves * (E + 1);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, tid = (int)threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * kChunk + wave * (64 * kRows) + lane;
    int id[kRows], rank[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) id[i] = expert_of(ids, first + 64 * i, slots, E);
    // expert e's slots in all chunks, and in earlier ones
    auto gather = [&](int e, int& total, int& earlier) {
        total = earlier = 0;
        if (e > E) return;
        if (MODE == kOnly) {
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) total += lds[w * (E + 1) + e];
        } else if (MODE == kSummed) {
#pragma unroll 8
            for (int c = 0; c < chunks; ++c) {
                const int v = cc[c * (E + 1) + e];
                total += v;
                if (c < (int)blockIdx.x) earlier += v;
            }
        } else {
            total = cc[(int64_t)chunks * (E + 1) + e];
            earlier = cc[(int64_t)blockIdx.x * (E + 1) + e];
        }
    };
    int total = 0, earlier = 0;
    if (MODE != kOnly) gather(tid, total, earlier);         // on its way meanwhile
    // lanes of the wave with this lane's id, in each row
    uint64_t same[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) same[i] = __ballot(id[i] >= 0);
    for (int b = 0; b < bits; ++b)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const bool one = (id[i] >> b) & 1;
            const uint64_t v = __ballot(one);
            same[i] &= one ? v : ~v;
        }
    for (int i = tid; i < kRouteWaves * (E + 1); i += kRouteThreads) lds[i] = 0;
    __syncthreads();
    // volatile: a row's places are read after the row before wrote them, by other lanes of the wave
    volatile int* const mine = lds + wave * (E + 1);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int below = __popcll(same[i] & ((1ull << lane) - 1ull));
        const int base = id[i] >= 0 ? mine[id[i]] : 0;
        rank[i] = base + below;
        if (id[i] >= 0 && below == 0) mine[id[i]] = base + __popcll(same[i]);
    }
    __syncthreads();
    int carry = 0;                              // slots of the experts below e0
    for (int e0 = 0; e0 <= E; e0 += kRouteThreads) {
        const int e = e0 + tid;
        if (MODE == kOnly || e0 > 0) gather(e, total, earlier);
        int all;
        const int offset = carry + exclusive_sum(total, sums, all);
        carry += all;
        if (e <= E) {
            if (blockIdx.x == 0) {
                offsets[e] = offset;
                if (e < E) counts[e] = total;
            }
            int at = offset + earlier;
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) {
                const int v = lds[w * (E + 1) + e];
                lds[w * (E + 1) + e] = at;
                at += v;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (id[i] >= 0) order[mine[id[i]] + rank[i]] = (int32_t)(first + 64 * i);
}

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const int32_t* ids, int64_t slots, int E,
                                                                    int32_t* cc) {
    extern __shared__ int lds[];                // [E + 1]
    const int tid = (int)threadIdx.x;
    int id[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        id[i] = expert_of(ids, (int64_t)blockIdx.x * kChunk + i * kRouteThreads + tid, slots, E);
    for (int i = tid; i <= E; i += kRouteThreads) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (id[i] >= 0) atomicAdd(&lds[id[i]], 1);      // whole numbers: any order gives the same count
    __syncthreads();
    for (int i = tid; i <= E; i += kRouteThreads) cc[(int64_t)blockIdx.x * (E + 1) + i] = lds[i];
}

// Column e = blockIdx.x of the chunks' counts -> its running sums, the total
// in row `chunks`.
__global__ void __launch_bounds__(kScanThreads) route_scan_kernel(int32_t* cc, int64_t chunks, int E) {
    __shared__ int part[kScanThreads / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int carry = 0;
    for (int64_t c0 = 0; c0 < chunks; c0 += kScanThreads) {
        const int64_t c = c0 + tid;
        const int v = c < chunks ? cc[c * (E + 1) + blockIdx.x] : 0;
        int inc = v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 63) part[wave] = inc;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kScanThreads / 64; ++w) {
            if (w < wave) inc += part[w];
            all += part[w];
        }
        if (c < chunks) cc[c * (E + 1) + blockIdx.x] = carry + inc - v;
        carry += all;
        __syncthreads();
    }
    if (tid == 0) cc[chunks * (E + 1) + blockIdx.x] = carry;
}

// ---------------------------------------------------------------- balance
//
// The loss is E / (n T) times the sum over tokens of s_t = sum_e c_e p_te, so
// tokens, T and n are counted in one pass, and the gradient of a token's part is
// p_te (w_e - sum_j w_j p_tj) with w = E c / (n T).  A row's E logits lie with L
// lanes (a power of two, 64 / L rows a wave at a time), eight consecutive ones each,
// read once; the maximum and the two sums are exchanged among the L lanes.
// Bound: about as many vector instructions as the logits' bytes take time (65536
// x 128 bf16: a dozen for each logit, three more in the gradient; 9.6 and 8.1 us in a
// replayed graph); the launches for few tokens.
constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;

// Eight weights or counts (within 2^-24) from w[0] on, `have` of them there; the others are 0.
template <class T>
__device__ __forceinline__ void load_weights(const T* w, int have, float* v) {
    typedef T Four __attribute__((ext_vector_type(4)));
    typedef Four FourAt __attribute__((aligned(4)));
    if (have >= 8) {
        const Four a = *(const FourAt*)w, b = *(const FourAt*)(w + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (float)a[i];
            v[4 + i] = (float)b[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < have ? (float)w[i] : 0.f;
}

// A row's logits to e = exp(z - top), 1 / sum e and sum w p.  False for a row of
// -inf only, which has no softmax.  The maximum is the one that keeps a NaN, which
// then takes the whole row; so does an infinity (inf - inf).
template <int L>
__device__ __forceinline__ bool row_softmax(float* e, const float* w, float& inv, float& s) {
    float top = e[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __builtin_elementwise_maximum(top, e[i]);
    top = group_max<L>(top);
    float sum = 0.f, ws = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // off by about (top - z) 2^-24 of itself, the rounding of its argument, and a unit
        e[i] = __builtin_amdgcn_exp2f((e[i] - top) * 1.44269504088896340736f);
        sum += e[i];
        ws = __builtin_fmaf(w[i], e[i], ws);
    }
    inv = __builtin_amdgcn_rcpf(group_sum<L>(sum));     // a unit off
    s = group_sum<L>(ws) * inv;
    return top != -__builtin_inff();
}

// loss and weights from the sum of s_t over tokens, their number T, and the counts, whose sum is n.
__device__ __forceinline__ void finish_balance(double sum, int64_t T, double n, int E, const int32_t* counts,
                                               float* loss, float* weights) {
    const bool some = T > 0 && n > 0.0;
    for (int e = (int)threadIdx.x; e < E; e += kBalThreads)
        weights[e] = some ? (float)((double)E * ((double)counts[e] / n) / (double)T) : 0.f;
    if (threadIdx.x == 0) loss[0] = some ? (float)(sum / (double)T * ((double)E / n)) : 0.f;
}

// Tokens of a workgroup of the loss: kTokens for each group of L lanes, all of
// their logits on their way before the first is used.
constexpr int kTokens = 4;
constexpr int loss_rows(int L) { return kTokens * kBalThreads / L; }

// partial [blocks][2]: the sum over a workgroup's tokens and how many take part;
// the only workgroup finishes by itself.
template <bool BF16, int L>
__global__ void __launch_bounds__(kBalThreads) balance_loss_kernel(const void* logits, int64_t M, int E, int64_t ldl,
                                                                   const uint8_t* mask, const int32_t* counts,
                                                                   float* loss, float* weights, double* partial) {
    __shared__ double part[3][kBalWaves];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int e0 = (lane % L) * 8, have = E - e0;
    float z[kTokens][8], w[8];
    bool live[kTokens];
    const int64_t t0 = (int64_t)blockIdx.x * loss_rows(L) + (int)threadIdx.x / L;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t t = t0 + i * (kBalThreads / L);
        live[i] = t < M;
        load_row8<BF16>(logits, live[i] ? t * ldl + e0 : 0, live[i] ? have : 0, z[i], -__builtin_inff());
        if (mask && live[i]) live[i] = mask[t] != 0;
    }
    load_weights(counts + e0, have, w);
    double sum = 0.0;
    int tokens = 0;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        float inv, s;
        if (row_softmax<L>(z[i], w, inv, s) && live[i]) sum += (double)s;
        tokens += __popcll(__ballot(live[i] && lane % L == 0));
    }
#pragma unroll
    for (int d = 32; d >= L; d >>= 1) sum += __shfl_xor(sum, d);        // the lanes of a row have the same
    if (lane == 0) {
        part[0][wave] = sum;
        part[1][wave] = (double)tokens;
    }
    const bool only = gridDim.x == 1;
    if (only) {
        double n = 0.0;
        for (int e = (int)threadIdx.x; e < E; e += kBalThreads) n += (double)counts[e];
        n = wave_sum(n);
        if (lane == 0) part[2][wave] = n;
    }
    __syncthreads();
    double v[3] = {0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        for (int i = 0; i < kBalWaves && (k < 2 || only); ++i) v[k] += part[k][i];
    if (only) {
        finish_balance(v[0], (int64_t)v[1], v[2], E, counts, loss, weights);
    } else if (threadIdx.x == 0) {
        partial[2 * (int64_t)blockIdx.x] = v[0];
        partial[2 * (int64_t)blockIdx.x + 1] = v[1];
    }
}

__global__ void __launch_bounds__(kBalThreads) balance_finish_kernel(const double* partial, int64_t blocks, int E,
                                                                     const int32_t* counts, float* loss,
                                                                     float* weights) {
    __shared__ double part[3][kBalWaves];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    double v[3] = {0.0, 0.0, 0.0};
    for (int64_t i = threadIdx.x; i < blocks; i += kBalThreads) {
        v[0] += partial[2 * i];
        v[1] += partial[2 * i + 1];
    }
    for (int e = (int)threadIdx.x; e < E; e += kBalThreads) v[2] += (double)counts[e];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = wave_sum(v[k]);
        if (lane == 0) part[k][wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = 0.0;
        for (int i = 0; i < kBalWaves; ++i) v[k] += part[k][i];
    }
    finish_balance(v[0], (int64_t)v[1], v[2], E, counts, loss, weights);
}

template <bool BF16, int L>
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const void* logits, int64_t M, int E, int64_t ldl,
                                                                   const uint8_t* mask, const float* weights,
                                                                   const float* dloss, void* dlogits) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t t = ((int64_t)blockIdx.x * kBalThreads + threadIdx.x) / L;
    const int e0 = (lane % L) * 8, have = E - e0;
    if (t >= M) return;
    float w[8], p[8];
    load_row8<BF16>(logits, t * ldl + e0, have, p, -__builtin_inff());
    load_weights(weights + e0, have, w);
    const bool live = !mask || mask[t] != 0;
    float inv, s;
    const bool some = row_softmax<L>(p, w, inv, s);
    // w_e - s, of a token that has chosen its expert, is far below the rounding of s:
    // what s is off by comes back as the mean of the differences and is taken off again
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] -= s;
        off = __builtin_fmaf(w[i], p[i], off);
    }
    off = group_sum<L>(off) * inv;
    const float up = dloss[0] * inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = up * p[i] * (w[i] - off);
    if (!(some && live)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = 0.f;
    }
    store_row8<BF16>(dlogits, t * E + e0, have, p);
}

int64_t route_chunks(int64_t slots) { return (slots + kChunk - 1) / kChunk; }

static_assert(kMoeMaxExperts <= 64 * 8, "a row fits a wave");

int64_t loss_blocks(int64_t M, int E) {
    const int rows = loss_rows(row_lanes(E));
    return M == 0 ? 1 : (M + rows - 1) / rows;
}

template <bool BF16, int L>
hipError_t balance(const void* logits, int64_t M, int E, int64_t ldl, const uint8_t* mask, const int32_t* counts,
                   float* loss, float* weights, double* partial, hipStream_t s) {
    const int64_t blocks = loss_blocks(M, E);
    balance_loss_kernel<BF16, L><<<(unsigned)blocks, kBalThreads, 0, s>>>(logits, M, E, ldl, mask, counts, loss,
                                                                         weights, partial);
    hipError_t e = hipGetLastError();
    if (blocks == 1 || e != hipSuccess) return e;
    balance_finish_kernel<<<1, kBalThreads, 0, s>>>(partial, blocks, E, counts, loss, weights);
    return hipGetLastError();
}

template <bool BF16, int L>
hipError_t grad(const void* logits, int64_t M, int E, int64_t ldl, const uint8_t* mask, const float* weights,
                const float* dloss, void* dlogits, hipStream_t s) {
    const int64_t blocks = (M * L + kBalThreads - 1) / kBalThreads;
    if (!grid_fits(blocks, kBalThreads)) return hipErrorInvalidConfiguration;
    balance_grad_kernel<BF16, L><<<(unsigned)blocks, kBalThreads, 0, s>>>(logits, M, E, ldl, mask, weights, dloss,
                                                                         dlogits);
    return hipGetLastError();
}

// f(integral constant L) for the lanes a row of E logits takes.
template <class F>
hipError_t with_lanes(int E, F f) {
    switch (row_lanes(E)) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 4: return f(std::integral_constant<int, 4>());
        case 8: return f(std::integral_constant<int, 8>());
        case 16: return f(std::integral_constant<int, 16>());
        case 32: return f(std::integral_constant<int, 32>());
        default: return f(std::integral_constant<int, 64>());
    }
}

}  // namespace

int64_t moe_route_ws_bytes(int64_t slots, int E) {
    const int64_t chunks = route_chunks(slots);
    return chunks <= 1 ? 0 : (chunks + 1) * (E + 1) * 4;
}

hipError_t launch_moe_route(const int32_t* ids, int64_t slots, int E, int32_t* counts, int32_t* offsets,
                            int32_t* order, void* workspace, hipStream_t s) {
    const int64_t chunks = route_chunks(slots);
    const int bits = 32 - __builtin_clz((unsigned)E);
    const size_t lds = (size_t)(kRouteWaves * (E + 1) + kRouteWaves) * 4;
    if (chunks <= 1) {
        route_place_kernel<kOnly><<<1, kRouteThreads, lds, s>>>(ids, slots, E, bits, nullptr, 1, counts, offsets,
                                                               order);
        return hipGetLastError();
    }
    int32_t* const cc = (int32_t*)workspace;
    route_count_kernel<<<(unsigned)chunks, kRouteThreads, (size_t)(E + 1) * 4, s>>>(ids, slots, E, cc);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (chunks <= kSumChunks) {
        route_place_kernel<kSummed><<<(unsigned)chunks, kRouteThreads, lds, s>>>(ids, slots, E, bits, cc, (int)chunks,
                                                                                counts, offsets, order);
        return hipGetLastError();
    }
    route_scan_kernel<<<(unsigned)(E + 1), kScanThreads, 0, s>>>(cc, chunks, E);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<kScanned><<<(unsigned)chunks, kRouteThreads, lds, s>>>(ids, slots, E, bits, cc, (int)chunks,
                                                                             counts, offsets, order);
    return hipGetLastError();
}

int64_t moe_balance_ws_bytes(int64_t M, int E) {
    const int64_t blocks = loss_blocks(M, E);
    return !grid_fits(blocks, kBalThreads) ? -1 : blocks == 1 ? 0 : blocks * 16;
}

hipError_t launch_moe_balance(const void* logits, int l_dtype, int64_t M, int E, int64_t ldl, const uint8_t* mask,
                              const int32_t* counts, float* loss, float* weights, void* workspace, hipStream_t s) {
    double* const part = (double*)workspace;
    return with_lanes(E, [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        return l_dtype == TQ_BF16 ? balance<true, L>(logits, M, E, ldl, mask, counts, loss, weights, part, s)
                                  : balance<false, L>(logits, M, E, ldl, mask, counts, loss, weights, part, s);
    });
}

hipError_t launch_moe_balance_grad(const void* logits, int l_dtype, int64_t M, int E, int64_t ldl,
                                   const uint8_t* mask, const float* weights, const float* dloss, void* dlogits,
                                   hipStream_t s) {
    return with_lanes(E, [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        return l_dtype == TQ_BF16 ? grad<true, L>(logits, M, E, ldl, mask, weights, dloss, dlogits, s)
                                  : grad<false, L>(logits, M, E, ldl, mask, weights, dloss, dlogits, s);
    });
}

}  // namespace dmm
