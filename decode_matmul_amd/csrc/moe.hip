// The router's side of the grouped experts: moe_route (counts and lists of the
// slots of each expert) and moe_balance / moe_balance_grad.
#include "common.h"

namespace dmm {

namespace {

// ------------------------------------------------------------------ route
//
// A stable counting sort of the slots by expert; ids of no expert count as
// expert E.  The slots are cut into chunks of kChunk consecutive ones, a
// workgroup each, and a slot's place is
//     offset of its expert + slots of that expert in earlier chunks
//     + slots of that expert earlier in its chunk.
// Within a chunk wave w holds the w-th sixteenth, in rows of 64 consecutive
// slots: lanes with the same expert find each other by one ballot for each
// bit of the id, and a count per (wave, expert) in LDS carries on from row to
// row.  No place depends on the order in which anything runs.
//
// One chunk is one launch.  More take three: counts per chunk, their running
// sums over the chunks, places.
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRows = 4;                        // rows of 64 slots a wave
constexpr int kChunk = kRouteThreads * kRows;
constexpr int kScanThreads = 256;
static_assert(kMoeMaxExperts < kRouteThreads, "a thread for each expert and one for no expert");

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t slot, int64_t slots, int E) {
    if (slot >= slots) return -1;               // behind the last slot: counted nowhere
    const int id = ids[slot];
    return id >= 0 && id < E ? id : E;
}

// Lanes of the wave with this lane's id (0 <= id <= E), out of those in `live`.
__device__ __forceinline__ uint64_t same_id(int id, uint64_t live, int bits) {
    uint64_t m = live;
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((id >> b) & 1);
        m &= ((id >> b) & 1) ? v : ~v;
    }
    return m;
}

// Exclusive sums of v over the workgroup's threads (kRouteThreads >= E + 1);
// `sums` holds kRouteWaves words.
__device__ __forceinline__ int exclusive_sum(int v, int* sums) {
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
    for (int w = 0; w < wave; ++w) before += sums[w];
    return before + inc - v;
}

// SINGLE: the only chunk.  Otherwise `before` [chunks + 1][E + 1] holds each
// chunk's running sums, the last row the totals.
template <bool SINGLE>
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const int32_t* ids, int64_t slots, int E,
                                                                    int bits, const int32_t* before,
                                                                    int64_t chunks, int32_t* counts,
                                                                    int32_t* offsets, int32_t* order) {
    extern __shared__ int lds[];                // [kRouteWaves][E + 1] counts, then places; kRouteWaves sums
    int* const sums = lds + kRouteWaves * (E + 1);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, tid = (int)threadIdx.x;
    for (int i = tid; i < kRouteWaves * (E + 1); i += kRouteThreads) lds[i] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kChunk + wave * (64 * kRows) + lane;
    int id[kRows], rank[kRows];
    // volatile: a row's places are read after the row before wrote them, by other lanes of the wave
    volatile int* const mine = lds + wave * (E + 1);
#pragma unroll
    for (int i = 0; i < kRows; ++i) id[i] = expert_of(ids, first + 64 * i, slots, E);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t same = same_id(id[i], __ballot(id[i] >= 0), bits);
        const int below = __popcll(same & ((1ull << lane) - 1ull));
        const int base = id[i] >= 0 ? mine[id[i]] : 0;
        rank[i] = base + below;
        if (id[i] >= 0 && below == 0) mine[id[i]] = base + __popcll(same);
    }
    __syncthreads();
    // thread e: the chunk's count of expert e, its total, and what earlier chunks hold
    int total = 0, earlier = 0;
    if (tid <= E) {
        if (SINGLE) {
            for (int w = 0; w < kRouteWaves; ++w) total += lds[w * (E + 1) + tid];
        } else {
            total = before[chunks * (E + 1) + tid];
            earlier = before[(int64_t)blockIdx.x * (E + 1) + tid];
        }
    }
    const int offset = exclusive_sum(total, sums);
    if (tid <= E) {
        if (blockIdx.x == 0) {
            offsets[tid] = offset;
            if (tid < E) counts[tid] = total;
        }
        int at = offset + earlier;
        for (int w = 0; w < kRouteWaves; ++w) {
            const int v = lds[w * (E + 1) + tid];
            lds[w * (E + 1) + tid] = at;
            at += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (id[i] >= 0) order[mine[id[i]] + rank[i]] = (int32_t)(first + 64 * i);
}

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const int32_t* ids, int64_t slots, int E,
                                                                    int32_t* chunk_counts) {
    extern __shared__ int lds[];                // [E + 1]
    const int tid = (int)threadIdx.x;
    for (int i = tid; i <= E; i += kRouteThreads) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int id = expert_of(ids, (int64_t)blockIdx.x * kChunk + i * kRouteThreads + tid, slots, E);
        if (id >= 0) atomicAdd(&lds[id], 1);    // whole numbers: any order gives the same count
    }
    __syncthreads();
    for (int i = tid; i <= E; i += kRouteThreads) chunk_counts[(int64_t)blockIdx.x * (E + 1) + i] = lds[i];
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
// loss = sum_t s_t with s_t = sum_e w_e p_te; the gradient of s_t is
// p_te (w_e - s_t).  A wave takes a row: lane l holds logits l, l + 64, ..
// (at most 8), so the row is read once; the maximum and the two sums are
// exchanged over the wave.  Bound: the logits' bytes.
constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;
constexpr int kWeightThreads = 1024;
constexpr int kBalRows = 16;                    // rows a wave of the loss takes

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// A row's softmax p (PER values a lane) and s = sum_e w_e p_e.  Rows of -inf give p = 0.
template <bool BF16, int PER>
__device__ __forceinline__ float row_softmax(const void* logits, int64_t at, int E, const float* w, float* p) {
    const int lane = (int)threadIdx.x & 63;
    float top = -__builtin_inff();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        p[i] = -__builtin_inff();
        if (e < E)
            p[i] = BF16 ? bf16_bits_to_f32(((const uint16_t*)logits)[at + e]) : ((const float*)logits)[at + e];
        nan |= p[i] != p[i];
        top = fmaxf(top, p[i]);
    }
    top = wave_max(top);
    if (__ballot(nan) != 0ull) top = __builtin_nanf("");
    if (top == -__builtin_inff()) {
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] = 0.f;
        return 0.f;
    }
    float sum = 0.f, ws = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        p[i] = expf(p[i] - top);
        sum += p[i];
        ws += w[i] * p[i];
    }
    sum = wave_sum(sum);
    ws = wave_sum(ws);
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] *= inv;
    return ws * inv;
}

// w_e from the counts and the number of tokens that take part.
__global__ void __launch_bounds__(kWeightThreads) balance_weights_kernel(const uint8_t* mask, int64_t M, int E,
                                                                      const int32_t* counts, float* weights) {
    __shared__ double part[2][kWeightThreads / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    double T = 0.0, n = tid < E ? (double)counts[tid] : 0.0;
    if (mask)
        for (int64_t t = tid; t < M; t += kWeightThreads) T += mask[t] != 0 ? 1.0 : 0.0;
    T = wave_sum(T);
    n = wave_sum(n);
    if (lane == 0) {
        part[0][wave] = T;
        part[1][wave] = n;
    }
    __syncthreads();
    T = n = 0.0;
    for (int w = 0; w < kWeightThreads / 64; ++w) {
        T += part[0][w];
        n += part[1][w];
    }
    if (!mask) T = (double)M;
    if (tid < E) weights[tid] = T > 0.0 && n > 0.0 ? (float)((double)E / T * ((double)counts[tid] / n)) : 0.f;
}

template <bool BF16, int PER>
__global__ void __launch_bounds__(kBalThreads) balance_loss_kernel(const void* logits, int64_t M, int E, int64_t ldl,
                                                                   const uint8_t* mask, const float* weights,
                                                                   double* partial) {
    __shared__ double part[kBalWaves];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    float w[PER], p[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) w[i] = lane + 64 * i < E ? weights[lane + 64 * i] : 0.f;
    double sum = 0.0;
    const int64_t t0 = ((int64_t)blockIdx.x * kBalWaves + wave) * kBalRows;
    for (int i = 0; i < kBalRows; ++i) {
        const int64_t t = t0 + i;
        if (t >= M || (mask && mask[t] == 0)) continue;
        sum += (double)row_softmax<BF16, PER>(logits, t * ldl, E, w, p);
    }
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < kBalWaves; ++i) s += part[i];
        partial[blockIdx.x] = s;
    }
}

__global__ void __launch_bounds__(kBalThreads) balance_sum_kernel(const double* partial, int64_t n, float* loss) {
    __shared__ double part[kBalWaves];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kBalThreads) s += partial[i];
    s = wave_sum(s);
    if (((int)threadIdx.x & 63) == 0) part[(int)threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int i = 0; i < kBalWaves; ++i) s += part[i];
        loss[0] = (float)s;
    }
}

template <bool BF16, int PER>
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const void* logits, int64_t M, int E, int64_t ldl,
                                                                   const uint8_t* mask, const float* weights,
                                                                   const float* dloss, void* dlogits) {
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kBalWaves + wave;
    if (t >= M) return;
    float w[PER], p[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        w[i] = lane + 64 * i < E ? weights[lane + 64 * i] : 0.f;
        p[i] = 0.f;
    }
    float s = 0.f, up = 0.f;
    if (!mask || mask[t] != 0) {
        s = row_softmax<BF16, PER>(logits, t * ldl, E, w, p);
        up = dloss[0];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        const float d = up * p[i] * (w[i] - s);
        if (BF16) ((uint16_t*)dlogits)[t * E + e] = f32_to_bf16_rne(d);
        else ((float*)dlogits)[t * E + e] = d;
    }
}

int64_t route_chunks(int64_t slots) { return (slots + kChunk - 1) / kChunk; }

int64_t loss_blocks(int64_t M) { return (M + kBalWaves * kBalRows - 1) / (kBalWaves * kBalRows); }

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
        route_place_kernel<true><<<1, kRouteThreads, lds, s>>>(ids, slots, E, bits, nullptr, 1, counts, offsets,
                                                              order);
        return hipGetLastError();
    }
    int32_t* const cc = (int32_t*)workspace;
    route_count_kernel<<<(unsigned)chunks, kRouteThreads, (size_t)(E + 1) * 4, s>>>(ids, slots, E, cc);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_scan_kernel<<<(unsigned)(E + 1), kScanThreads, 0, s>>>(cc, chunks, E);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<false><<<(unsigned)chunks, kRouteThreads, lds, s>>>(ids, slots, E, bits, cc, chunks, counts,
                                                                          offsets, order);
    return hipGetLastError();
}

int64_t moe_balance_ws_bytes(int64_t M, int) { return loss_blocks(M) * 8; }

template <bool BF16, int PER>
static hipError_t balance(const void* logits, int64_t M, int E, int64_t ldl, const uint8_t* mask, float* weights,
                          double* partial, float* loss, hipStream_t s) {
    const int64_t blocks = loss_blocks(M);
    if (blocks > 0) {
        balance_loss_kernel<BF16, PER><<<(unsigned)blocks, kBalThreads, 0, s>>>(logits, M, E, ldl, mask, weights,
                                                                               partial);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    balance_sum_kernel<<<1, kBalThreads, 0, s>>>(partial, blocks, loss);
    return hipGetLastError();
}

template <bool BF16, int PER>
static hipError_t grad(const void* logits, int64_t M, int E, int64_t ldl, const uint8_t* mask, const float* weights,
                       const float* dloss, void* dlogits, hipStream_t s) {
    if (!grid_fits((M + kBalWaves - 1) / kBalWaves, kBalThreads)) return hipErrorInvalidConfiguration;
    balance_grad_kernel<BF16, PER><<<(unsigned)((M + kBalWaves - 1) / kBalWaves), kBalThreads, 0, s>>>(
        logits, M, E, ldl, mask, weights, dloss, dlogits);
    return hipGetLastError();
}

hipError_t launch_moe_balance(const void* logits, int l_dtype, int64_t M, int E, int64_t ldl, const uint8_t* mask,
                              const int32_t* counts, float* loss, float* weights, void* workspace, hipStream_t s) {
    balance_weights_kernel<<<1, kWeightThreads, 0, s>>>(mask, M, E, counts, weights);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    double* const part = (double*)workspace;
    const bool bf = l_dtype == TQ_BF16;
#define DMM_BALANCE(PER)                                                                     \
    return bf ? balance<true, PER>(logits, M, E, ldl, mask, weights, part, loss, s)          \
              : balance<false, PER>(logits, M, E, ldl, mask, weights, part, loss, s)
    if (E <= 64) DMM_BALANCE(1);
    if (E <= 256) DMM_BALANCE(4);
    DMM_BALANCE(8);
#undef DMM_BALANCE
}

hipError_t launch_moe_balance_grad(const void* logits, int l_dtype, int64_t M, int E, int64_t ldl,
                                   const uint8_t* mask, const float* weights, const float* dloss, void* dlogits,
                                   hipStream_t s) {
    const bool bf = l_dtype == TQ_BF16;
#define DMM_GRAD(PER)                                                                        \
    return bf ? grad<true, PER>(logits, M, E, ldl, mask, weights, dloss, dlogits, s)         \
              : grad<false, PER>(logits, M, E, ldl, mask, weights, dloss, dlogits, s)
    if (E <= 64) DMM_GRAD(1);
    if (E <= 256) DMM_GRAD(4);
    DMM_GRAD(8);
#undef DMM_GRAD
}

}  // namespace dmm
