// moe_combine and moe_combine_grad: the experts' rows of a token into one, and back.
//
// Mathematics.  out[t] = sum_j w[t, j] y[t, j] (+ add[t]) over the slots that have an
// expert, in fp32, in the slots' order; dy[t, j] = w[t, j] dout[t] and dw[t, j] =
// sum_n dout[t, n] y[t, j, n].
//
// Bound: memory, a multiply and an addition a value.  2048 tokens top 8, 4096 columns, bf16: 29.1 us
// (5.1 TB/s), with the gradients 88.7 (4.9 TB/s); 16 tokens 3.1, the launch and one latency.
#include "lanes.h"

namespace dmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// kAtOnce slots' rows are on their way at once.
constexpr int kAtOnce = 8;

template <bool YBF16, bool OBF16>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a, int64_t pieces) {
    const int64_t t = blockIdx.x / pieces, n = ((blockIdx.x - t * pieces) * blockDim.x + threadIdx.x) * 8;
    const int64_t left = a.N - n;
    const int have = left < 8 ? (int)left : 8;
    if (have <= 0) return;
    float sum[8];
    if (a.add) {
        load_row8<OBF16>(a.add, t * a.N + n, have, sum, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    }
    for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
        float y[kAtOnce][8], w[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t slot = t * a.top_k + j0 + j;
            const bool some = j0 + j < a.top_k && (uint32_t)a.ids[slot] < (uint32_t)a.n_experts;
            w[j] = some ? a.weights[slot] : 0.f;
            load_row8<YBF16, true>(a.y, slot * a.N + n, some ? have : 0, y[j], 0.f);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], y[j][i], sum[i]);
    }
    store_row8<OBF16>(a.out, t * a.N + n, have, sum);
}

// A workgroup a slot.
template <bool YBF16, bool OBF16>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(CombineGradArgs a) {
    __shared__ float part[kWaves];
    const int64_t slot = blockIdx.x, t = slot / a.top_k;
    const bool some = (uint32_t)a.ids[slot] < (uint32_t)a.n_experts;
    const float w = some ? a.weights[slot] : 0.f;
    float dot = 0.f;
    for (int64_t n = (int64_t)threadIdx.x * 8; n < a.N; n += kThreads * 8) {
        const int have = a.N - n < 8 ? (int)(a.N - n) : 8;
        float y[8], d[8];
        load_row8<YBF16, true>(a.y, slot * a.N + n, some ? have : 0, y, 0.f);
        load_row8<OBF16>(a.dout, t * a.N + n, some ? have : 0, d, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dot = __builtin_fmaf(y[i], d[i], dot);
            d[i] *= w;
        }
        store_row8<YBF16, true>(a.dy, slot * a.N + n, have, d);
    }
    dot = group_sum<64>(dot);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = part[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) dot += part[i];
        a.dweights[slot] = dot;
    }
}

}  // namespace

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t s) {
    // few tokens: a wave a workgroup, to have more compute units at work
    const int64_t wide = (a.N + kThreads * 8 - 1) / (kThreads * 8);
    const int threads = a.M * wide < 2 * compute_unit_count() ? 64 : kThreads;
    const int64_t pieces = (a.N + threads * 8 - 1) / (threads * 8), blocks = a.M * pieces;
    if (!grid_fits(a.M * wide, kThreads)) return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, threads, 0, s>>>(a, pieces);
        return hipGetLastError();
    };
    if (a.y_dtype == TQ_BF16)
        return a.o_dtype == TQ_BF16 ? go(combine_kernel<true, true>) : go(combine_kernel<true, false>);
    return a.o_dtype == TQ_BF16 ? go(combine_kernel<false, true>) : go(combine_kernel<false, false>);
}

hipError_t launch_moe_combine_grad(const CombineGradArgs& a, hipStream_t s) {
    const int64_t blocks = a.M * a.top_k;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a);
        return hipGetLastError();
    };
    if (a.y_dtype == TQ_BF16)
        return a.o_dtype == TQ_BF16 ? go(combine_grad_kernel<true, true>) : go(combine_grad_kernel<true, false>);
    return a.o_dtype == TQ_BF16 ? go(combine_grad_kernel<false, true>) : go(combine_grad_kernel<false, false>);
}

}  // namespace dmm
