// Products of e4m3 packages:
//     y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in block b} cx[m, k] cw[n, k]  (+ bias[n]).
//
// Mathematics.  A block's 128 columns are four 16x16x32 bf16 matrix instructions (e4m3
// values are exact in bf16), whose sum starts at 0 and is added to y's with the product of
// the two scales, in fp32.  The e4m3 instructions lose bits of their sums: of each eight
// products those 2^-13 below the largest.
#include "f8.h"

namespace dmm {

namespace {

// The lane's 32 bytes of a block: 16-byte pieces g and 4 + g, zeros from column `kept` on.
__device__ __forceinline__ i32x8 operand(const uint8_t* block, int g, int kept) {
    u32x4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[h] = *(const u32x4*)(block + (4 * h + g) * 16);
        const int left = kept - (4 * h + g) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = left - 4 * i;
            v[h][i] &= n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        }
    }
    return (i32x8){(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w, (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
}

// A wave: 16 rows of W, 16 tokens (positions of an expert's list).
__global__ void __launch_bounds__(64) f8_matmul_kernel(F8MatmulArgs a) {
    const int lane = (int)threadIdx.x, r = lane & 15, g = lane >> 4;
    const int64_t nt = (a.N + 15) / 16, nb = (a.K + kF8Block - 1) / kF8Block;
    const int64_t by = blockIdx.x / nt, n0 = (blockIdx.x - by * nt) * 16;
    const int64_t slots = a.M * a.top_k;
    int64_t begin = by * 16, end = begin + 16 < a.M ? begin + 16 : a.M, expert = 0;
    if (a.n_experts > 0) {
        expert = by;
        begin = a.offsets[by];
        end = by < a.n_experts ? (int64_t)a.offsets[by + 1] : slots;
        begin = begin < 0 ? 0 : begin;
        end = end > slots ? slots : end;
    }
    const int64_t wrow = n0 + r < a.N ? n0 + r : a.N - 1;
    for (int64_t m0 = begin; m0 < end; m0 += 16) {
        const int64_t at = m0 + r < end ? m0 + r : end - 1;
        const int64_t slot = a.n_experts > 0 ? a.order[at] : at;
        const bool ok = slot >= 0 && slot < slots;
        const int64_t xrow = ok ? slot / a.top_k : 0;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        if (expert < a.n_experts || a.n_experts == 0) {
            for (int64_t b = 0; b < nb; ++b) {
                const int kept = a.K - b * kF8Block < kF8Block ? (int)(a.K - b * kF8Block) : kF8Block;
                const i32x8 w = operand(a.codes + ((expert * a.N + wrow) * nb + b) * kF8Block, g, kept);
                const i32x8 x = operand(a.x_codes + (xrow * nb + b) * kF8Block, g, kept);
                f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_bf16((uint32_t)w[i], (uint32_t)w[i + 1]),
                                                                   f8_bf16((uint32_t)x[i], (uint32_t)x[i + 1]), part, 0, 0, 0);
                const float s = a.x_scales[xrow * nb + b] * a.scales[(expert * ((a.N + 127) / 128) + n0 / 128) * nb + b];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s, part[i], acc[i]);
            }
        }
        if (!ok || m0 + r >= end) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + 4 * g + i;
            if (n >= a.N) continue;
            float y = acc[i];
            if (a.bias && (a.n_experts == 0 || expert < a.n_experts)) y += a.bias[expert * a.N + n];
            if (a.n_experts > 0 && expert == a.n_experts) y = __builtin_nanf("");
            if (a.y_dtype == TQ_F32) ((float*)a.y)[slot * a.N + n] = y;
            else ((uint16_t*)a.y)[slot * a.N + n] = f32_to_bf16_rne(y);
        }
    }
}

}  // namespace

hipError_t launch_f8_matmul(const F8MatmulArgs& a, hipStream_t s) {
    const int64_t nt = (a.N + 15) / 16, rows = a.n_experts > 0 ? (int64_t)a.n_experts + 1 : (a.M + 15) / 16;
    if (rows > (int64_t)0xffffffffll / 64 / nt) return hipErrorInvalidConfiguration;
    f8_matmul_kernel<<<(unsigned)(rows * nt), 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dmm
