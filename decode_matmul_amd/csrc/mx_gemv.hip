// MXFP4 products, weight-streaming form: y[m, n] = sum_k x[m, k] w_hat[n, k] (+ bias[n]).
//
// Mathematics.  A block of 32 weights is 16 code bytes and one scale byte, so
// 128 weights of 16 rows are exactly one 16-byte load and one byte a lane:
// lane (r, g) = (lane % 16, lane / 16) takes block 4 s + g of row n0 + r.  That
// is the operand layout of the 16x16x128 scaled matrix instruction, which
// takes MXFP4 activations loaded the same way (mx_matmul_mx).  For bf16
// activations the hardware turns eight codes and their scale into eight exact
// bf16 values (four conversions), and the four octets of the lane's block go
// through four 16x16x32 bf16 matrix instructions; the sum over k may be taken
// in any order, so octet j pairs w[n, 32 b + 8 j ..] with x[m, 32 b + 8 j ..].
//
// Bound: the package's bytes.  The waves of a workgroup share 16 rows and
// take the 128-wide steps of K in turn (few tokens leave no other work to
// spread over the chip); their sums meet in LDS, in wave order.
#include "mx.h"

namespace dmm {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// One lane's eight activations at column k of a row (past K they are 0).
__device__ __forceinline__ u32x4 load_x8(const uint16_t* row, int64_t k, int64_t K) {
    if (k + 8 <= K) return *(const u32x4h*)(row + k);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
    return v;
}

// MXX: activations in MXFP4.  MT: 16-token tiles of a workgroup.
template <bool MXX, int MT, bool GROUPED>
__global__ void __launch_bounds__(kThreads) mx_gemv_kernel(MxMatmulArgs a) {
    __shared__ f32x4 red[kWaves][MT][64];
    const int lane = (int)threadIdx.x & 63, wave = readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t nb = (a.K + 31) / 32, steps = (nb + 3) / 4;
    const int64_t ntiles = (a.N + 15) / 16, by = blockIdx.x / ntiles;
    const int64_t n0 = (blockIdx.x - by * ntiles) * 16;
    const int64_t n = n0 + r < a.N ? n0 + r : a.N - 1;          // rows past N repeat the last
    const int64_t expert = GROUPED ? by : 0;

    int64_t begin = 0, end = a.M;                               // tokens, or positions in the order list
    const int64_t slots = a.M * a.top_k;
    if (GROUPED) {
        begin = a.offsets[expert];
        end = expert < a.n_experts ? (int64_t)a.offsets[expert + 1] : slots;
        begin = begin < 0 ? 0 : begin;
        end = end > slots ? slots : end;
        if (expert == a.n_experts) {                            // slots of no expert
            for (int64_t i = begin * 16 + threadIdx.x; i < end * 16; i += kThreads) {
                const int64_t slot = a.order[i >> 4], col = n0 + (i & 15);
                if (slot < 0 || slot >= slots || col >= a.N) continue;
                if (a.y_dtype == TQ_F32) ((float*)a.y)[slot * a.N + col] = __builtin_nanf("");
                else ((uint16_t*)a.y)[slot * a.N + col] = 0x7fc0u;
            }
            return;
        }
    } else {
        begin = by * (16 * MT);
        end = begin + 16 * MT < a.M ? begin + 16 * MT : a.M;
    }
    const uint8_t* const wc = a.codes + (expert * a.N + n) * nb * 16;
    const uint8_t* const ws = a.scales + (expert * a.N + n) * nb;

    for (int64_t t0 = begin; t0 < end; t0 += 16 * MT) {
        // this lane's tokens: row of x, and whether it is there
        int64_t row[MT];
        bool there[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t t = t0 + 16 * i + r;
            there[i] = t < end;
            row[i] = there[i] ? t : 0;
            if (GROUPED && there[i]) {
                const int64_t slot = a.order[t];
                there[i] = slot >= 0 && slot < slots;
                row[i] = there[i] ? slot / a.top_k : 0;
            }
        }
        f32x4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        for (int64_t s = wave; s < steps; s += kWaves) {
            const int64_t b = 4 * s + g;
            const bool in = b < nb;
            u32x4 c = {0u, 0u, 0u, 0u};
            uint32_t sb = 127u;
            if (in) {
                c = *(const u32x4*)(wc + b * 16);
                sb = ws[b];
            }
            if (MXX) {
                const i32x8 A = mx_operand(c);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    u32x4 xc = {0u, 0u, 0u, 0u};
                    uint32_t xs = 127u;
                    if (in && there[i]) {
                        xc = *(const u32x4*)(a.x_codes + (row[i] * nb + b) * 16);
                        xs = a.x_scales[row[i] * nb + b];
                    }
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, mx_operand(xc), acc[i], 4, 4, 0,
                                                                              (int)sb, 0, (int)xs);
                }
            } else {
                const float scale = e8m0_bits(sb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 w = mx_decode8(c[j], scale);
                    const int64_t k = b * 32 + j * 8;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        u32x4 xv = {0u, 0u, 0u, 0u};
                        if (there[i] && k < a.K) xv = load_x8(a.x + row[i] * a.ldx, k, a.K);
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, xv), acc[i],
                                                                         0, 0, 0);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        // lane (m, q) of tile i holds y[m, n0 + 4 q ..]
        if ((int)threadIdx.x < 64 * MT) {
            const int i = (int)threadIdx.x >> 6;
            f32x4 v = red[0][i][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += red[w][i][lane];
            const int64_t t = t0 + 16 * i + r;
            int64_t out = t;
            bool store = t < end;
            if (GROUPED && store) {
                out = a.order[t];
                store = out >= 0 && out < slots;
            }
            if (store) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t col = n0 + 4 * g + q;
                    if (col >= a.N) continue;
                    const float u = a.bias ? v[q] + a.bias[expert * a.N + col] : v[q];
                    if (a.y_dtype == TQ_F32) ((float*)a.y)[out * a.N + col] = u;
                    else ((uint16_t*)a.y)[out * a.N + col] = f32_to_bf16_rne(u);
                }
            }
        }
        __syncthreads();
    }
}

template <bool MXX, int MT, bool GROUPED>
hipError_t launch(const MxMatmulArgs& a, hipStream_t s) {
    const int64_t tiles = GROUPED ? a.n_experts + 1 : (a.M + 16 * MT - 1) / (16 * MT);
    const int64_t blocks = (a.N + 15) / 16 * tiles;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    mx_gemv_kernel<MXX, MT, GROUPED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t s) {
    const bool many = a.n_experts > 0 ? a.M * a.top_k >= 32 * (int64_t)a.n_experts : a.M > 64 && a.M * a.N >= (int64_t)64 << 16;
    if (many && mx_gemm_takes(a)) return launch_mx_gemm(a, s);
    if (a.n_experts > 0) return launch<false, 2, true>(a, s);
    if (a.x_codes) return a.M <= 16 ? launch<true, 1, false>(a, s) : launch<true, 4, false>(a, s);
    return a.M <= 16 ? launch<false, 1, false>(a, s) : launch<false, 4, false>(a, s);
}

}  // namespace dmm
