// Exchanges and sums among the lanes of a wave.
#pragma once

#include "mx.h"

namespace dmm {

// A value of another lane of 16, by the data-parallel moves: 0xb1 and 0x4e are
// lanes ^ 1 and ^ 2; 0x141 and 0x140 mirror 8 and 16 lanes, which brings the other
// half's value once all lanes of a half have the same.
template <int CTRL, class T>
__device__ __forceinline__ T moved(T v) {
    static_assert(sizeof(T) == 4, "one register");
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// f of a value and the one 16 lanes on or back (32), for a symmetric f: of two copies, the
// odd rows of one change places with the even rows of the other.
template <int D, class T, class F>
__device__ __forceinline__ T with_row(T v, F f) {
    static_assert(sizeof(T) == 4 && (D == 16 || D == 32), "rows of 16 lanes");
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    if (D == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        return f(__builtin_bit_cast(T, (uint32_t)p[0]), __builtin_bit_cast(T, (uint32_t)p[1]));
    }
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return f(__builtin_bit_cast(T, (uint32_t)p[0]), __builtin_bit_cast(T, (uint32_t)p[1]));
}

// f over the values of each L lanes (a power of two), in all of them.
template <int L, class T, class F>
__device__ __forceinline__ T over_group(T v, F f) {
    if (L >= 2) v = f(v, moved<0xb1>(v));
    if (L >= 4) v = f(v, moved<0x4e>(v));
    if (L >= 8) v = f(v, moved<0x141>(v));
    if (L >= 16) v = f(v, moved<0x140>(v));
    if (L >= 32) v = with_row<16>(v, f);
    if (L >= 64) v = with_row<32>(v, f);
    return v;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
    return over_group<L>(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
    return over_group<L>(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Eight values of a row from element `at` on (any alignment of their type), `have` of
// them there; the others are `fill`.  STREAM: what is read once, past the caches.
template <bool BF16, bool STREAM = false>
__device__ __forceinline__ void load_row8(const void* base, int64_t at, int have, float* v, float fill) {
    if (have >= 8) {
        if (BF16) {
            const u32x4h* const p = (const u32x4h*)((const uint16_t*)base + at);
            const u32x4 d = STREAM ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __builtin_bit_cast(float, d[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, d[i] & 0xffff0000u);
            }
        } else {
            const f32x4a* const p = (const f32x4a*)((const float*)base + at);
            const f32x4a* const q = (const f32x4a*)((const float*)base + at + 4);
            const f32x4 a = STREAM ? __builtin_nontemporal_load(p) : *p, b = STREAM ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = fill;
        if (i < have)
            v[i] = BF16 ? bf16_bits_to_f32(((const uint16_t*)base)[at + i]) : ((const float*)base)[at + i];
    }
}

// The first `have` of eight values to a row, from element `at` on; bf16 rounds to nearest, ties to
// even.  STREAM: what is not read soon, past the caches.
template <bool BF16, bool STREAM = false>
__device__ __forceinline__ void store_row8(void* base, int64_t at, int have, const float* v) {
    if (BF16) {
        uint16_t* const d = (uint16_t*)base + at;
        if (have >= 8) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
            if (STREAM) __builtin_nontemporal_store(w, (u32x4h*)d);
            else *(u32x4h*)d = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) d[i] = f32_to_bf16_rne(v[i]);
        }
    } else {
        float* const d = (float*)base + at;
        if (have >= 8) {
            const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (STREAM) {
                __builtin_nontemporal_store(lo, (f32x4a*)d);
                __builtin_nontemporal_store(hi, (f32x4a*)(d + 4));
            } else {
                *(f32x4a*)d = lo;
                *(f32x4a*)(d + 4) = hi;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) d[i] = v[i];
        }
    }
}

// Lanes of a row of E values, eight each.
inline int row_lanes(int E) {
    int L = 1;
    while (8 * L < E) L *= 2;
    return L;
}

}  // namespace dmm
