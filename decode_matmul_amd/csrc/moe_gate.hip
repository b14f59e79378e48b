// moe_gate and moe_gate_grad: which experts a token goes to, with what weights, and the
// gradient of the weights.
//
// Mathematics.  p = softmax or sigmoid of the logits z; experts are chosen by c = p + bias,
// or, without a bias, by z, whose order is the same.  c is compared as float64 holds it.
// An expert whose logit or bias is -inf is not there.  NaN ranks above everything, equal
// values by index.
//
// Form.  Nearly always fp32 decides the order: a token takes L lanes of a wave, eight
// experts each, and its choices come one after another as the largest of 32-bit keys, the
// distance from the token's best in fixed point above the index (gate_kernel).  Where two
// choices next to each other, or the last and the first that is not chosen, lie within the
// error of that, the wave takes the token again in float64 (choose).  bf16 logits without a
// bias fit a key as they are.  Groups that do not fit a wave take float64 throughout
// (gate_exact_kernel).
//
// Bound: the vector instructions of the choice, a dozen for each choice and token and forty
// to sort each lane's experts, beside the logits' bytes; for few tokens the chain of launch, loads
// and choices.  us in a replayed graph, top 8: 65536 tokens x 128 experts bf16 11.9 (its logits' bytes
// at a copy's rate take 3.2), fp32 12.5, by sigmoid with a bias 19.8 (16.1 without the few dozen
// tokens that float64 decides, whose waves end last); 64 experts 10.7; 32768 x 256 in eight groups 29.5
// (21.4); 16 x 256 in eight groups 4.8.  In float64 throughout: 119 for the first, 90 for 64 experts,
// 172 for 65536 x 480 in forty groups (73 to 76 in 32, which fit a wave).  The gradient of the first: 8.5,
// its bytes 6.5; by whole rows 12.3, of fp32 logits 13.3 and 13.8.
//
// What float64 decides costs a wave's time each.  fp32 logits without a bias go there where two of the first
// top_k + 1 are equal or a chosen one lies 16 and more below the best; 65536 x 128 in us: normal logits
// 13.5, times 8 20, times 16 52, rounded to bf16's values 41, all equal 70 (bf16 logits 11 in all of these).
#include "lanes.h"

namespace dmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxGroups = 64;

// A float64 as an integer of the same order: 0 for an expert that is not there, NaN highest.
__device__ __forceinline__ uint64_t order_of(double c) {
    if (c != c) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, c + 0.0);       // one zero
    return (u >> 63) ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return a < b ? a : b; }

// The largest key of the wave, of equal ones the lowest index.
__device__ __forceinline__ void wave_first(uint64_t& key, int& at) {
    const uint32_t hi = over_group<64>((uint32_t)(key >> 32), larger);
    const uint32_t lo = over_group<64>((uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u, larger);
    const uint64_t first = (uint64_t)hi << 32 | lo;
    at = (int)over_group<64>(key == first ? (uint32_t)at : 0xffffffffu, smaller);
    key = first;
}

__device__ __forceinline__ float logit(const GateArgs& a, int64_t at) {
    return a.l_dtype == TQ_BF16 ? bf16_bits_to_f32(((const uint16_t*)a.logits)[at]) : ((const float*)a.logits)[at];
}

// e^x by the hardware's exp2, off by |x| 2^-24 of itself, the rounding of its argument, and a unit.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// Token t by one wave, EACH experts a lane; lds: n_experts doubles of its own.
template <int EACH>
__device__ __forceinline__ void choose(const GateArgs& a, int64_t t, double* lds) {
    const int lane = (int)threadIdx.x & 63, E = a.E, size = E / a.n_groups;
    const bool live = !a.mask || a.mask[t] != 0;
    const bool by_score = a.bias || (a.n_groups > 1 && a.group_top > 1);
    float z[EACH];
    bool there[EACH];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = lane + 64 * i;
        z[i] = live && e < E ? logit(a, t * a.ldl + e) : -__builtin_inff();
        there[i] = z[i] != -__builtin_inff() && (!a.bias || a.bias[e] != -__builtin_inff());
        top = __builtin_elementwise_maximum(top, z[i]);
    }
    top = group_max<64>(top);
    // float64 scores
    double p[EACH];
    if (by_score) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            p[i] = 0.0;
            if (z[i] == -__builtin_inff()) continue;
            p[i] = a.score == DMM_SIGMOID ? 1.0 / (1.0 + exp(-(double)z[i])) : exp((double)z[i] - (double)top);
            sum += p[i];
        }
        if (a.score != DMM_SIGMOID) {
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < EACH; ++i) p[i] /= sum;
        }
    }
    uint64_t key[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = lane + 64 * i;
        key[i] = there[i] ? order_of(a.bias ? p[i] + (double)a.bias[e] : (double)z[i]) : 0ull;
    }
    if (a.n_groups > 1) {
        // what a group's score is made of
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int e = lane + 64 * i;
            if (e < E)
                lds[e] = !there[i] ? -(double)__builtin_inff()
                         : a.bias  ? p[i] + (double)a.bias[e]
                                   : (by_score ? p[i] : (double)z[i]);
        }
        asm volatile("" ::: "memory");          // a wave's LDS accesses happen in order
        uint64_t score = 0ull;
        if (lane < a.n_groups) {
            double first = -(double)__builtin_inff(), second = first;
            bool nan = false;
#pragma unroll 8
            for (int i = 0; i < size; ++i) {
                const double v = lds[lane * size + i];
                nan |= v != v;
                if (v > first) {
                    second = first;
                    first = v;
                } else if (v > second) {
                    second = v;
                }
            }
            if (a.group_top > 1 && size > 1) first += second;
            score = nan ? ~0ull : order_of(first);
        }
        uint64_t kept = 0ull;
        for (int j = 0; j < a.top_groups; ++j) {
            uint64_t k = score;
            int at = lane;
            wave_first(k, at);
            kept |= 1ull << at;
            if (lane == at) score = 0ull;
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int e = lane + 64 * i;
            if (e < E && !((kept >> (e / size)) & 1)) key[i] = 0ull;
        }
        asm volatile("" ::: "memory");
    }
    // lane j takes the j-th choice
    int mine = -1;
    for (int j = 0; j < a.top_k; ++j) {
        uint64_t k = 0ull;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (key[i] > k) {
                k = key[i];
                at = lane + 64 * i;
            }
        wave_first(k, at);
        if (k == 0ull) break;
        if (lane == j) mine = at;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (lane + 64 * i == at) key[i] = 0ull;
    }
    // weights in fp32
    const bool has = mine >= 0;
    const float zj = has ? logit(a, t * a.ldl + mine) : -__builtin_inff();
    float w;
    if (a.score == DMM_SIGMOID) {
        if (a.renorm) {
            // p e^-m with m = min(0, the largest chosen logit): never 0 for all
            float m = group_max<64>(zj);
            m = m < 0.f ? m : 0.f;
            w = zj > 0.f ? 1.f / (1.f + expf(-zj)) : expf(zj - m) / (1.f + expf(zj));
            if (!has) w = 0.f;
            w /= group_sum<64>(w);
        } else {
            w = 1.f / (1.f + expf(-zj));
        }
    } else {
        const float m = a.renorm ? group_max<64>(zj) : top;
        w = has ? expf(zj - m) : 0.f;
        float sum = w;
        if (!a.renorm) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (z[i] != -__builtin_inff()) sum += expf(z[i] - m);
        }
        w /= group_sum<64>(sum);
    }
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = mine;
        a.weights[t * a.top_k + lane] = has ? w * a.scale : 0.f;
    }
}

__global__ void __launch_bounds__(kThreads) gate_exact_kernel(GateArgs a) {
    __shared__ double lds[kWaves][kMoeMaxExperts];
    const int wave = readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t < a.M) choose<kMoeMaxExperts / 64>(a, t, lds[wave]);
}

// Eight keys in falling order (19 exchanges, of odd and even merges).
__device__ __forceinline__ void sort8(uint32_t* k) {
    auto cx = [&](int i, int j) {
        const uint32_t hi = k[i] > k[j] ? k[i] : k[j], lo = k[i] > k[j] ? k[j] : k[i];
        k[i] = hi;
        k[j] = lo;
    };
    cx(0, 1), cx(2, 3), cx(4, 5), cx(6, 7);
    cx(0, 2), cx(1, 3), cx(4, 6), cx(5, 7);
    cx(1, 2), cx(5, 6);
    cx(0, 4), cx(1, 5), cx(2, 6), cx(3, 7);
    cx(2, 4), cx(3, 5);
    cx(1, 2), cx(3, 4), cx(5, 6);
}

// A token by L lanes, a group of experts by 2^shift of them (without groups: all), whose places
// l 8 + i are in the experts' order.  A key is Q - (best - x) S, with x = c or z in fp32, above the place:
// 32 - log2(8 L) bits of fixed point over W below the best.  Keys further down share the
// least one.  (A bf16 z: its 16 bits, of the same order.)  Eight waves a SIMD, at the price of a few
// registers that choose spills: 65536 x 128 bf16 12.5 -> 11.9 us, 160 experts in eight groups 28 -> 26.
template <bool BF16, int L>
__global__ void __launch_bounds__(kThreads, 8) gate_kernel(GateArgs a, int shift) {
    constexpr int kBits = L == 8 ? 6 : L == 16 ? 7 : L == 32 ? 8 : 9;       // of the place
    constexpr uint32_t kMask = 8 * L - 1, kQ = 0xffffffffu >> kBits;
    __shared__ double lds[kWaves][kMoeMaxExperts];
    const int lane = (int)threadIdx.x & 63, l = lane % L;
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
    const bool live = t < a.M && (!a.mask || a.mask[t] != 0);
    const int size = a.E / a.n_groups, S = 1 << shift, group = l >> shift, in = (l & (S - 1)) * 8;
    const int e0 = group * size + in, have = group < a.n_groups ? size - in : 0;
    const bool sigmoid = a.score == DMM_SIGMOID, grouped = a.n_groups > 1;
    const bool by_score = a.bias || (grouped && a.group_top > 1);
    const float none = -__builtin_inff();
    float z[8], b[8];
    load_row8<BF16>(a.logits, live ? t * a.ldl + e0 : 0, live ? have : 0, z, none);
    if (a.bias) load_row8<false>(a.bias, e0, have, b, none);
    float top = z[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __builtin_elementwise_maximum(top, z[i]);
    top = group_max<L>(top);
    // fp32 scores; inv is 1 / (sum of e^(z - top)) of a softmax
    float x[8], inv = 1.f, best = top;
    if (!sigmoid && (by_score || !a.renorm)) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_amdgcn_exp2f((z[i] - top) * 1.44269504088896340736f);
            sum += z[i] == none ? 0.f : x[i];
        }
        inv = __builtin_amdgcn_rcpf(group_sum<L>(sum));
    }
    if (!by_score) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = z[i];
    } else {
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z[i] * -1.44269504088896340736f));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= inv;
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = b[i] == none ? none : x[i] + b[i];
        }
        best = none;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = z[i] == none ? none : x[i];
            best = __builtin_elementwise_maximum(best, x[i]);
        }
        best = group_max<L>(best);
    }
    // W = 2 for scores (p lies in [0, 1]), 16 for logits
    const bool whole = BF16 && !by_score;       // a key says all
    const float unit = (float)(1u << (32 - kBits - 1)) * (by_score ? 1.f : 0.125f);
    uint32_t k[8];
    if (whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = __builtin_bit_cast(uint32_t, x[i] + 0.f);        // one zero
            const uint32_t q = (u ^ ((uint32_t)((int)u >> 31) | 0x80000000u)) >> 16;
            k[i] = x[i] == none ? 0u : q << kBits | (kMask - (uint32_t)(l * 8 + i));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t down = (uint32_t)__builtin_fminf((best - x[i]) * unit, 4294967040.f);
            const uint32_t q = down < kQ ? kQ - down : 1u;
            k[i] = x[i] == none ? 0u : q << kBits | (kMask - (uint32_t)(l * 8 + i));
        }
    }
    sort8(k);
    // How far keys of values in the other order can lie apart.  Rounding and truncation keep the
    // order; scores are off by the error of p (sigmoid: 2^-21; softmax: p (d + 32) 2^-23 at a
    // distance d from the best, at most 2^-18 inv), of the sum and of the distance.
    const float err = (sigmoid ? 0x1p-21f : inv * 0x1p-18f) + (__builtin_fabsf(best) + 2.f) * 0x1p-23f;
    // (Beyond 2^30, for a bias of 2^28 and more, no two keys are further apart: at most 2^27.)
    const uint32_t margin = by_score ? 2u + (uint32_t)__builtin_fminf(2.f * err * unit, 0x1p30f) : 0u;
    bool again = live && best != none && !(__builtin_fabsf(best) < __builtin_inff());    // NaN or +inf
    if (grouped) {
        // a group's score from the keys of its two best
        uint32_t m1 = k[0] >> kBits, m2 = k[1] >> kBits;
        auto merge = [&](uint32_t o1, uint32_t o2) {
            const uint32_t lo = m1 < o1 ? m1 : o1, hi2 = m2 > o2 ? m2 : o2;
            m1 = m1 > o1 ? m1 : o1;
            m2 = lo > hi2 ? lo : hi2;
        };
        if (S >= 2) merge(moved<0xb1>(m1), moved<0xb1>(m2));
        if (S >= 4) merge(moved<0x4e>(m1), moved<0x4e>(m2));
        if (S >= 8) merge(moved<0x141>(m1), moved<0x141>(m2));
        if (S >= 16) merge(moved<0x140>(m1), moved<0x140>(m2));
        if (S >= 32) merge((uint32_t)__shfl_xor((int)m1, 16), (uint32_t)__shfl_xor((int)m2, 16));
        // (kQ has at most 26 bits and n_groups is at most L: 27 + 6 bits would not fit, so the
        // group's number goes beside the score)
        const bool there = group < a.n_groups;
        uint32_t score = !there ? 0u : 1u + (a.group_top > 1 ? m1 + (size > 1 ? m2 : 0u) : m1);
        // fewer experts there than group_top counts (float64's -inf), or one below W
        again |= !whole && live && there && (m1 == 0u || (a.group_top > 1 && size > 1 && m2 <= 1u));
        bool kept = false;
        uint32_t last = 0u;
        for (int j = 0; j <= a.top_groups && j < a.n_groups; ++j) {
            const uint32_t s = over_group<L>(score, larger);
            const uint32_t g = over_group<L>(score == s ? (uint32_t)group : 0xffffu, smaller);
            if (j == a.top_groups) {
                again |= !whole && live && last - s <= 2u * margin;
            } else {
                last = s;
                if ((uint32_t)group == g) {
                    kept = true;
                    score = 0u;
                }
            }
        }
        if (!kept) {
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = 0u;
        }
    }
    // lane j keeps the j-th largest key, j <= top_k; a lane whose best it was moves up the `left`
    // that later rounds may want
    uint32_t mine = 0u;
    auto round = [&](int j, int left) {
        const uint32_t first = over_group<L>(k[0], larger);
        if (l == j) mine = first;
        const bool won = k[0] == first;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) k[i] = won ? (i < 7 ? k[i < 7 ? i + 1 : 7] : 0u) : k[i];
    };
    if (a.top_k <= 8) {
#pragma unroll
        for (int j = 0; j <= 8; ++j) {
            if (j > a.top_k) break;
            round(j, 8 - j);
        }
    } else {
        for (int j = 0; j <= a.top_k; ++j) round(j, 8);
    }
    const bool has = mine != 0u;
    const int place = (int)(kMask - (mine & kMask)), of = place >> (3 + shift);
    const int id = of * size + place - (of << (3 + shift));
    float zj = none;
    if (whole) {                                // the key has it
        const uint32_t q = mine >> kBits;
        zj = __builtin_bit_cast(float, ((q & 0x8000u) ? q ^ 0x8000u : q ^ 0xffffu) << 16);
    } else if (has) {
        zj = logit(a, t * a.ldl + id);
    }
    if (!whole) {
        const uint32_t next = (uint32_t)__shfl_down((int)mine, 1);  // in lane j + 1
        const bool near = next != 0u && (mine >> kBits) - (next >> kBits) <= margin;
        // (again: with groups a lane knows of its own only; the token's lanes agree, so that it is written once)
        const int any = again || (l < a.top_k && has && (near || (mine >> kBits) == 1u));
        again = over_group<L>(any, [](int p, int q) { return p | q; }) != 0;
    }
    const bool chosen = has && l < a.top_k;
    if (!chosen) zj = none;
    float w;
    if (sigmoid) {
        const float up = expf(-__builtin_fabsf(zj));            // e^-|z|
        if (a.renorm) {
            // p e^-m with m = min(0, the largest chosen logit): never 0 for all
            float m = group_max<L>(zj);
            m = m < 0.f ? m : 0.f;
            w = (zj > 0.f ? 1.f : expf(zj - m)) / (1.f + up);
            if (!chosen) w = 0.f;
            w /= group_sum<L>(w);
        } else {
            w = (zj > 0.f ? 1.f : up) / (1.f + up);
        }
    } else if (a.renorm) {
        const float m = group_max<L>(zj);
        w = chosen ? expf(zj - m) : 0.f;
        w /= group_sum<L>(w);
    } else {
        w = expf(zj - top) * inv;
    }
    if (t < a.M && l < a.top_k && !again) {
        a.ids[t * a.top_k + l] = chosen ? id : -1;
        a.weights[t * a.top_k + l] = chosen ? w * a.scale : 0.f;
    }
    uint64_t left = __ballot(again);
    const int wave = readfirstlane((int)threadIdx.x >> 6);
    while (left) {
        const int at = __builtin_ctzll(left) / L;
        choose<L / 8>(a, ((int64_t)blockIdx.x * kThreads + wave * 64) / L + at, lds[wave]);
        left &= L == 64 ? 0ull : ~(((1ull << (L & 63)) - 1ull) << (at * L));
    }
}

// --------------------------------------------------------------- gradient
//
// With q_j the chosen weights over their sum (renorm) and d_j = dw_j - sum_i q_i dw_i,
//     softmax, renorm   dz_j = scale q_j d_j
//     sigmoid, renorm   dz_j = scale q_j d_j (1 - p_j)
//     sigmoid           dz_j = scale dw_j p_j (1 - p_j)
//     softmax           dz_e = p_e (g_e - sum_i p_i g_i), g = scale dw at the chosen experts, else 0
// summed over the slots that name the expert.  Where one weight is nearly all, d is far
// below the rounding of its mean: what the mean is off by comes back as the mean of the
// differences and is taken off again.  A row of E logits lies with L lanes, eight
// consecutive ones each; the slots are dealt over the same lanes.
template <bool BF16, int L, int SLOTS>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(GateGradArgs a) {
    __shared__ __attribute__((aligned(16))) float rows[kWaves][8 * 64];     // of a wave's tokens
    const int lane = (int)threadIdx.x & 63, l = lane % L;
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
    if (t >= a.M) return;                       // all L lanes alike; nothing below crosses waves
    const int E = a.E, e0 = l * 8, have = E - e0;
    const bool dense = a.score != DMM_SIGMOID && !a.renorm;
    // this lane's slots
    int id[SLOTS], some = 0;
    float zj[SLOTS], dw[SLOTS], v[SLOTS];
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        const int j = l + i * L;
        id[i] = j < a.top_k ? a.ids[t * a.top_k + j] : -1;
        if ((uint32_t)id[i] >= (uint32_t)E) id[i] = -1;
        dw[i] = id[i] >= 0 ? a.dweights[t * a.top_k + j] : 0.f;
        zj[i] = -__builtin_inff();
        if (id[i] >= 0)
            zj[i] = BF16 ? bf16_bits_to_f32(((const uint16_t*)a.logits)[t * a.ldl + id[i]])
                         : ((const float*)a.logits)[t * a.ldl + id[i]];
        m = __builtin_elementwise_maximum(m, zj[i]);
        some |= id[i] >= 0;
        v[i] = 0.f;
    }
    float z[8], p[8], g[8];
    float off = 0.f;
    some = over_group<L>(some, [](int x, int y) { return x | y; });
    if (!some) {                                // a masked token, whatever its logits hold
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 0.f;
        store_row8<BF16>(a.dlogits, t * E + e0, have, g);
        return;
    }
    if (dense) {
        load_row8<BF16>(a.logits, t * a.ldl + e0, have, z, -__builtin_inff());
        float top = z[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = __builtin_elementwise_maximum(top, z[i]);
        top = group_max<L>(top);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = z[i] == -__builtin_inff() ? 0.f : exp_of(z[i] - top);
            sum += p[i];
        }
        sum = group_sum<L>(sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = sum > 0.f || sum != sum ? p[i] / sum : 0.f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) v[i] = a.scale * dw[i];
    } else {
        m = group_max<L>(m);
        const bool sigmoid = a.score == DMM_SIGMOID;
        const float base = sigmoid ? (m < 0.f ? m : 0.f) : m;
        float q[SLOTS], rest[SLOTS], sum = 0.f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            q[i] = rest[i] = 0.f;
            if (id[i] < 0 || zj[i] == -__builtin_inff()) continue;
            const float up = exp_of(-__builtin_fabsf(zj[i]));         // e^-|z|
            rest[i] = sigmoid ? (zj[i] > 0.f ? up / (1.f + up) : 1.f / (1.f + up)) : 1.f;   // 1 - p
            if (!sigmoid) q[i] = exp_of(zj[i] - base);
            else if (zj[i] > 0.f) q[i] = 1.f / (1.f + up);
            else q[i] = (a.renorm ? exp_of(zj[i] - base) : up) / (1.f + up);
            sum += q[i];
        }
        if (a.renorm) {
            sum = group_sum<L>(sum);
            float mean = 0.f;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (id[i] >= 0) q[i] /= sum;
                mean += q[i] * dw[i];
            }
            mean = group_sum<L>(mean);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                dw[i] -= mean;
                off += q[i] * dw[i];
            }
            off = group_sum<L>(off);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) dw[i] -= off;
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) v[i] = q[i] != 0.f || q[i] != q[i] ? a.scale * q[i] * dw[i] * rest[i] : 0.f;
    }
    // slots in order to the experts they name: a wave's LDS accesses happen in order
    float* const row = &rows[threadIdx.x >> 6][(lane - l) * 8];
    *(f32x4*)(row + e0) = *(f32x4*)(row + e0 + 4) = (f32x4){0.f, 0.f, 0.f, 0.f};
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
        for (int j = 0; j < L && j + i * L < a.top_k; ++j) {
            if (l == j && id[i] >= 0) __builtin_amdgcn_ds_faddf((__attribute__((address_space(3))) float*)(row + id[i]), v[i], 0, 0, false);
            asm volatile("" ::: "memory");
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = row[e0 + i];
    if (dense) {
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mean += p[i] * g[i];
        mean = group_sum<L>(mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] -= mean;
            off += p[i] * g[i];
        }
        off = group_sum<L>(off);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = p[i] * (g[i] - off);
    }
    store_row8<BF16>(a.dlogits, t * E + e0, have, g);
}

template <bool BF16, int L>
hipError_t gate(const GateArgs& a, int shift, hipStream_t s) {
    gate_kernel<BF16, L><<<(unsigned)((a.M * L + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, shift);
    return hipGetLastError();
}

template <bool BF16>
hipError_t gate_by_lanes(const GateArgs& a, hipStream_t s) {
    // a power of two of lanes for each group; lanes for all of them, and for one choice more than top_k
    int shift = 0;
    while ((8 << shift) < a.E / a.n_groups) ++shift;
    int L = 8;
    while (L < (a.n_groups << shift) || L <= a.top_k) L *= 2;
    if (a.n_groups == 1) shift = 6;             // the kernel's l has no more bits
    switch (L) {
        case 8: return gate<BF16, 8>(a, shift, s);
        case 16: return gate<BF16, 16>(a, shift, s);
        case 32: return gate<BF16, 32>(a, shift, s);
        case 64: return gate<BF16, 64>(a, shift, s);
        default:                                // groups that do not fit a wave
            gate_exact_kernel<<<(unsigned)((a.M + kWaves - 1) / kWaves), kThreads, 0, s>>>(a);
            return hipGetLastError();
    }
}

template <bool BF16, int L>
hipError_t grad(const GateGradArgs& a, hipStream_t s) {
    const int64_t blocks = (a.M * L + kThreads - 1) / kThreads;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    // a slot a lane, or as many as kGateMaxTopK needs
    constexpr int most = (kGateMaxTopK + L - 1) / L;
    if (most == 1 || a.top_k <= L) gate_grad_kernel<BF16, L, 1><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else gate_grad_kernel<BF16, L, most><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t grad_by_lanes(const GateGradArgs& a, hipStream_t s) {
    switch (row_lanes(a.E)) {
        case 16: return grad<BF16, 16>(a, s);
        case 32: return grad<BF16, 32>(a, s);
        case 64: return grad<BF16, 64>(a, s);
        default: return grad<BF16, 8>(a, s);
    }
}

}  // namespace

hipError_t launch_moe_gate(const GateArgs& a, hipStream_t s) {
    if (!grid_fits((a.M + kWaves - 1) / kWaves, kThreads)) return hipErrorInvalidConfiguration;
    return a.l_dtype == TQ_BF16 ? gate_by_lanes<true>(a, s) : gate_by_lanes<false>(a, s);
}

hipError_t launch_moe_gate_grad(const GateGradArgs& a, hipStream_t s) {
    return a.l_dtype == TQ_BF16 ? grad_by_lanes<true>(a, s) : grad_by_lanes<false>(a, s);
}

}  // namespace dmm
