// moe_gate and moe_gate_grad: which experts a token goes to, with what weights, and the
// gradient of the weights.
//
// Mathematics.  p = softmax or sigmoid of the logits z; experts are chosen by c = p + bias,
// or, without a bias, by z, whose order is the same.  c is compared as float64 holds it.
// An expert whose logit or bias is -inf is not there.  NaN ranks above everything, equal
// values by index.
#include "lanes.h"

namespace dmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxGroups = 64;
constexpr int kEach = kMoeMaxExperts / 64;      // experts a lane, at most

// A float64 as an integer of the same order: 0 for an expert that is not there, NaN highest.
__device__ __forceinline__ uint64_t order_of(double c) {
    if (c != c) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, c + 0.0);       // one zero
    return (u >> 63) ? ~u : u | (1ull << 63);
}

// The largest key of the wave, of equal ones the lowest index.
__device__ __forceinline__ void wave_first(uint64_t& key, int& at) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint64_t k = (uint64_t)__shfl_xor((unsigned long long)key, d);
        const int i = __shfl_xor(at, d);
        if (k > key || (k == key && i < at)) {
            key = k;
            at = i;
        }
    }
}

__device__ __forceinline__ float logit(const GateArgs& a, int64_t at) {
    return a.l_dtype == TQ_BF16 ? bf16_bits_to_f32(((const uint16_t*)a.logits)[at]) : ((const float*)a.logits)[at];
}

// Token t by one wave; lds: n_experts doubles of its own.
__device__ void choose(const GateArgs& a, int64_t t, double* lds) {
    const int lane = (int)threadIdx.x & 63, E = a.E, size = E / a.n_groups;
    const bool live = !a.mask || a.mask[t] != 0;
    const bool by_score = a.bias || (a.n_groups > 1 && a.group_top > 1);
    float z[kEach];
    bool there[kEach];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = lane + 64 * i;
        z[i] = live && e < E ? logit(a, t * a.ldl + e) : -__builtin_inff();
        there[i] = z[i] != -__builtin_inff() && (!a.bias || a.bias[e] != -__builtin_inff());
        top = __builtin_elementwise_maximum(top, z[i]);
    }
    top = group_max<64>(top);
    // float64 scores
    double p[kEach];
    if (by_score) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            p[i] = 0.0;
            if (z[i] == -__builtin_inff()) continue;
            p[i] = a.score == DMM_SIGMOID ? 1.0 / (1.0 + exp(-(double)z[i])) : exp((double)z[i] - (double)top);
            sum += p[i];
        }
        if (a.score != DMM_SIGMOID) {
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < kEach; ++i) p[i] /= sum;
        }
    }
    uint64_t key[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = lane + 64 * i;
        key[i] = there[i] ? order_of(a.bias ? p[i] + (double)a.bias[e] : (double)z[i]) : 0ull;
    }
    if (a.n_groups > 1) {
        // what a group's score is made of
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
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
        for (int i = 0; i < kEach; ++i) {
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
        for (int i = 0; i < kEach; ++i)
            if (key[i] > k) {
                k = key[i];
                at = lane + 64 * i;
            }
        wave_first(k, at);
        if (k == 0ull) break;
        if (lane == j) mine = at;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
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
            for (int i = 0; i < kEach; ++i)
                if (z[i] != -__builtin_inff()) sum += expf(z[i] - m);
        }
        w /= group_sum<64>(sum);
    }
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = mine;
        a.weights[t * a.top_k + lane] = has ? w * a.scale : 0.f;
    }
}

__global__ void __launch_bounds__(kThreads) gate_kernel(GateArgs a) {
    __shared__ double lds[kWaves][kMoeMaxExperts];
    const int wave = readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t < a.M) choose(a, t, lds[wave]);
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
constexpr int kSlots = kGateMaxTopK / 8;        // slots a lane of eight, at most

template <bool BF16, int L>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(GateGradArgs a) {
    const int lane = (int)threadIdx.x & 63, l = lane % L;
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
    if (t >= a.M) return;                       // all L lanes alike
    const int E = a.E, e0 = l * 8, have = E - e0;
    const bool dense = a.score != DMM_SIGMOID && !a.renorm;
    // this lane's slots
    int id[kSlots];
    float zj[kSlots], dw[kSlots], v[kSlots];
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = l + i * L;
        id[i] = j < a.top_k ? a.ids[t * a.top_k + j] : -1;
        if ((uint32_t)id[i] >= (uint32_t)E) id[i] = -1;
        dw[i] = id[i] >= 0 ? a.dweights[t * a.top_k + j] : 0.f;
        zj[i] = -__builtin_inff();
        if (id[i] >= 0)
            zj[i] = BF16 ? bf16_bits_to_f32(((const uint16_t*)a.logits)[t * a.ldl + id[i]])
                         : ((const float*)a.logits)[t * a.ldl + id[i]];
        m = __builtin_elementwise_maximum(m, zj[i]);
        v[i] = 0.f;
    }
    float z[8], p[8], g[8];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 0.f;
    int some = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) some |= id[i] >= 0;
    some = over_group<L>(some, [](int x, int y) { return x | y; });
    if (!some) {                                // a masked token, whatever its logits hold
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
            p[i] = z[i] == -__builtin_inff() ? 0.f : expf(z[i] - top);
            sum += p[i];
        }
        sum = group_sum<L>(sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = sum > 0.f || sum != sum ? p[i] / sum : 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) v[i] = a.scale * dw[i];
    } else {
        m = group_max<L>(m);
        const bool sigmoid = a.score == DMM_SIGMOID;
        const float base = sigmoid ? (m < 0.f ? m : 0.f) : m;
        float q[kSlots], rest[kSlots], sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            q[i] = rest[i] = 0.f;
            if (id[i] < 0 || zj[i] == -__builtin_inff()) continue;
            const float up = expf(-__builtin_fabsf(zj[i]));         // e^-|z|
            rest[i] = sigmoid ? (zj[i] > 0.f ? up / (1.f + up) : 1.f / (1.f + up)) : 1.f;   // 1 - p
            if (!sigmoid) q[i] = expf(zj[i] - base);
            else if (zj[i] > 0.f) q[i] = 1.f / (1.f + up);
            else q[i] = (a.renorm ? expf(zj[i] - base) : up) / (1.f + up);
            sum += q[i];
        }
        if (a.renorm) {
            sum = group_sum<L>(sum);
            float mean = 0.f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                if (id[i] >= 0) q[i] /= sum;
                mean += q[i] * dw[i];
            }
            mean = group_sum<L>(mean);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                dw[i] -= mean;
                off += q[i] * dw[i];
            }
            off = group_sum<L>(off);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) dw[i] -= off;
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) v[i] = q[i] != 0.f || q[i] != q[i] ? a.scale * q[i] * dw[i] * rest[i] : 0.f;
    }
    // slots in order to the experts they name
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (i * L >= a.top_k) break;
        const int n = a.top_k - i * L < L ? a.top_k - i * L : L;
        for (int j = 0; j < n; ++j) {
            const int from = lane - l + j;
            const int e = __shfl(id[i], from) - e0;
            const float x = __shfl(v[i], from);
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] += e == k ? x : 0.f;
        }
    }
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
hipError_t grad(const GateGradArgs& a, hipStream_t s) {
    const int64_t blocks = (a.M * L + kThreads - 1) / kThreads;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    gate_grad_kernel<BF16, L><<<(unsigned)blocks, kThreads, 0, s>>>(a);
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
    const int64_t blocks = (a.M + kWaves - 1) / kWaves;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    gate_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_gate_grad(const GateGradArgs& a, hipStream_t s) {
    return a.l_dtype == TQ_BF16 ? grad_by_lanes<true>(a, s) : grad_by_lanes<false>(a, s);
}

}  // namespace dmm
