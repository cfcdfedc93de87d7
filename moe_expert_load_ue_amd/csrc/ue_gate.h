// Choice of the k best experts of one token by one wave, shared by the gate
// kernel and the few-token layer.
//
// Ranks are compared as 32-bit keys that order like the floats they come
// from (negative values with all bits flipped, others with the sign bit
// set). -0 counts as +0, so that the two tie; -inf and NaN are below every
// key a round may take. Expert e = lane * V + i sits in slot i of its lane,
// so the lowest id among equal keys is the lowest lane's lowest slot.
#pragma once

#include "ue_internal.h"

namespace ue {

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // key of -inf: not taken

__device__ __forceinline__ uint32_t rank_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);          // -0 -> +0
    const uint32_t k = b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
    return x != x ? 0u : k;
}

__device__ __forceinline__ float bf16_to_f32(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Round to nearest even (one instruction on gfx950); NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// 1 / (1 + exp(-x)), and its slope without the cancellation of 1 - p.
__device__ __forceinline__ float sigmoid_of(float x) {
    return 1.0f / (1.0f + expf(-x));
}
__device__ __forceinline__ float sigmoid_slope(float x) {
    const float e = expf(-fabsf(x));
    return e / ((1.0f + e) * (1.0f + e));
}

// exp(x) within 4 u (u = 2^-24), 0 below 2^-126: through base 2, the product's
// rounding put back as a factor of 1 + r ln 2. (The instruction alone is off by
// 1.2 |x| u more.) The rest r means nothing where the product overflows: an
// exponential of 0 or infinity is taken as it is.
__device__ __forceinline__ float exp_of(float x) {
    constexpr float kLog2eHi = 1.44269502162933349609f;
    constexpr float kLog2eLo = 1.92596299112661746888e-8f;
    constexpr int kPositiveNormal = 0x100;
    const float t = x * kLog2eHi;
    const float r = __builtin_fmaf(x, kLog2eHi, -t) + x * kLog2eLo;
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_amdgcn_classf(e, kPositiveNormal)
               ? __builtin_fmaf(e, r * 0.693147180559945f, e) : e;
}

// v / (1 + exp(-v)) within 8 u where the exponential is finite, by the
// reciprocal instruction, one ulp (the full division and exponential took the
// gated product's epilogue 40 instructions per value, this takes 10). v comes
// back for large v, also infinite. A quarter of the denominator keeps its
// reciprocal a normal number, which is all that the instruction makes.
__device__ __forceinline__ float silu_of(float v) {
    return (0.25f * v) * __builtin_amdgcn_rcpf(__builtin_fmaf(0.25f, exp_of(-v), 0.25f));
}

// Maximum over the 64 lanes, wave-uniform.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return ~wave_min_u32(~v);
}

// Sum over the 64 lanes in a fixed order, the same in every lane.
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// One round per expert taken: the largest key of the wave, its lowest id.
// `emit(r, id, slot)` is called with wave-uniform arguments (id = L V + slot
// of lane L). Returns how many were taken (fewer than k when the rest are -inf
// or NaN). The keys are consumed.
template <int V, class Emit>
__device__ __forceinline__ int take_best(uint32_t (&key)[V], int k, Emit emit) {
    const int lane = lane_id();
    for (int r = 0; r < k; ++r) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = key[i] > m ? key[i] : m;
        m = wave_max_u32(m);
        if (m <= kKeyNegInf) return r;
        uint64_t at[V], any = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            at[i] = __ballot(key[i] == m);
            any |= at[i];
        }
        const int L = __builtin_ctzll(any);
        int id = -1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool hit = id < 0 && ((at[i] >> L) & 1);
            if (hit) id = L * V + i;
            if (hit && lane == L) key[i] = 0;
        }
        emit(r, id, id & (V - 1));
    }
    return k;
}

// +inf as the largest float (so that it can be subtracted from itself).
__device__ __forceinline__ float finite_top(float x) {
    return x > __FLT_MAX__ ? __FLT_MAX__ : x;
}

// Largest of the lanes' values that is no NaN, made finite above.
__device__ __forceinline__ float wave_top(float v) {
    const uint32_t m = wave_max_u32(rank_key(v));
    return finite_top(__uint_as_float((m & 0x80000000u) ? m ^ 0x80000000u : ~m));
}

template <int V>
__device__ __forceinline__ void load_bias(const GateRule &g, float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane_id() * V + i;
        b[i] = g.bias && e < g.E ? g.bias[e] : 0.f;
    }
}

// One token's choice by one wave. `x`: its logits, slot i of lane l expert
// l V + i, -inf past the last; `bias`: likewise, 0 where there is none (read
// by load_bias before the logits are waited for); `ids`, `weights`: its k
// results; `taken(id)` is called, wave-uniform, for each expert taken.
template <int V, class Taken>
__device__ __forceinline__ void gate_row(const GateRule &g, const float (&x)[V],
                                         const float (&bias)[V],
                                         int32_t *ids, float *weights,
                                         Taken taken) {
    const int lane = lane_id();
    bool nan = false;
    uint32_t key[V];
    float top = -__builtin_inff(), all = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        nan |= x[i] != x[i];
        top = x[i] > top ? x[i] : top;
    }
    if (g.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = x[i] == -__builtin_inff()
                         ? 0u : rank_key(sigmoid_of(x[i]) + bias[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = rank_key(x[i]);
        top = wave_top(top);
        if (!g.renorm) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                all += x[i] == -__builtin_inff()
                           ? 0.f : expf(finite_top(x[i]) - top);
            all = wave_sum_f32(all);
        }
    }
    const bool poisoned = __ballot(nan) != 0;
    // lane j keeps the ids and logits of rounds j, j + 64, ...: the last one in
    // registers, with more than 64 rounds all of them in `ids` and `weights`
    int my = -1;
    float mine = 0.f;
    const bool many = g.k > 64;
    const int got = take_best<V>(key, g.k, [&](int r, int id, int slot) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) v = slot == i ? x[i] : v;
        v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), id / V));
        if (lane == (r & 63)) {
            my = id;
            mine = v;
            if (many) {
                ids[r] = id;
                weights[r] = v;
            }
        }
        taken(id);
    });
    auto score = [&](float v) {
        return g.sigmoid ? sigmoid_of(v) : expf(finite_top(v) - top);
    };
    float sum = 0.f, p = 0.f;
    for (int r = lane; r < got; r += 64) {
        p = score(many ? weights[r] : mine);
        sum += p;
    }
    // (the softmax's own denominator cancels in the renormalised weights)
    float n = 1.f;
    if (g.renorm) n = wave_sum_f32(sum) + (g.sigmoid ? 1e-20f : 0.f);
    else if (!g.sigmoid) n = all;
    for (int r = lane; r < g.k; r += 64) {
        const bool have = r < got;
        if (have && many) p = score(weights[r]);
        const float w = have ? p / n * g.scale : 0.f;
        weights[r] = poisoned ? __builtin_nanf("") : w;
        if (!many || !have) ids[r] = have ? my : -1;
    }
}

}  // namespace ue
