// Expert choice from router logits (ue_gate) and its gradient
// (ue_gate_backward).
//
// Forward, per token with logits l: scores p = softmax(l) or
// 1 / (1 + exp(-l)); experts ranked by l, or by p + bias for the sigmoid;
// weights c p_j / n over the k best, n = 1 or the sum of the chosen scores.
// Backward, with g = c dw on the chosen and 0 elsewhere, and for n the sum
// g <- (g - sum r g) / n, r = p / n: the gradient is p (g - sum p g) for the
// softmax, g p (1 - p) for the sigmoid. With the chosen scores' sum the
// softmax's denominator drops out, so only the chosen logits matter.
//
// Two forms. Up to 256 experts and top-8 (top-16 backward): L = 16 lanes per
// token, or 8 up to 128 experts, so four or eight tokens per wave, every
// reduction a few lane moves inside a row of 16. Else one wave per token,
// lane l holding experts l V .. l V + V - 1.
//
// The choice by L lanes works on 32-bit keys: the upper 24 bits of the rank
// (as ue_gate.h orders floats) over the expert's id, inverted so that the
// lowest wins ties. Each lane sorts its best eight by insertion (one median
// per place), then log2 L steps merge the lanes' lists, the better half of a
// bitonic merge each, until every lane has the token's best eight. Two ranks
// may share their upper 24 bits, and the sigmoid's are made with the fast
// exponential and reciprocal (within 3e-7). So the eight are put in order by
// their exact ranks, each lane counting the better ones; and if an expert
// left out is within those margins of the last one taken, the token is chosen
// again by the rounds on exact keys (of normal fp32 logits of 256 experts, 1
// token in 210 with the sigmoid, in 1100 with the softmax). The upper 24 bits
// hold all of a bf16 logit.
//
// Bound: instruction issue, not bytes. 65,536 fp32 tokens of 256 experts,
// sigmoid: 33 us for 71 MB (2.2 TB/s; a copy's rate would be 15 us), 181
// vector instructions per token, about 22 us of issue. 131,072 bf16 tokens of
// 128 experts, softmax: 29 us forward, 16 us backward (42 MB read, 34 written).
// The rounds over the whole wave took 89, 115 and 60 us. The grid is eight
// workgroups per CU: forward within 8% from three to sixteen, backward 16.4 at
// eight and sixteen, 18.8 at three.
#include "ue_gate.h"

namespace ue {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ float load_logit(const void *p, int64_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const void *p, int64_t i) {
    return static_cast<const float *>(p)[i];
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const void *p, int64_t i) {
    return bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}
__device__ __forceinline__ void store_logit(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t *p, float v) {
    *p = f32_to_bf16(v);
}

// Logits lane * V .. of one row as floats, -inf past the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_row(const void *logits, int64_t row, int E,
                                         bool vec, float (&x)[V]) {
    const int e0 = lane_id() * V;
    constexpr int kBytes = V * static_cast<int>(sizeof(T));
    if constexpr (kBytes == 4 || kBytes == 8 || kBytes == 16 || kBytes == 32 ||
                  kBytes == 64) {
        if (vec) {
            // whole lanes only (E % V == 0), kBytes at a time
            if (e0 >= E) {
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = -__builtin_inff();
                return;
            }
            struct alignas(kBytes < 16 ? kBytes : 16) Pack { T v[V]; };
            const Pack p = *reinterpret_cast<const Pack *>(
                static_cast<const T *>(logits) + row + e0);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = load_logit<T>(p.v, i);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        x[i] = e0 + i < E ? load_logit<T>(logits, row + e0 + i)
                          : -__builtin_inff();
}

template <typename T, int V>
__global__ __launch_bounds__(kBlock) void k_gate(GateArgs g) {
    const int waves = gridDim.x * kWaves;
    float bias[V];
    load_bias<V>(g.rule, bias);
    for (int t = blockIdx.x * kWaves + (threadIdx.x >> 6); t < g.T; t += waves) {
        const int64_t row = static_cast<int64_t>(t) * g.ld;
        const int64_t o = static_cast<int64_t>(t) * g.rule.k;
        float x[V];
        load_row<T, V>(g.logits, row, g.rule.E, g.vec, x);
        gate_row<V>(g.rule, x, bias, g.ids + o, g.weights + o, [](int) {});
    }
}

template <typename T, int V>
__global__ __launch_bounds__(kBlock) void k_gate_backward(GateBackArgs g) {
    // gradient of the scores by expert, one row per wave
    extern __shared__ float dense[];
    const int lane = lane_id(), wv = threadIdx.x >> 6;
    float *d = dense + wv * (64 * V);
    const int waves = gridDim.x * kWaves;
    for (int t = blockIdx.x * kWaves + wv; t < g.T; t += waves) {
        const int64_t row = static_cast<int64_t>(t) * g.ld;
        const int64_t o = static_cast<int64_t>(t) * g.rule.k;
        const bool full = !g.rule.sigmoid && !g.rule.renorm;   // needs every logit
        float x[V], top = -__builtin_inff(), all = 1.f;
        if (full) {
            load_row<T, V>(g.logits, row, g.rule.E, g.vec, x);
#pragma unroll
            for (int i = 0; i < V; ++i) top = x[i] > top ? x[i] : top;
        } else if (!g.rule.sigmoid) {
            for (int r = lane; r < g.rule.k; r += 64) {
                const int id = g.ids[o + r];
                if (static_cast<uint32_t>(id) < static_cast<uint32_t>(g.rule.E)) {
                    const float v = load_logit<T>(g.logits, row + id);
                    top = v > top ? v : top;
                }
            }
        }
        if (!g.rule.sigmoid) top = wave_top(top);
        if (full) {
            all = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = x[i] == -__builtin_inff()
                           ? 0.f : expf(finite_top(x[i]) - top);
                all += x[i];
            }
            all = wave_sum_f32(all);
            if (all == 0.f) all = 1.f;      // every expert masked: all zeros
        }
#pragma unroll
        for (int i = 0; i < V; ++i) d[lane * V + i] = 0.f;
        auto score = [&](float v) {
            return g.rule.sigmoid ? sigmoid_of(v) : expf(finite_top(v) - top) / all;
        };
        // sums over the chosen: of their scores, and of score times gradient
        float n = 0.f, pg = 0.f;
        for (int r = lane; r < g.rule.k; r += 64) {
            const int id = g.ids[o + r];
            if (static_cast<uint32_t>(id) < static_cast<uint32_t>(g.rule.E)) {
                const float p = score(load_logit<T>(g.logits, row + id));
                n += p;
                pg += p * (g.rule.scale * g.dweights[o + r]);
            }
        }
        n = wave_sum_f32(n) + (g.rule.sigmoid ? 1e-20f : 0.f);
        pg = wave_sum_f32(pg);
        __builtin_amdgcn_wave_barrier();
        for (int r = lane; r < g.rule.k; r += 64) {
            const int id = g.ids[o + r];
            if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(g.rule.E)) continue;
            const float gk = g.rule.scale * g.dweights[o + r];
            const float v = load_logit<T>(g.logits, row + id);
            float y;
            if (g.rule.sigmoid)
                y = (g.rule.renorm ? (gk - pg / n) / n : gk) * sigmoid_slope(v);
            else
                y = g.rule.renorm ? score(v) / n * (gk - pg / n) : gk;
            d[id] = y;
        }
        __builtin_amdgcn_wave_barrier();
        T *out = static_cast<T *>(g.dlogits) + static_cast<int64_t>(t) * g.ld_out;
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            y[i] = d[lane * V + i];
            if (full) y[i] = x[i] / all * (y[i] - pg);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i < g.rule.E) store_logit(out + lane * V + i, y[i]);
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- 8 or 16 lanes per token --------------------------------------------------

constexpr int kFastExperts = 256, kFastTopk = 8, kFastBackTopk = 16;

template <int CTRL>
__device__ __forceinline__ uint32_t move_row(uint32_t v) {
    // (every lane has a source: the old value and the bound bit only let the
    // move fold into the instruction that uses it)
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// Lane moves that pair up 8 lanes in three steps, all 16 of a row in four.
constexpr int kPair1 = 0xB1, kPair2 = 0x4E, kPair4 = 0x141, kPair8 = 0x140;

template <int CTRL>
__device__ __forceinline__ float add_row(float v) {
    return v + __uint_as_float(move_row<CTRL>(__float_as_uint(v)));
}
// Sum over a token's L lanes, in all of them, in a fixed order.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
    v = add_row<kPair4>(add_row<kPair2>(add_row<kPair1>(v)));
    return L == 16 ? add_row<kPair8>(v) : v;
}
template <int CTRL>
__device__ __forceinline__ float max_row(float v) {
    const float o = __uint_as_float(move_row<CTRL>(__float_as_uint(v)));
    return o > v ? o : v;
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
    v = max_row<kPair4>(max_row<kPair2>(max_row<kPair1>(v)));
    return L == 16 ? max_row<kPair8>(v) : v;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
    return umax(umin(a, b), umin(umax(a, b), c));
}

// Keeps the better half of this lane's list and its partner's, sorted again.
template <int CTRL>
__device__ __forceinline__ void merge_lists(uint32_t (&a)[8]) {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = umax(a[i], move_row<CTRL>(a[7 - i]));
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) {
                const uint32_t hi = umax(m[i], m[i | d]), lo = umin(m[i], m[i | d]);
                m[i] = hi;
                m[i | d] = lo;
            }
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = m[i];
}

// The float a key was made from, with its lowest 8 bits zero.
__device__ __forceinline__ float key_value(uint32_t key) {
    const uint32_t k = (key & 0x80000000u) ? key ^ 0x80000000u : ~key;
    return __uint_as_float(k & ~0xFFu);
}

// exp(x) within (2 + 1.2 |x|) u: for ranks that are looked at again, and for
// the softmax's denominator, where a term x below the top counts with its
// weight e^x (the weighted mean of |x| over 256 terms is at most 3.4, so the
// sum is within 7 u).
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * kLog2e);
}

// This lane's VP logits of its L lanes' token, -inf past the last expert, and
// their ids: four at a time when `vec`. WHOLE: L VP experts, in rows that
// load so.
template <int L, bool WHOLE>
__device__ __forceinline__ int slot_expert(int i, bool vec) {
    const int l = lane_id() & (L - 1);
    return WHOLE || vec ? (i >> 2) * 4 * L + l * 4 + (i & 3) : i * L + l;
}
template <typename T, int L, int VP, bool WHOLE>
__device__ __forceinline__ void load_slots(const void *logits, int64_t row, int E,
                                           bool vec, float (&x)[VP]) {
    const T *p = static_cast<const T *>(logits) + row;
    if (WHOLE || vec) {
        struct alignas(4 * sizeof(T)) Pack { T v[4]; };
#pragma unroll
        for (int c = 0; c < VP / 4; ++c) {
            const int e = slot_expert<L, WHOLE>(4 * c, true);
            const bool in = WHOLE || e < E;
            const Pack q = *reinterpret_cast<const Pack *>(p + (in ? e : 0));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 * c + i] = in ? load_logit<T>(q.v, i) : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int e = slot_expert<L, false>(i, false);
            const float v = load_logit<T>(p, e < E ? e : 0);
            x[i] = e < E ? v : -__builtin_inff();
        }
    }
}

// Lane l gets lane l ^ N of its eight.
template <int N>
__device__ __forceinline__ uint32_t swap_lanes(uint32_t v) {
    if constexpr (N & 4) v = move_row<kPair4>(v);             // l ^ 7
    constexpr int M = N & 4 ? N ^ 7 : N;
    if constexpr (M == 1) v = move_row<kPair1>(v);
    if constexpr (M == 2) v = move_row<kPair2>(v);
    if constexpr (M == 3) v = move_row<0x1B>(v);
    return v;
}
// How many of the other seven entries (one per lane of eight) rank higher,
// ties to the lower id.
template <int N = 1>
__device__ __forceinline__ int better_ones(uint32_t key, uint32_t id) {
    if constexpr (N == 8) {
        return 0;
    } else {
        const uint32_t ok = swap_lanes<N>(key), oi = swap_lanes<N>(id);
        const int above = ok > key || (ok == key && oi < id);
        return above + better_ones<N + 1>(key, id);
    }
}

// L lanes per token; VP: logits a lane holds (L VP >= E).
template <typename T, int L, int VP, bool SIGMOID, bool WHOLE>
__global__ __launch_bounds__(kBlock) void k_gate_rows(GateArgs g) {
    constexpr int V = L * VP <= 64 ? 1 : L * VP / 64;   // slots of the rounds
    constexpr int kEach = 64 / L;                       // tokens of a wave
    constexpr bool kExact = sizeof(T) == 2 && !SIGMOID; // keys hold the rank
    const int lane = lane_id(), at = lane & (L - 1), sub = lane / L;
    const int E = g.rule.E, k = g.rule.k;
    const int step = gridDim.x * kWaves * kEach;
    float bias[VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) {
        const int e = slot_expert<L, WHOLE>(i, g.vec4);
        bias[i] = SIGMOID && g.rule.bias ? g.rule.bias[WHOLE || e < E ? e : 0] : 0.f;
    }
    // The logits again (and the biases), for the second look at the chosen
    // ones: from LDS, so that it does not wait on memory. (A bf16 logit is in
    // its key.)
    __shared__ __align__(16) float seen[kExact ? 1 : kWaves * kEach][L * VP];
    __shared__ float seen_bias[SIGMOID ? L * VP : 1];
    float *const mine_seen = seen[kExact ? 0 : (threadIdx.x >> 6) * kEach + sub];
    if (SIGMOID) {
        for (int e = threadIdx.x; e < E; e += kBlock)
            seen_bias[e] = g.rule.bias ? g.rule.bias[e] : 0.f;
        __syncthreads();
    }
    // 0, or NaN where a bias is infinite or NaN
    float odd_bias = 0.f;
#pragma unroll
    for (int i = 0; i < VP; ++i) odd_bias += bias[i] * 0.f;
    // (rows past the last token repeat it and write nothing)
    auto row_of = [&](int t) { return t < g.T ? t : g.T - 1; };
    const int first = (blockIdx.x * kWaves + (threadIdx.x >> 6)) * kEach;
    float next[VP];
    if (first < g.T)
        load_slots<T, L, VP, WHOLE>(g.logits, row_of(first + sub) * g.ld, E, g.vec4, next);
    for (int t0 = first; t0 < g.T; t0 += step) {
        const bool real = t0 + sub < g.T;
        const int64_t o = static_cast<int64_t>(row_of(t0 + sub)) * k;
        float x[VP];
#pragma unroll
        for (int i = 0; i < VP; ++i) x[i] = next[i];
        if (!kExact) {
#pragma unroll
            for (int i = 0; i < VP; i += 4)
                if (WHOLE || g.vec4)
                    *reinterpret_cast<f32x4 *>(mine_seen + slot_expert<L, WHOLE>(i, true)) =
                        f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
                else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mine_seen[slot_expert<L, false>(i + j, false)] = x[i + j];
            __builtin_amdgcn_wave_barrier();
        }
        // likewise for the logits: only then are the keys made with care for
        // such values
        float odd = odd_bias;
#pragma unroll
        for (int i = 0; i < VP; ++i) odd += x[i] * 0.f;
        uint32_t key[VP], best[8] = {};
        auto insert = [&](int i, uint32_t upper) {
            key[i] = (upper & ~0xFFu) |
                     static_cast<uint32_t>(255 - slot_expert<L, WHOLE>(i, g.vec4));
#pragma unroll
            for (int j = 7; j > 0; --j)
                if (j <= i) best[j] = med3(best[j - 1], best[j], key[i]);
            best[0] = umax(best[0], key[i]);
        };
        bool nan = false;
        const bool careful = __ballot(odd != odd) != 0;
        if (careful) {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                nan |= x[i] != x[i];
                float r = x[i];
                if (SIGMOID && r != -__builtin_inff())
                    r = __builtin_amdgcn_rcpf(1.0f + fast_exp(-r)) + bias[i];
                insert(i, rank_key(r));
            }
        } else {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                float r = x[i];
                if (SIGMOID) r = __builtin_amdgcn_rcpf(1.0f + fast_exp(-r)) + bias[i];
                // rank_key of a number
                const uint32_t b = __float_as_uint(r + 0.0f);
                insert(i, b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) |
                               0x80000000u));
            }
        }
        // the next tokens' logits, on their way while these are chosen
        if (t0 + step < g.T)
            load_slots<T, L, VP, WHOLE>(g.logits, row_of(t0 + step + sub) * g.ld, E,
                                     g.vec4, next);
        merge_lists<kPair1>(best);
        merge_lists<kPair2>(best);
        merge_lists<kPair4>(best);
        if constexpr (L == 16) merge_lists<kPair8>(best);

        bool clear = true;
        if constexpr (!kExact) {
            uint32_t last = best[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) last = j < k ? best[j] : last;
            // the least key that could belong to a rank as good as the last
            uint32_t bar = (last & ~0xFFu) - 0x100u;
            if (SIGMOID) bar = umin(bar, rank_key(key_value(last) - 1e-6f) & ~0xFFu);
            int above = 0;
#pragma unroll
            for (int i = 0; i < VP; ++i) above += key[i] >= bar;
            clear = row_sum<L>(static_cast<float>(above)) == static_cast<float>(k) &&
                    last > kKeyNegInf;
        }
        // lane j (and j + 8 of 16): place j of the list
        uint32_t mine = best[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mine = (at & 7) == j ? best[j] : mine;
        const bool have = (at & 7) < k && mine > kKeyNegInf;
        const int id = 255 - static_cast<int>(mine & 0xFFu);
        float v = -__builtin_inff(), p = 0.f;
        if (have) v = kExact ? key_value(mine) : mine_seen[id];
        // the denominator over all experts, taken at the best logit
        float top = 0.f, all = 1.f;
        if (!SIGMOID) {
            top = row_max<L>(v);
            if (!g.rule.renorm) {
                all = 0.f;
#pragma unroll
                for (int i = 0; i < VP; ++i) all += fast_exp(x[i] - top);
                all = row_sum<L>(all);
            }
        }
        uint32_t exact = 0;
        if (have) {
            p = SIGMOID ? sigmoid_of(v) : expf(v - top);
            if (SIGMOID)
                exact = rank_key(p + seen_bias[id]);
            else
                exact = rank_key(v);
        }
        int place = at & 7;
        if constexpr (!kExact) place = better_ones(exact, have ? id : 256 + (at & 7));
        float n = all;
        if (g.rule.renorm) {
            n = row_sum<L>(at < 8 ? p : 0.f) + (SIGMOID ? 1e-20f : 0.f);
            if (!SIGMOID && n == 0.f) n = 1.f;
        }
        // an infinite logit takes the rounds too, where +inf is a number
        if (careful) clear &= !(top > __FLT_MAX__);
        const bool poisoned = (__ballot(nan) >> (sub * L)) & ((1u << L) - 1);
        if (clear && real && at < 8 && place < k) {
            const float w = have ? p / n * g.rule.scale : 0.f;
            g.ids[o + place] = have ? id : -1;
            g.weights[o + place] = poisoned ? __builtin_nanf("") : w;
        }
        uint64_t again = __ballot(!clear && real);
        while (again) {
            const int which = __builtin_ctzll(again) / L;
            again &= ~(((1ull << L) - 1) << (which * L));
            const int64_t tt = t0 + which;
            float y[V], b[V];
            load_bias<V>(g.rule, b);
            load_row<T, V>(g.logits, tt * g.ld, E, false, y);
            gate_row<V>(g.rule, y, b, g.ids + tt * k, g.weights + tt * k, [](int) {});
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int L, int VP, bool WHOLE>
__global__ __launch_bounds__(kBlock) void k_gate_backward_rows(GateBackArgs g) {
    constexpr int kEach = 64 / L;                       // tokens of a wave
    // gradient of the scores by expert, one row per token
    __shared__ __align__(16) float dense[kWaves * kEach][L * VP];
    const int lane = lane_id(), at = lane & (L - 1), sub = lane / L;
    const int wv = threadIdx.x >> 6, E = g.rule.E, k = g.rule.k;
    float *d = dense[wv * kEach + sub];
    const bool full = !g.rule.sigmoid && !g.rule.renorm;   // needs every logit
    const int step = gridDim.x * kWaves * kEach;
    for (int t0 = (blockIdx.x * kWaves + wv) * kEach; t0 < g.T; t0 += step) {
        const int t = t0 + sub < g.T ? t0 + sub : g.T - 1;
        const int64_t row = static_cast<int64_t>(t) * g.ld;
        const int64_t o = static_cast<int64_t>(t) * k;
        const int id = at < k ? g.ids[o + at] : -1;
        const bool have = static_cast<uint32_t>(id) < static_cast<uint32_t>(E);
        const float gk = have ? g.rule.scale * g.dweights[o + at] : 0.f;
        float v = have ? load_logit<T>(g.logits, row + id) : -__builtin_inff();
        float x[VP], top = v, all = 1.f;
        if (full) {
            load_slots<T, L, VP, WHOLE>(g.logits, row, E, g.vec4, x);
#pragma unroll
            for (int i = 0; i < VP; ++i) top = x[i] > top ? x[i] : top;
        }
        top = finite_top(row_max<L>(top));
        if (full) {
            all = 0.f;
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                // (an fp32 gradient shows an unlikely expert's error in full;
                // in bf16 100 u are lost in the rounding)
                const float below = finite_top(x[i]) - top;
                x[i] = x[i] == -__builtin_inff() ? 0.f
                       : sizeof(T) == 4 ? exp_of(below) : fast_exp(below);
                all += x[i];
            }
            all = row_sum<L>(all);
            if (all == 0.f) all = 1.f;      // every expert masked: all zeros
        }
        float p = 0.f;
        if (have) p = g.rule.sigmoid ? sigmoid_of(v) : expf(finite_top(v) - top) / all;
        const float n = row_sum<L>(p) + (g.rule.sigmoid ? 1e-20f : 0.f);
        const float pg = row_sum<L>(p * gk);
        float y = gk;
        if (g.rule.renorm && have) {
            y = (gk - pg / n) / n;
            if (!g.rule.sigmoid) y *= p;
        }
        if (g.rule.sigmoid && have) y *= sigmoid_slope(v);
#pragma unroll
        for (int i = 0; i < VP; i += 4)
            *reinterpret_cast<f32x4 *>(d + at * VP + i) = f32x4{0, 0, 0, 0};
        __builtin_amdgcn_wave_barrier();
        if (have) d[id] = y;
        __builtin_amdgcn_wave_barrier();
        T *out = static_cast<T *>(g.dlogits) + static_cast<int64_t>(t) * g.ld_out;
        const float rest = 1.f / all;
        if (WHOLE || g.vec4) {
            struct alignas(4 * sizeof(T)) Pack { T v[4]; };
#pragma unroll
            for (int c = 0; c < VP / 4; ++c) {
                const int e = slot_expert<L, WHOLE>(4 * c, true);
                if ((!WHOLE && e >= E) || t0 + sub >= g.T) continue;
                const f32x4 q = *reinterpret_cast<const f32x4 *>(d + e);
                Pack r;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_logit(&r.v[i], full ? x[4 * c + i] * rest * (q[i] - pg) : q[i]);
                *reinterpret_cast<Pack *>(out + e) = r;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const int e = slot_expert<L, WHOLE>(i, false);
                if (e < E && t0 + sub < g.T)
                    store_logit(out + e, full ? x[i] * rest * (d[e] - pg) : d[e]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// A workgroup's waves take `each` tokens at a time; enough workgroups to fill
// the device, the rest in a loop.
int wave_grid(int64_t T, int each, int num_cu) {
    const int64_t blocks = (T + kWaves * each - 1) / (kWaves * each);
    const int64_t cap = static_cast<int64_t>(num_cu) * 8;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

template <typename T, int L, int VP>
void gate_rows_any(const ue_ctx &c, const GateArgs &g, hipStream_t s) {
    const bool whole = g.rule.E == L * VP && g.vec4;
    const dim3 gr(wave_grid(g.T, 64 / L, c.num_cu)), bl(kBlock);
    if (g.rule.sigmoid) {
        if (whole) hipLaunchKernelGGL((k_gate_rows<T, L, VP, true, true>), gr, bl, 0, s, g);
        else hipLaunchKernelGGL((k_gate_rows<T, L, VP, true, false>), gr, bl, 0, s, g);
    } else {
        if (whole) hipLaunchKernelGGL((k_gate_rows<T, L, VP, false, true>), gr, bl, 0, s, g);
        else hipLaunchKernelGGL((k_gate_rows<T, L, VP, false, false>), gr, bl, 0, s, g);
    }
}

template <typename T, int L, int VP>
void back_rows_any(const ue_ctx &c, const GateBackArgs &g, hipStream_t s) {
    const dim3 gr(wave_grid(g.T, 64 / L, c.num_cu)), bl(kBlock);
    if (g.rule.E == L * VP && g.vec4)
        hipLaunchKernelGGL((k_gate_backward_rows<T, L, VP, true>), gr, bl, 0, s, g);
    else
        hipLaunchKernelGGL((k_gate_backward_rows<T, L, VP, false>), gr, bl, 0, s, g);
}

template <typename T>
hipError_t gate_any(const ue_ctx &c, const GateArgs &g, hipStream_t s) {
    const int E = g.rule.E;
    if (E <= kFastExperts && g.rule.k <= kFastTopk) {
        if (E <= 32) gate_rows_any<T, 8, 4>(c, g, s);
        else if (E <= 64) gate_rows_any<T, 8, 8>(c, g, s);
        else if (E <= 128) gate_rows_any<T, 8, 16>(c, g, s);
        else gate_rows_any<T, 16, 16>(c, g, s);
    } else {
        const dim3 gr(wave_grid(g.T, 1, c.num_cu)), bl(kBlock);
        switch (lane_slots(E)) {
            case 1: hipLaunchKernelGGL((k_gate<T, 1>), gr, bl, 0, s, g); break;
            case 2: hipLaunchKernelGGL((k_gate<T, 2>), gr, bl, 0, s, g); break;
            case 4: hipLaunchKernelGGL((k_gate<T, 4>), gr, bl, 0, s, g); break;
            case 8: hipLaunchKernelGGL((k_gate<T, 8>), gr, bl, 0, s, g); break;
            default: hipLaunchKernelGGL((k_gate<T, 16>), gr, bl, 0, s, g); break;
        }
    }
    return hipGetLastError();
}

template <typename T>
hipError_t back_any(const ue_ctx &c, const GateBackArgs &g, hipStream_t s) {
    const int E = g.rule.E;
    if (E <= 128 && g.rule.k <= 8) {
        if (E <= 32) back_rows_any<T, 8, 4>(c, g, s);
        else if (E <= 64) back_rows_any<T, 8, 8>(c, g, s);
        else back_rows_any<T, 8, 16>(c, g, s);
    } else if (E <= kFastExperts && g.rule.k <= kFastBackTopk) {
        back_rows_any<T, 16, 16>(c, g, s);
    } else {
        const dim3 gr(wave_grid(g.T, 1, c.num_cu)), bl(kBlock);
        const int v = lane_slots(E);
        const size_t lds = sizeof(float) * kBlock * v;
        switch (v) {
            case 1: hipLaunchKernelGGL((k_gate_backward<T, 1>), gr, bl, lds, s, g); break;
            case 2: hipLaunchKernelGGL((k_gate_backward<T, 2>), gr, bl, lds, s, g); break;
            case 4: hipLaunchKernelGGL((k_gate_backward<T, 4>), gr, bl, lds, s, g); break;
            case 8: hipLaunchKernelGGL((k_gate_backward<T, 8>), gr, bl, lds, s, g); break;
            default: hipLaunchKernelGGL((k_gate_backward<T, 16>), gr, bl, lds, s, g); break;
        }
    }
    return hipGetLastError();
}

}  // namespace

int lane_slots(int E) {
    int v = 1;
    while (64 * v < E) v *= 2;
    return v;
}

hipError_t launch_gate(const ue_ctx &c, const GateArgs &g, hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    return g.bf16 ? gate_any<uint16_t>(c, g, s) : gate_any<float>(c, g, s);
}

hipError_t launch_gate_backward(const ue_ctx &c, const GateBackArgs &g,
                                hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    return g.bf16 ? back_any<uint16_t>(c, g, s) : back_any<float>(c, g, s);
}

}  // namespace ue
