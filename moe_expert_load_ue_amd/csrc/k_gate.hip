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
// One wave per token; lane l holds experts l V .. l V + V - 1.
#include "ue_gate.h"

namespace ue {
namespace {

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

int wave_grid(int64_t T, int num_cu) {
    const int64_t blocks = (T + kWaves - 1) / kWaves;
    const int64_t cap = static_cast<int64_t>(num_cu) * 8;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

template <typename T>
hipError_t gate_any(const GateArgs &g, int grid, hipStream_t s) {
    const dim3 gr(grid), bl(kBlock);
    if (g.rule.E <= 64) hipLaunchKernelGGL((k_gate<T, 1>), gr, bl, 0, s, g);
    else if (g.rule.E <= 128) hipLaunchKernelGGL((k_gate<T, 2>), gr, bl, 0, s, g);
    else if (g.rule.E <= 256) hipLaunchKernelGGL((k_gate<T, 4>), gr, bl, 0, s, g);
    else if (g.rule.E <= 512) hipLaunchKernelGGL((k_gate<T, 8>), gr, bl, 0, s, g);
    else hipLaunchKernelGGL((k_gate<T, 16>), gr, bl, 0, s, g);
    return hipGetLastError();
}

template <typename T>
hipError_t back_any(const GateBackArgs &g, int grid, hipStream_t s) {
    const dim3 gr(grid), bl(kBlock);
    const int v = lane_slots(g.rule.E);
    const size_t lds = sizeof(float) * kBlock * v;
    if (v == 1) hipLaunchKernelGGL((k_gate_backward<T, 1>), gr, bl, lds, s, g);
    else if (v == 2) hipLaunchKernelGGL((k_gate_backward<T, 2>), gr, bl, lds, s, g);
    else if (v == 4) hipLaunchKernelGGL((k_gate_backward<T, 4>), gr, bl, lds, s, g);
    else if (v == 8) hipLaunchKernelGGL((k_gate_backward<T, 8>), gr, bl, lds, s, g);
    else hipLaunchKernelGGL((k_gate_backward<T, 16>), gr, bl, lds, s, g);
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
    const int grid = wave_grid(g.T, c.num_cu);
    return g.bf16 ? gate_any<uint16_t>(g, grid, s) : gate_any<float>(g, grid, s);
}

hipError_t launch_gate_backward(const ue_ctx &c, const GateBackArgs &g,
                                hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    const int grid = wave_grid(g.T, c.num_cu);
    return g.bf16 ? back_any<uint16_t>(g, grid, s) : back_any<float>(g, grid, s);
}

}  // namespace ue
