// A mixture-of-experts layer for a few tokens (ue_moe_tokens): router,
// choice of experts, gated experts, weighted sum.
//
//   logits = x Wr^T;  (ids, w) = gate(logits)
//   h_tj = silu(x_t Wg^T) (x_t Wu^T)   of expert ids[t, j]
//   out_t = sum_j w_tj h_tj Wd^T
//
// With few tokens the bytes of the chosen experts' matrices bound the layer:
// each is read once, straight from HBM into the registers of the wave that
// multiplies it (no reuse, so no LDS), for all tokens of the expert at once.
// The matrix is the matrix instruction's first operand (16 of its rows by 32
// of K), the tokens its second, so up to 16 tokens cost what one does.
// Activations come from cache, the same few rows for every workgroup.
// Weights in 8 bits are widened to bf16 (exact) and their channel scale
// multiplies the 32-bit sum.
//
// h is kept as a sum of two bf16 numbers (its rounding and the rest), each
// multiplied on its own: the second product's operands then carry 16 bits
// of h, and the layer's result is rounded once, at the end. The extra matrix
// instructions are free while bytes bound the kernel.
#include "ue_gate.h"

namespace ue {
namespace {

typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 hbf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(hbf16x8, w), __builtin_bit_cast(hbf16x8, x), c, 0, 0, 0);
}

// Four int8 as bf16 (exact: 8 bits fit the significand).
__device__ __forceinline__ u32x2 widen4(uint32_t v) {
    const float f0 = static_cast<float>(static_cast<int8_t>(v));
    const float f1 = static_cast<float>(static_cast<int8_t>(v >> 8));
    const float f2 = static_cast<float>(static_cast<int8_t>(v >> 16));
    const float f3 = static_cast<float>(static_cast<int8_t>(v >> 24));
    // the low halves are zero: take the high ones
    return u32x2{__builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0),
                                       0x07060302u),
                 __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2),
                                       0x07060302u)};
}

// A wave's pass over K of 16 matrix rows (this lane's row starts at w) for
// RT tiles of 16 tokens (this lane's rows at x[], and x2[] where the
// activations are sums of two parts). One step covers kK elements of K: a
// lane group q reads the 16 bytes of the matrix at q * 16 of each 64. `k`
// runs from k0 to k1, a multiple of the step apart but for the last.
template <bool I8>
struct Weights;
template <>
struct Weights<false> {
    static constexpr int kK = 32;             // elements per load of 64 bytes
    typedef u32x4 Frag;                       // 8 bf16
    static __device__ __forceinline__ Frag load(const char *row, int k, int q) {
        return *reinterpret_cast<const u32x4 *>(row + 2 * (k + 8 * q));
    }
};
template <>
struct Weights<true> {
    static constexpr int kK = 64;
    typedef u32x4 Frag;                       // 16 int8
    static __device__ __forceinline__ Frag load(const char *row, int k, int q) {
        return *reinterpret_cast<const u32x4 *>(row + k + 16 * q);
    }
};

// NW matrix streams against RT token tiles of P parts each, K in [k0, k1).
template <bool I8, int NW, int RT, int P>
__device__ __forceinline__ void stream(const char *const (&w)[NW],
                                       const uint16_t *const (&x)[RT][P],
                                       int k0, int k1, int K,
                                       f32x4 (&acc)[NW][RT]) {
    constexpr int kK = Weights<I8>::kK;
    constexpr int kEl = I8 ? 16 : 8;          // elements a lane holds
    const int q = lane_id() >> 4;
    for (int k = k0; k < k1; k += kK) {
        // a lane past K reads the row's start and multiplies by zero
        const bool in = k + q * kEl < K;
        const int kk = in ? k : -q * kEl;
        u32x4 wf[NW];
#pragma unroll
        for (int n = 0; n < NW; ++n) wf[n] = Weights<I8>::load(w[n], kk, q);
        if constexpr (!I8) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    u32x4 xf = *reinterpret_cast<const u32x4 *>(x[r][p] + kk + 8 * q);
                    if (!in) xf = u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int n = 0; n < NW; ++n) {
                        u32x4 v = wf[n];
                        if (!in) v = u32x4{0, 0, 0, 0};
                        acc[n][r] = mfma(v, xf, acc[n][r]);
                    }
                }
        } else {
            u32x4 lo[NW], hi[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const u32x2 a = widen4(wf[n].x), b = widen4(wf[n].y);
                const u32x2 c = widen4(wf[n].z), d = widen4(wf[n].w);
                lo[n] = u32x4{a.x, a.y, b.x, b.y};
                hi[n] = u32x4{c.x, c.y, d.x, d.y};
            }
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const u32x4 *xp = reinterpret_cast<const u32x4 *>(x[r][p] + kk + 16 * q);
                    u32x4 x0 = xp[0], x1 = xp[1];
                    if (!in) x0 = x1 = u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int n = 0; n < NW; ++n) {
                        acc[n][r] = mfma(lo[n], x0, acc[n][r]);
                        acc[n][r] = mfma(hi[n], x1, acc[n][r]);
                    }
                }
        }
    }
}

// K split over W waves in whole steps: wave v's share.
__device__ __forceinline__ void share(int K, int step, int W, int v, int &k0,
                                      int &k1) {
    const int n = (K + step - 1) / step;
    const int per = (n + W - 1) / W;
    k0 = v * per * step;
    k1 = (v + 1) * per * step;
    k1 = k1 < n * step ? k1 : n * step;
}

// ---- router ---------------------------------------------------------------
// Logits of 16 experts per workgroup, K split over the waves.
constexpr int kRouterWaves = 8;

template <int RT>
__global__ __launch_bounds__(kRouterWaves * 64) void k_router(MoeArgs g) {
    __shared__ f32x4 part[kRouterWaves][RT][64];
    const int lane = lane_id(), l16 = lane & 15, q = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e = blockIdx.x * 16 + l16;
    const char *w[1] = {reinterpret_cast<const char *>(
        g.router + static_cast<int64_t>(e < g.rule.E ? e : g.rule.E - 1) * g.H)};
    const uint16_t *x[RT][1];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int t = r * 16 + l16;
        x[r][0] = g.x + static_cast<int64_t>(t < g.T ? t : g.T - 1) * g.ldx;
    }
    f32x4 acc[1][RT] = {};
    int k0, k1;
    share(g.H, 32, kRouterWaves, wv, k0, k1);
    stream<false, 1, RT, 1>(w, x, k0, k1, g.H, acc);
#pragma unroll
    for (int r = 0; r < RT; ++r) part[wv][r][lane] = acc[0][r];
    __syncthreads();
    for (int r = wv; r < RT; r += kRouterWaves) {
        f32x4 s = part[0][r][lane];
        for (int v = 1; v < kRouterWaves; ++v) {
            const f32x4 b = part[v][r][lane];
            s.x += b.x; s.y += b.y; s.z += b.z; s.w += b.w;
        }
        const int t = r * 16 + l16;
        if (t >= g.T) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ee = blockIdx.x * 16 + 4 * q + i;
            if (ee < g.rule.E) g.logits[static_cast<int64_t>(t) * g.rule.E + ee] = s[i];
        }
    }
}

// ---- choice ----------------------------------------------------------------
// One workgroup: every token's experts and weights, then the experts in use
// with their tokens, as one 64-bit set per expert.
constexpr int kChooseWaves = 16;

template <int V>
__global__ __launch_bounds__(kChooseWaves * 64) void k_choose(MoeArgs g) {
    __shared__ unsigned long long set[kMaxExperts];
    __shared__ int base[kMaxExperts];
    const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
    const int E = g.rule.E;
    for (int e = tid; e < E; e += kChooseWaves * 64) set[e] = 0;
    __syncthreads();
    for (int t = wv; t < g.T; t += kChooseWaves) {
        const float *lg = g.logits + static_cast<int64_t>(t) * E;
        const int64_t o = static_cast<int64_t>(t) * g.rule.k;
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            x[i] = e < E ? lg[e] : -__builtin_inff();
        }
        gate_row<V>(
            g.rule, x, [&](int id) { return lg[id]; }, g.ids + o, g.weights + o,
            [&](int id) {
                if (lane == 0) atomicOr(&set[id], 1ull << t);
            });
    }
    __syncthreads();
    // experts in use, in id order, and where their tokens start: one wave,
    // 64 experts at a time
    if (wv == 0) {
        int n_act = 0, rows = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const unsigned long long s = e < E ? set[e] : 0;
            const int c = __popcll(s);
            const uint64_t used = __ballot(c > 0);
            const int incl = wave_inclusive_sum(c);
            if (e < E) base[e] = rows + incl - c;
            if (c > 0) {
                MoeExpert a;
                a.tokens = s;
                a.expert = e;
                a.base = rows + incl - c;
                g.active[n_act + mask_rank(used)] = a;
            }
            n_act += __popcll(used);
            rows += __builtin_amdgcn_readlane(incl, 63);
        }
        if (lane == 0) *g.n_active = n_act;
    }
    __syncthreads();
    // the weight of each (expert, token) row, and the token
    for (int a = tid; a < g.T * g.rule.k; a += kChooseWaves * 64) {
        const int t = a / g.rule.k;
        const int e = g.ids[a];
        if (e < 0) continue;
        const int r = base[e] + __popcll(set[e] & ((1ull << t) - 1));
        g.row_weight[r] = g.weights[a];
        g.row_token[r] = t;
    }
}

// ---- gate and up -------------------------------------------------------------
// 16 channels of one expert per workgroup, K split over the waves.
constexpr int kUpWaves = 4;

template <bool I8, int RT>
__device__ __forceinline__ void up_tile(const MoeArgs &g, const MoeExpert &a,
                                        int cnt, int n0, f32x4 *part) {
    const int lane = lane_id(), l16 = lane & 15, q = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kB = I8 ? 1 : 2;
    const int n = n0 + l16 < g.I ? n0 + l16 : g.I - 1;
    const char *mat = static_cast<const char *>(g.gate_up) +
                      a.expert * g.gate_up_stride * kB;
    const char *w[2] = {mat + static_cast<int64_t>(n) * g.H * kB,
                        mat + (static_cast<int64_t>(g.I) + n) * g.H * kB};
    const uint16_t *x[RT][1];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = r * 16 + l16;
        const int t = g.row_token[a.base + (i < cnt ? i : cnt - 1)];
        x[r][0] = g.x + static_cast<int64_t>(t) * g.ldx;
    }
    f32x4 acc[2][RT] = {};
    int k0, k1;
    share(g.H, Weights<I8>::kK, kUpWaves, wv, k0, k1);
    stream<I8, 2, RT, 1>(w, x, k0, k1, g.H, acc);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
            part[((wv * 2 + m) * RT + r) * 64 + lane] = acc[m][r];
    __syncthreads();
    for (int r = wv; r < RT; r += kUpWaves) {
        f32x4 s[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            s[m] = part[(m * RT + r) * 64 + lane];
            for (int v = 1; v < kUpWaves; ++v) {
                const f32x4 b = part[((v * 2 + m) * RT + r) * 64 + lane];
                s[m].x += b.x; s[m].y += b.y; s[m].z += b.z; s[m].w += b.w;
            }
        }
        const int i = r * 16 + l16;
        if (i >= cnt) continue;
        const int64_t row = static_cast<int64_t>(a.base + i) * g.I;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int nn = n0 + 4 * q + c;
            if (nn >= g.I) continue;
            float gt = s[0][c], up = s[1][c];
            if (I8) {
                const float *sc = g.gate_up_scale + static_cast<int64_t>(a.expert) * 2 * g.I;
                gt *= sc[nn];
                up *= sc[g.I + nn];
            }
            const float h = gt / (1.0f + expf(-gt)) * up;
            const uint16_t hi = f32_to_bf16(h);
            const float rest = h - bf16_to_f32(hi);
            g.h_hi[row + nn] = hi;
            // (an infinite h has no finite rest)
            g.h_lo[row + nn] = fabsf(h) <= __FLT_MAX__ ? f32_to_bf16(rest) : 0;
        }
    }
}

template <bool I8>
__global__ __launch_bounds__(kUpWaves * 64) void k_moe_up(MoeArgs g) {
    __shared__ f32x4 part[kUpWaves * 2 * 4 * 64];
    const int a = blockIdx.y;
    if (a >= *g.n_active) return;
    const MoeExpert ex = g.active[a];
    const int cnt = __popcll(ex.tokens);
    const int n0 = blockIdx.x * 16;
    if (cnt <= 16) up_tile<I8, 1>(g, ex, cnt, n0, part);
    else if (cnt <= 32) up_tile<I8, 2>(g, ex, cnt, n0, part);
    else up_tile<I8, 4>(g, ex, cnt, n0, part);
}

// ---- down and weighted sum -----------------------------------------------------
// 16 output channels per workgroup. A unit is an expert and a share of its K;
// each wave adds its units' weighted rows to its own sums (LDS), which are
// joined in wave order: no atomics, so the result does not depend on timing.
constexpr int kDownWaves = 8;

template <bool I8, int RT>
__device__ __forceinline__ void down_unit(const MoeArgs &g, const MoeExpert &a,
                                          int cnt, int n0, int k0, int k1,
                                          f32x4 *sum) {
    const int lane = lane_id(), l16 = lane & 15, q = lane >> 4;
    constexpr int kB = I8 ? 1 : 2;
    const int n = n0 + l16 < g.H ? n0 + l16 : g.H - 1;
    const char *w[1] = {static_cast<const char *>(g.down) +
                        (a.expert * g.down_stride +
                         static_cast<int64_t>(n) * g.I) * kB};
    const uint16_t *x[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = r * 16 + l16;
        const int64_t row = static_cast<int64_t>(a.base + (i < cnt ? i : cnt - 1)) * g.I;
        x[r][0] = g.h_hi + row;
        x[r][1] = g.h_lo + row;
    }
    f32x4 acc[1][RT] = {};
    stream<I8, 1, RT, 2>(w, x, k0, k1, g.I, acc);
    f32x4 sc = {1.f, 1.f, 1.f, 1.f};
    if (I8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int nn = n0 + 4 * q + c;
            sc[c] = g.down_scale[static_cast<int64_t>(a.expert) * g.H +
                                 (nn < g.H ? nn : g.H - 1)];
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = r * 16 + l16;
        if (i >= cnt) continue;
        const int t = g.row_token[a.base + i];
        const float wt = g.row_weight[a.base + i];
        f32x4 &s = sum[t * 4 + q];
        f32x4 v = s;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += acc[0][r][c] * sc[c] * wt;
        s = v;
    }
}

template <bool I8>
__global__ __launch_bounds__(kDownWaves * 64) void k_moe_down(MoeArgs g) {
    extern __shared__ f32x4 sums[];               // [waves][T][4]
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16;
    f32x4 *mine = sums + wv * g.T * 4;
    for (int i = lane; i < g.T * 4; i += 64) mine[i] = f32x4{0, 0, 0, 0};
    const int n_act = *g.n_active;
    // shares of K so that few experts still occupy every wave
    int split = 1;
    while (n_act * split < kDownWaves && split < kDownWaves) split *= 2;
    for (int u = wv; u < n_act * split; u += kDownWaves) {
        const MoeExpert ex = g.active[u / split];
        const int cnt = __popcll(ex.tokens);
        int k0, k1;
        share(g.I, Weights<I8>::kK, split, u % split, k0, k1);
        if (cnt <= 16) down_unit<I8, 1>(g, ex, cnt, n0, k0, k1, mine);
        else if (cnt <= 32) down_unit<I8, 2>(g, ex, cnt, n0, k0, k1, mine);
        else down_unit<I8, 4>(g, ex, cnt, n0, k0, k1, mine);
    }
    __syncthreads();
    const float *fs = reinterpret_cast<const float *>(sums);
    for (int i = tid; i < g.T * 16; i += kDownWaves * 64) {
        float s = 0.f;
        for (int v = 0; v < kDownWaves; ++v) s += fs[v * g.T * 16 + i];
        const int t = i >> 4, n = n0 + (i & 15);
        // a row whose weights are NaN (a NaN logit) is NaN, also where no
        // expert could be chosen
        if (g.weights[t * g.rule.k] != g.weights[t * g.rule.k])
            s = __builtin_nanf("");
        if (n < g.H) g.out[static_cast<int64_t>(t) * g.ldo + n] = f32_to_bf16(s);
    }
}

}  // namespace

hipError_t launch_moe_route(const MoeArgs &g, hipStream_t s) {
    const int rt = (g.T + 15) / 16;
    const dim3 rg((g.rule.E + 15) / 16), rb(kRouterWaves * 64);
    if (rt == 1) hipLaunchKernelGGL((k_router<1>), rg, rb, 0, s, g);
    else if (rt == 2) hipLaunchKernelGGL((k_router<2>), rg, rb, 0, s, g);
    else hipLaunchKernelGGL((k_router<4>), rg, rb, 0, s, g);
    hipError_t he = hipGetLastError();
    if (he != hipSuccess) return he;
    const dim3 cb(kChooseWaves * 64);
    switch (lane_slots(g.rule.E)) {
        case 1: hipLaunchKernelGGL((k_choose<1>), dim3(1), cb, 0, s, g); break;
        case 2: hipLaunchKernelGGL((k_choose<2>), dim3(1), cb, 0, s, g); break;
        case 4: hipLaunchKernelGGL((k_choose<4>), dim3(1), cb, 0, s, g); break;
        case 8: hipLaunchKernelGGL((k_choose<8>), dim3(1), cb, 0, s, g); break;
        default: hipLaunchKernelGGL((k_choose<16>), dim3(1), cb, 0, s, g); break;
    }
    return hipGetLastError();
}

hipError_t launch_moe_up(const MoeArgs &g, hipStream_t s) {
    const int rows = g.T * g.rule.k;
    const int most = g.rule.E < rows ? g.rule.E : rows;   // experts in use
    const dim3 gr((g.I + 15) / 16, most), bl(kUpWaves * 64);
    if (g.i8) hipLaunchKernelGGL((k_moe_up<true>), gr, bl, 0, s, g);
    else hipLaunchKernelGGL((k_moe_up<false>), gr, bl, 0, s, g);
    return hipGetLastError();
}

hipError_t launch_moe_down(const MoeArgs &g, hipStream_t s) {
    const dim3 gr((g.H + 15) / 16), bl(kDownWaves * 64);
    const size_t lds = sizeof(float) * 16 * kDownWaves * g.T;
    if (g.i8) hipLaunchKernelGGL((k_moe_down<true>), gr, bl, lds, s, g);
    else hipLaunchKernelGGL((k_moe_down<false>), gr, bl, lds, s, g);
    return hipGetLastError();
}

}  // namespace ue
