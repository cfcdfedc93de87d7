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
// of h (the only sums or values of the layer held in fewer than 32), and the
// layer's result is rounded once, at the end. That costs 8% of the second
// product's time (532 against 492 us in the batch below, three shares)
// and takes the layer's error from 1.4 roundings to one. An expert with more
// than 16 tokens takes passes of 16, its matrices read again from cache.
//
// Bound: HBM reads, 6.9 TB/s at most on this device. Layer of 256 experts,
// top-8, H=7168, I=2048: 32 tokens, bf16, 96 experts in use: router and choice
// 18 us, first product 850 us (6.6 TB/s), second 495 (5.7), join 5. One token,
// int8: 13, 43 (5.5) and 25 us (4.7), where each kernel's start and end weigh.
// The first product reads exactly its matrices (5.64 GB of 5.64), the second 3%
// more than its own (the hidden activations, once per L2).
#include "ue_rows.h"

namespace ue {
namespace {

// K split over W waves in whole steps: wave v's share.
__device__ __forceinline__ void share(int K, int step, int W, int v, int &k0,
                                      int &k1) {
    const int n = (K + step - 1) / step;
    const int per = (n + W - 1) / W;
    k0 = v * per * step;
    k1 = (v + 1) * per * step;
    k1 = k1 < n * step ? k1 : n * step;
}

// ---- choice ----------------------------------------------------------------
// Every token's experts and weights, one wave per token; the workgroup that
// ends last then lists the experts in use with their tokens (one 64-bit set
// per expert) and the rows of all chosen (expert, token) pairs. Up to
// kChooseWaves tokens are chosen by the router's last workgroup, without a
// launch of their own.
constexpr int kChooseWaves = 4;
constexpr int kRouterK = 1024;           // of K per workgroup of the router

__host__ __device__ inline int router_parts(int hidden) {
    return (hidden + kRouterK - 1) / kRouterK;
}

// Whether this workgroup is the last of `all` to get here; what the others
// wrote before is then visible. (The counter returns to zero: the next call,
// or graph replay, starts anew.)
// One wave releases and acquires for the workgroup, on either side of a
// barrier: a fence writes back or invalidates a whole L2, and one in every
// wave made the choice 11 us instead of 5. Each wave waits for its own stores
// ahead of the first barrier.
__device__ __forceinline__ bool ends_last(uint32_t *done, uint32_t all, int *sh) {
    wait_stores();
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL,
                                                 __HIP_MEMORY_SCOPE_AGENT) == all - 1;
        if (last)
            __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *sh = last;
    }
    __syncthreads();
    return *sh;
}

struct ChooseLds {
    unsigned long long set[kMaxExperts];
    int base[kMaxExperts];
    // one workgroup's choices stay here until they are listed
    int32_t ids[kChooseWaves * 64];
    float weights[kChooseWaves * 64];
    int last;
};

// The choice of tokens t0 .. t0 + kChooseWaves - 1 by one workgroup of
// `blocks`.
template <int V>
__device__ __forceinline__ void choose(const MoeArgs &g, int t0, int blocks,
                                       ChooseLds &sh) {
    const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
    const int E = g.rule.E, k = g.rule.k, parts = router_parts(g.H);
    constexpr int kBatch = V <= 4 ? 8 : 32 / V;      // parts loaded together
    const int t = t0 + wv;
    const bool one = blocks == 1 && k <= 64;
    int32_t *ids = one ? sh.ids : g.ids;
    float *weights = one ? sh.weights : g.weights;
    if (t < g.T) {
        const float *lg = g.logits + static_cast<int64_t>(t) * E;
        float x[V], bias[V];
        load_bias<V>(g.rule, bias);
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = lane * V + i < E ? 0.f : -__builtin_inff();
        for (int p0 = 0; p0 < parts; p0 += kBatch) {
            float v[kBatch][V];
#pragma unroll
            for (int p = 0; p < kBatch; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane * V + i;
                    v[p][i] = p0 + p < parts && e < E
                                  ? lg[static_cast<int64_t>(p0 + p) * g.T * E + e]
                                  : 0.f;
                }
#pragma unroll
            for (int p = 0; p < kBatch; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] += v[p][i];
        }
        gate_row<V>(g.rule, x, bias, ids + t * k, weights + t * k, [](int) {});
    }
    if (blocks > 1 && !ends_last(g.done, blocks, &sh.last)) return;
    for (int e = tid; e < E; e += kChooseWaves * 64) sh.set[e] = 0;
    __syncthreads();
    for (int a = tid; a < g.T * k; a += kChooseWaves * 64) {
        const int e = ids[a];
        if (one) {
            g.ids[a] = e;
            g.weights[a] = weights[a];
        }
        if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E))
            atomicOr(&sh.set[e], 1ull << (a / k));
    }
    __syncthreads();
    // experts in use, in id order, and where their tokens start: one wave,
    // 64 experts at a time
    if (wv == 0) {
        int n_act = 0, rows = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const unsigned long long s = e < E ? sh.set[e] : 0;
            const int c = __popcll(s);
            const uint64_t used = __ballot(c > 0);
            const int incl = wave_inclusive_sum(c);
            if (e < E) sh.base[e] = rows + incl - c;
            if (c > 0)
                g.active[n_act + mask_rank(used)] = MoeExpert{s, e, rows + incl - c};
            n_act += __popcll(used);
            rows += __builtin_amdgcn_readlane(incl, 63);
        }
        if (lane == 0) *g.n_active = n_act;
    }
    __syncthreads();
    // the weight of each (expert, token) row, and the token
    for (int a = tid; a < g.T * k; a += kChooseWaves * 64) {
        const int e = ids[a], tok = a / k;
        if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E)) continue;
        const int r = sh.base[e] + __popcll(sh.set[e] & ((1ull << tok) - 1));
        g.row_weight[r] = weights[a];
        g.row_token[r] = tok;
    }
}

template <int V>
__global__ __launch_bounds__(kChooseWaves * 64) void k_choose(MoeArgs g) {
    __shared__ ChooseLds sh;
    choose<V>(g, blockIdx.x * kChooseWaves, gridDim.x, sh);
}

// ---- router ---------------------------------------------------------------
// Part sums of the logits of 16 experts per workgroup: K is split over the
// workgroups of a column of the grid and their waves, for enough loads in
// flight (256 experts alone make 16 workgroups: 16 us at K = 7168 and one
// token, against 5 split). The choice adds the parts in order.
constexpr int kRouterWaves = 4;
static_assert(kRouterWaves == kChooseWaves, "the router's last workgroup chooses");

// V: lane slots of the choice made here, 0 for none (see k_choose).
template <int FOLD, int RT, int V>
__global__ __launch_bounds__(kRouterWaves * 64) void k_router(MoeArgs g) {
    typedef RowStream<Bf16Rows, 1, FOLD, RT, 1> S;
    __shared__ f32x4 part[kRouterWaves][S::kAcc][64];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int E = g.rule.E, e0 = blockIdx.x * 16;
    const char *w[1] = {reinterpret_cast<const char *>(g.router)};
    const char *x[1] = {reinterpret_cast<const char *>(g.x)};
    uint32_t wo[S::LD], xo[RT];
#pragma unroll
    for (int j = 0; j < S::LD; ++j) {
        const int e = e0 + S::row(j);
        wo[j] = 2u * (e < E ? e : E - 1) * g.H;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int t = S::token(r);
        xo[r] = 2u * (t < g.T ? t : g.T - 1) * static_cast<uint32_t>(g.ldx);
    }
    f32x4 acc[1][S::kAcc] = {};
    const int k0 = blockIdx.y * kRouterK + wv * (kRouterK / kRouterWaves);
    const int k1 = k0 + kRouterK / kRouterWaves;
    S::run(w, wo, x, xo, k0, k1 < g.H ? k1 : g.H, g.H, acc);
#pragma unroll
    for (int r = 0; r < S::kAcc; ++r) part[wv][r][lane] = acc[0][r];
    __syncthreads();
    const float *f = reinterpret_cast<const float *>(part);
    for (int i = tid; i < 16 * g.T; i += kRouterWaves * 64) {
        const int n = i & 15, t = i >> 4;
        if (e0 + n >= E) continue;
        float sum = 0.f;
        for (int v = 0; v < kRouterWaves; ++v)
#pragma unroll
            for (int b = 0; b < S::kParts; ++b) {
                int a, at;
                S::where(n, t, b, a, at);
                sum += f[(v * S::kAcc + a) * 256 + at];
            }
        g.logits[(static_cast<int64_t>(blockIdx.y) * g.T + t) * E + e0 + n] = sum;
    }
    if constexpr (V > 0) {
        __shared__ ChooseLds sh;
        if (ends_last(g.done, gridDim.x * gridDim.y, &sh.last))
            choose<V>(g, 0, 1, sh);
    }
}

// ---- gate and up -------------------------------------------------------------
// 16 channels of one expert per workgroup, K split over the waves: with one
// token and eight experts of I=2048 that is 1,024 workgroups, four to a CU.
constexpr int kUpWaves = 4;

template <bool I8>
struct KindOf { typedef Bf16Rows type; };
template <>
struct KindOf<true> { typedef WideRows type; };

template <bool I8, int FOLD, int RT>
__device__ __forceinline__ void up_tile(const MoeArgs &g, const MoeExpert &a,
                                        int cnt, int n0, f32x4 *part) {
    typedef RowStream<typename KindOf<I8>::type, 2, FOLD, RT, 1> S;
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int kB = I8 ? 1 : 2;
    const char *mat = static_cast<const char *>(g.gate_up) +
                      a.expert * g.gate_up_stride * kB;
    const char *w[2] = {mat, mat + static_cast<int64_t>(g.I) * g.H * kB};
    const char *x[1] = {reinterpret_cast<const char *>(g.x)};
    uint32_t wo[S::LD], xo[RT];
#pragma unroll
    for (int j = 0; j < S::LD; ++j) {
        const int n = n0 + S::row(j) < g.I ? n0 + S::row(j) : g.I - 1;
        wo[j] = static_cast<uint32_t>(kB) * n * g.H;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        // the i-th token of the set, the last one past the end
        const int i = S::token(r);
        unsigned long long left = a.tokens;
        for (int c = 1; c < cnt; ++c)
            if (c <= i) left &= left - 1;
        xo[r] = 2u * __builtin_ctzll(left) * static_cast<uint32_t>(g.ldx);
    }
    f32x4 acc[2][S::kAcc] = {};
    int k0, k1;
    share(g.H, S::kWindow, kUpWaves, wv, k0, k1);
    S::run(w, wo, x, xo, k0, k1, g.H, acc);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < S::kAcc; ++r)
            part[((wv * 2 + m) * S::kAcc + r) * 64 + lane] = acc[m][r];
    __syncthreads();
    const float *f = reinterpret_cast<const float *>(part);
    for (int o = tid; o < 16 * cnt; o += kUpWaves * 64) {
        const int n = o & 15, t = o >> 4, nn = n0 + n;
        if (nn >= g.I) continue;
        float v[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            v[m] = 0.f;
            for (int u = 0; u < kUpWaves; ++u)
#pragma unroll
                for (int b = 0; b < S::kParts; ++b) {
                    int c, at;
                    S::where(n, t, b, c, at);
                    v[m] += f[((u * 2 + m) * S::kAcc + c) * 256 + at];
                }
        }
        if (I8) {
            const float *sc = g.gate_up_scale + static_cast<int64_t>(a.expert) * 2 * g.I;
            v[0] *= sc[nn];
            v[1] *= sc[g.I + nn];
        }
        const float h = silu_of(v[0]) * v[1];
        // (a finite h that rounds to infinity takes the largest bf16 as its
        // first half; an infinite one has no finite rest)
        const bool finite = fabsf(h) <= __FLT_MAX__;
        uint16_t hi = f32_to_bf16(h);
        if (finite && (hi & 0x7FFFu) == 0x7F80u) --hi;
        const int64_t at = static_cast<int64_t>(a.base + t) * g.I + nn;
        g.h_hi[at] = hi;
        g.h_lo[at] = finite ? f32_to_bf16(h - bf16_to_f32(hi)) : 0;
    }
}

// MOST: tokens of the call at most 4, 8 or any number; one expert's tokens
// choose the product's form below that. (An instance for few tokens keeps its
// registers: with every form in it, it spilled.)
template <bool I8, int MOST>
__global__ __launch_bounds__(kUpWaves * 64, 4) void k_moe_up(MoeArgs g) {
    // (most: two matrices times four results)
    __shared__ f32x4 part[kUpWaves * 2 * 4 * 64];
    // (the table has room for every blockIdx.y: both reads at once)
    const MoeExpert ex = g.active[blockIdx.y];
    if (static_cast<int>(blockIdx.y) >= *g.n_active) return;
    const int cnt = __popcll(ex.tokens);
    const int n0 = blockIdx.x * 16;
    if (MOST <= 4 || cnt <= 4) {
        up_tile<I8, 4, 1>(g, ex, cnt, n0, part);
    } else if (MOST <= 8 || cnt <= 8) {
        if constexpr (MOST > 4) up_tile<I8, 2, 1>(g, ex, cnt, n0, part);
    } else if constexpr (MOST > 8) {
        for (int t0 = 0; t0 < cnt; t0 += 16) {
            MoeExpert some = ex;
            some.base += t0;
            for (int c = 0; c < t0; ++c) some.tokens &= some.tokens - 1;
            if (t0) __syncthreads();            // part is free again
            up_tile<I8, 1, 1>(g, some, cnt - t0 < 16 ? cnt - t0 : 16, n0, part);
        }
    }
}

// ---- down and weighted sum -----------------------------------------------------
// A workgroup makes 16 (or 8) output channels of every token, from the
// experts in use (or a share of them, blockIdx.y). A unit is an expert and a
// share of its K; each wave adds its units' weighted rows to its own sums
// (LDS), which are joined in wave order: no atomics, so the result does not
// depend on timing. With several shares of the experts their sums are joined
// by k_moe_join.
constexpr int kDownWaves = 8;

// REGIONS: sums of a wave that a folded product's parts may go to at once (4,
// or 1: the parts are added one after another). ROWS: channels of the
// workgroup.
template <bool I8, int FOLD, int ROWS, int REGIONS>
__device__ __forceinline__ void down_unit(const MoeArgs &g, const MoeExpert &a,
                                          int cnt, int n0, int split, int part,
                                          f32x4 *sum) {
    typedef RowStream<typename KindOf<I8>::type, 1, FOLD, 1, 2,
                      FOLD == 1 ? 0 : ROWS * FOLD / 16> S;
    const int lane = lane_id(), l16 = lane & 15, q = lane >> 4;
    constexpr int kB = I8 ? 1 : 2;
    const char *w[1] = {static_cast<const char *>(g.down) +
                        a.expert * g.down_stride * kB};
    const int64_t first = static_cast<int64_t>(a.base) * g.I;
    const char *x[2] = {reinterpret_cast<const char *>(g.h_hi + first),
                        reinterpret_cast<const char *>(g.h_lo + first)};
    uint32_t wo[S::LD], xo[1];
#pragma unroll
    for (int j = 0; j < S::LD; ++j) {
        const int n = n0 + S::row(j) < g.H ? n0 + S::row(j) : g.H - 1;
        wo[j] = static_cast<uint32_t>(kB) * n * g.I;
    }
    // this lane's token among the expert's, its weight, and the scales of the
    // channels it will hold: on their way while the products are made
    const int i = S::token(0), row = a.base + (i < cnt ? i : cnt - 1);
    xo[0] = 2u * (row - a.base) * g.I;
    const int t = g.row_token[row];
    const float wt = g.row_weight[row];
    // channel of value 0 in accumulator r: folded, the lanes whose row and
    // column parts agree hold 4 channels of a token
    constexpr int kRows = S::kRows;
    const int c0 = FOLD == 1 ? 4 * q : 4 * q % kRows;
    f32x4 scale[S::kAcc];
    if (I8) {
        const float *sc = g.down_scale + static_cast<int64_t>(a.expert) * g.H;
#pragma unroll
        for (int r = 0; r < S::kAcc; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + r * kRows + c0 + e;
                scale[r][e] = sc[n < g.H ? n : g.H - 1];
            }
    }
    f32x4 acc[1][S::kAcc] = {};
    int k0, k1;
    share(g.I, S::kWindow, split, part, k0, k1);
    S::run(w, wo, x, xo, k0, k1, g.I, acc);
    const int b = FOLD == 1 ? 0 : l16 / kRows;
    const bool mine = (FOLD == 1 || 4 * q / kRows == b) && i < cnt;
#pragma unroll
    for (int turn = 0; turn < (REGIONS == 1 ? S::kParts : 1); ++turn) {
        if (mine && (REGIONS > 1 || b == turn)) {
#pragma unroll
            for (int r = 0; r < S::kAcc; ++r) {
                f32x4 v = acc[0][r];
                if (I8) v *= scale[r];
                f32x4 &y = sum[((REGIONS > 1 ? b * g.T : 0) + t) * (ROWS / 4) +
                               (r * kRows + c0) / 4];
                y += v * wt;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// A row whose weights are NaN (a NaN logit) is NaN, also where no expert
// could be chosen.
__device__ __forceinline__ void store_token(const MoeArgs &g, int t, int n, float s) {
    const float w = g.weights[t * g.rule.k];
    g.out[static_cast<int64_t>(t) * g.ldo + n] =
        f32_to_bf16(w != w ? __builtin_nanf("") : s);
}

// MOST as in k_moe_up; ROWS: channels a workgroup makes.
template <bool I8, int MOST, int ROWS>
__global__ __launch_bounds__(kDownWaves * 64, 4) void k_moe_down(MoeArgs g, int most) {
    constexpr int kRows = ROWS, kRegions = MOST <= 8 ? 4 : 1;
    // sums [waves][regions][T][kRows / 4], then this share's experts (read
    // once: a read before each unit would hold its first loads back)
    extern __shared__ f32x4 sums[];
    MoeExpert *experts = reinterpret_cast<MoeExpert *>(
        sums + kDownWaves * kRegions * g.T * (kRows / 4));
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * kRows, each = kRegions * g.T * (kRows / 4);
    f32x4 *mine = sums + wv * each;
    for (int i = lane; i < each; i += 64) mine[i] = f32x4{0, 0, 0, 0};
    // this share of the experts (a single share reads the table without
    // waiting for how many entries count: it has `most`)
    if (gridDim.y == 1)
        for (int i = tid; i < most; i += kDownWaves * 64) experts[i] = g.active[i];
    const int n_all = *g.n_active, per = (n_all + gridDim.y - 1) / gridDim.y;
    const int a0 = blockIdx.y * per, left = n_all - a0;
    const int n_act = left < per ? (left > 0 ? left : 0) : per;
    if (gridDim.y > 1)
        for (int i = tid; i < n_act; i += kDownWaves * 64)
            experts[i] = g.active[a0 + i];
    __syncthreads();
    // shares of K so that few experts still occupy every wave
    int split = 1;
    while (n_act * split < kDownWaves && split < kDownWaves) split *= 2;
    for (int u = wv; u < n_act * split; u += kDownWaves) {
        MoeExpert ex = experts[u / split];
        ex.expert = __builtin_amdgcn_readfirstlane(ex.expert);
        ex.base = __builtin_amdgcn_readfirstlane(ex.base);
        const int cnt = __popcll(ex.tokens), part = u % split;
        if (MOST <= 4 || cnt <= 4) {
            down_unit<I8, 4, ROWS, kRegions>(g, ex, cnt, n0, split, part, mine);
        } else if (MOST <= 8 || cnt <= 8) {
            if constexpr (MOST > 4) down_unit<I8, 2, ROWS, kRegions>(g, ex, cnt, n0, split, part, mine);
        } else if constexpr (MOST > 8) {
            for (int t0 = 0; t0 < cnt; t0 += 16) {
                MoeExpert some = ex;
                some.base += t0;
                down_unit<I8, 1, ROWS, kRegions>(g, some, cnt - t0 < 16 ? cnt - t0 : 16, n0,
                                    split, part, mine);
            }
        }
    }
    __syncthreads();
    const float *fs = reinterpret_cast<const float *>(sums);
    for (int i = tid; i < g.T * kRows; i += kDownWaves * 64) {
        float s = 0.f;
        for (int v = 0; v < kDownWaves * kRegions; ++v) s += fs[v * g.T * kRows + i];
        const int t = i / kRows, n = n0 + i % kRows;
        if (n >= g.H) continue;
        if (gridDim.y > 1)
            g.part[(static_cast<int64_t>(blockIdx.y) * g.T + t) * g.H + n] = s;
        else
            store_token(g, t, n, s);
    }
}

__global__ __launch_bounds__(kBlock) void k_moe_join(MoeArgs g, int shares) {
    const int n = blockIdx.x * kBlock + threadIdx.x, t = blockIdx.y;
    if (n >= g.H) return;
    float s = 0.f;
    for (int p = 0; p < shares; ++p)
        s += g.part[(static_cast<int64_t>(p) * g.T + t) * g.H + n];
    store_token(g, t, n, s);
}

template <bool I8>
hipError_t up_any(const MoeArgs &g, dim3 gr, dim3 bl, hipStream_t s) {
    if (g.T <= 4) hipLaunchKernelGGL((k_moe_up<I8, 4>), gr, bl, 0, s, g);
    else if (g.T <= 8) hipLaunchKernelGGL((k_moe_up<I8, 8>), gr, bl, 0, s, g);
    else hipLaunchKernelGGL((k_moe_up<I8, kMoeTokens>), gr, bl, 0, s, g);
    return hipGetLastError();
}

template <bool I8, int MOST, int ROWS>
hipError_t down_as(const MoeArgs &g, int shares, hipStream_t s) {
    const int rows = g.T * g.rule.k;
    const int most = g.rule.E < rows ? g.rule.E : rows;   // experts in use
    const size_t lds = sizeof(float) * ROWS * kDownWaves * (MOST <= 8 ? 4 : 1) * g.T +
                       sizeof(MoeExpert) * ((most + shares - 1) / shares);
    hipLaunchKernelGGL((k_moe_down<I8, MOST, ROWS>),
                       dim3((g.H + ROWS - 1) / ROWS, shares),
                       dim3(kDownWaves * 64), lds, s, g, most);
    return hipGetLastError();
}

template <bool I8>
hipError_t down_any(const ue_ctx &c, const MoeArgs &g, int shares, hipStream_t s) {
    if (g.T > 8) return down_as<I8, kMoeTokens, 16>(g, shares, s);
    // 8 channels a workgroup where 16 would leave CUs without one (one bf16
    // token of H=2048, I=1024: 8.2 against 13.5 us; int8, H=7168, I=2048, where
    // it only doubles the reads of h: 32 against 24 us)
    const bool narrow = (g.H + 15) / 16 < c.num_cu;
    if (g.T > 4)
        return narrow ? down_as<I8, 8, 8>(g, shares, s)
                      : down_as<I8, 8, 16>(g, shares, s);
    return narrow ? down_as<I8, 4, 8>(g, shares, s)
                  : down_as<I8, 4, 16>(g, shares, s);
}

}  // namespace

int moe_router_parts(int hidden) { return router_parts(hidden); }

template <int V>
static hipError_t route_as(const MoeArgs &g, hipStream_t s) {
    const dim3 rg((g.rule.E + 15) / 16, moe_router_parts(g.H)), rb(kRouterWaves * 64);
    if (g.T <= kChooseWaves) {
        hipLaunchKernelGGL((k_router<4, 1, V>), rg, rb, 0, s, g);
        return hipGetLastError();
    }
    if (g.T <= 8) hipLaunchKernelGGL((k_router<2, 1, 0>), rg, rb, 0, s, g);
    else if (g.T <= 16) hipLaunchKernelGGL((k_router<1, 1, 0>), rg, rb, 0, s, g);
    else if (g.T <= 32) hipLaunchKernelGGL((k_router<1, 2, 0>), rg, rb, 0, s, g);
    else hipLaunchKernelGGL((k_router<1, 4, 0>), rg, rb, 0, s, g);
    const hipError_t he = hipGetLastError();
    if (he != hipSuccess) return he;
    hipLaunchKernelGGL((k_choose<V>), dim3((g.T + kChooseWaves - 1) / kChooseWaves),
                       dim3(kChooseWaves * 64), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_moe_route(const MoeArgs &g, hipStream_t s) {
    switch (lane_slots(g.rule.E)) {
        case 1: return route_as<1>(g, s);
        case 2: return route_as<2>(g, s);
        case 4: return route_as<4>(g, s);
        case 8: return route_as<8>(g, s);
        default: return route_as<16>(g, s);
    }
}

hipError_t launch_moe_up(const MoeArgs &g, hipStream_t s) {
    const int rows = g.T * g.rule.k;
    const int most = g.rule.E < rows ? g.rule.E : rows;   // experts in use
    const dim3 gr((g.I + 15) / 16, most), bl(kUpWaves * 64);
    return g.i8 ? up_any<true>(g, gr, bl, s) : up_any<false>(g, gr, bl, s);
}

// Shares of the experts in the second product: with more than 8 tokens many
// experts are in use, and eight workgroups for every CU level their load (32
// tokens, 96 experts in use, H=7168, I=2048, bf16: 505 us with five shares,
// 532 with three, 541 with two).
int moe_down_shares(int hidden, int T, int num_cu) {
    if (T <= 8) return 1;
    const int cols = (hidden + 15) / 16;
    const int want = (8 * num_cu + cols - 1) / cols;
    return want < 1 ? 1 : want > 8 ? 8 : want;
}

hipError_t launch_moe_down(const ue_ctx &c, const MoeArgs &g, hipStream_t s) {
    const int shares = moe_down_shares(g.H, g.T, c.num_cu);
    hipError_t he = g.i8 ? down_any<true>(c, g, shares, s)
                         : down_any<false>(c, g, shares, s);
    if (he != hipSuccess || shares == 1) return he;
    hipLaunchKernelGGL(k_moe_join, dim3((g.H + kBlock - 1) / kBlock, g.T),
                       dim3(kBlock), 0, s, g, shares);
    return hipGetLastError();
}

}  // namespace ue
