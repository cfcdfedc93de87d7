// Balance loss of packed sequences (ue_balance) and the gradient of the
// router's logits (ue_balance_backward).
//
// With p_t the scores of token t (softmax, or sigmoids over their sum) and c_e
// the assignments to expert e in a sequence of n tokens:
//   loss = E / (k n^2) sum_e c_e sum_t p_te
//   dl_te = dloss E / (k n^2) p_te (c_e - sum_j p_tj c_j) [1 - sigmoid(l_te)]
// Counts are constants, so the forward pass is one over the logits and ids that
// sums p and counts ids, and the backward pass one over the logits.
//
// L lanes share a token, VP experts each, 64 / L tokens per wave; a lane's
// experts are the same for every token, so it adds their p in registers. Sums
// are in a fixed order without atomics on values: a workgroup takes a share of
// consecutive tokens and writes one row of partial sums for every sequence it
// meets. Share c and sequence s meet in slot c + s: going along the tokens
// either grows by one, so no two meetings share a slot, and shares + sequences
// slots are enough for any lengths. A second launch adds a sequence's rows,
// shares in order.
//
// Bound: 65536 tokens of 256 experts, fp32, sigmoid: HBM going back (23 us, 134 MB,
// 5.8 TB/s); forward (25 us, 69 MB, of which 4.5 are the launch that adds the partial
// sums) about half instruction issue (20 per logit, 5.2 M a wave's: 8-9 us of the 21,
// 11 with the quarter-rate exponentials and reciprocals) and half latency: eight
// tokens of a wave one after another with one ahead, the ids' counts ahead of the
// first, a workgroup's start and end; which of them most has not been measured. A few
// thousand tokens are bound by the latency of the launches (3001 tokens of 60
// experts 10.6 us, back 7), a few hundred take one launch, which the host's calls
// outlast.
#include "ue_train.h"

namespace ue {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Lane `at` holds runs of four experts, L runs apart, so that it loads 16 bytes (8
// of bf16) and the lanes of a token 64 and more side by side. Place of slot i:
template <int L>
__device__ __forceinline__ int place_of_slot(int at, int i) {
    return 4 * (at + L * (i / 4)) + i % 4;
}
// A place is its expert, but for the last run: where the experts do not fill it, it
// holds the last four, and the first of those are another run's as well and not
// looked at. So every run is loaded without a branch (2221 tokens of 442 experts
// 14.6 us and back 6.9, with branches on a run's length 15.6 and 8.2). RUNS: E >=
// 4; with fewer experts, element by element, places are experts.
template <bool RUNS>
__device__ __forceinline__ int run_begin(int place, int E) {
    return RUNS && place > E - 4 ? (place < E ? E - 4 : 0) : place;
}
template <bool RUNS>
__device__ __forceinline__ int place_of_expert(int e, int E) {
    return !RUNS || e < (E & ~3) ? e : e + 4 - (E & 3);
}
// Whether slot i of a run (its first place's) is its lane's to look at.
template <bool RUNS>
__device__ __forceinline__ bool own_slot(int place, int i, int E) {
    return RUNS ? place < E && i >= place + 4 - E : place + i < E;
}

// The logits of one row that lane `at` holds, as they lie there, and as floats,
// -inf in slots that are not its own. (Whatever looks at them waits for them.)
template <typename T, int L, int VP, bool RUNS>
struct Token {
    typedef typename Words<4 * sizeof(T)>::type W;
    W v[VP / 4];

    __device__ __forceinline__ void load(const T *row, int at, int E) {
#pragma unroll
        for (int c = 0; c < VP / 4; ++c) {
            const int e = place_of_slot<L>(at, 4 * c);
            if constexpr (RUNS) {
                v[c] = *reinterpret_cast<const W *>(row + run_begin<RUNS>(e, E));
            } else {
                struct { T e[4]; } few = {};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) few.e[i] = row[e + i];
                v[c] = __builtin_bit_cast(W, few);
            }
        }
    }
    __device__ __forceinline__ void get(int at, int E, float (&x)[VP]) const {
#pragma unroll
        for (int c = 0; c < VP / 4; ++c) {
            struct Elements { T e[4]; };
            const Elements f = __builtin_bit_cast(Elements, v[c]);
            const int e = place_of_slot<L>(at, 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 * c + i] = own_slot<RUNS>(e, i, E) ? widen<T>(f.e[i]) : -__builtin_inff();
        }
    }
};

// Scores of a token in place of its logits, 0 where all are masked, but for the
// factor that is returned; `slope`: 1 - sigmoid (untouched for the softmax).
template <int L, int VP, bool SIGMOID, bool SLOPE>
__device__ __forceinline__ float scores(float (&x)[VP], float (&slope)[SLOPE ? VP : 1]) {
    float sum = 0.f;
    if (SIGMOID) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            // (an infinite exponential leaves a score of 0; the slope is 1 there,
            // and where the reciprocal is no normal number)
            const float e = exp_of(-x[i]), r = __builtin_amdgcn_rcpf(1.0f + e);
            if constexpr (SLOPE) slope[i] = e > 0x1p125f ? 1.0f : e * r;
            x[i] = r;
            sum += x[i];
        }
        sum = lanes_sum<L>(sum) + 1e-20f;
    } else {
        float top = x[0];
#pragma unroll
        for (int i = 1; i < VP; ++i) top = fmaxf(top, x[i]);
        top = finite_top(lanes_max<L>(top));
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            x[i] = x[i] == -__builtin_inff() ? 0.f : exp_of(finite_top(x[i]) - top);
            sum += x[i];
        }
        sum = lanes_sum<L>(sum);
        if (sum == 0.f) sum = 1.f;
    }
    return 1.0f / sum;
}

// Experts of a row of partial sums: rows in pieces of four.
__device__ __forceinline__ int padded(int E) { return (E + 3) & ~3; }

// Bounds of sequences, clamped to the tokens there are. What is asked for by a
// whole wave alike comes, of up to 63 sequences, from one load that every lane
// makes at the start (the loads that follow on each other are what bounds of
// sequences cost).
struct Sequences {
    const int32_t *offsets;
    int T, n;
    int held;                   // begin(lane), if there are few
    __device__ __forceinline__ int begin(int s) const {
        if (!offsets) return s ? T : 0;
        const int o = offsets[s];
        return o < 0 ? 0 : o > T ? T : o;
    }
    __device__ __forceinline__ Sequences(const int32_t *o, int T, int n, int lane)
        : offsets(o), T(T), n(n), held(0) {
        if (n < 64) held = begin(lane < n ? lane : n);
    }
    __device__ __forceinline__ int begin_wave(int s) const {
        return n < 64 ? __builtin_amdgcn_readlane(held, s) : begin(s);
    }
    // the first sequence that ends behind token t, all lanes of a wave looking for
    // the same: of 64 at once
    __device__ __forceinline__ int find_wave(int t, int lane) const {
        if (n < 64) {
            const uint64_t m = __ballot(lane > 0 && lane <= n && held > t);
            return m ? __builtin_ctzll(m) - 1 : n;
        }
        int lo = 0, hi = n;
        while (lo < hi) {
            const int step = (hi - lo + 63) >> 6, last = lo + (lane + 1) * step - 1;
            // lane i: does sequence lo + (i + 1) step - 1 end behind t?
            const uint64_t m = __ballot(last >= hi || begin(last + 1) > t);
            if (m == 0) return hi;
            const int i = __builtin_ctzll(m), from = lo + i * step;
            hi = from + step - 1 < hi ? from + step - 1 : hi;
            lo = from;
        }
        return lo;
    }
    // the same, for a lane on its own
    __device__ __forceinline__ int find(int t) const {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (begin(mid + 1) > t) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
};

constexpr int kFwdWaves = 8, kFwdBlock = kFwdWaves * 64;

// WHOLE: a workgroup per sequence, which writes the results itself.
template <typename T, int L, int VP, bool SIGMOID, bool WHOLE>
__global__ __launch_bounds__(kFwdBlock) void k_balance(BalanceArgs g) {
    constexpr int kEach = 64 / L, kAll = L * VP;
    __shared__ float sums[kFwdWaves][kAll];
    __shared__ int hist[kAll];
    const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
    const int at = lane & (L - 1), sub = lane / L, E = g.E;
    const Sequences seqs(g.offsets, g.T, g.n_seq, lane);
    const int c = blockIdx.x, t0 = WHOLE ? 0 : c * g.chunk;
    const int t1 = WHOLE || g.T - t0 < g.chunk ? g.T : t0 + g.chunk;
    const T *logits = static_cast<const T *>(g.logits);
    // (the next sequence is looked for behind this one's end, past any number of
    // empty ones; offsets that decrease may not lead back)
    for (int s = WHOLE ? c : seqs.find_wave(t0, lane), after; s < g.n_seq; s = after) {
        int a = seqs.begin_wave(s), b = seqs.begin_wave(s + 1);
        after = g.n_seq;
        if constexpr (!WHOLE) {
            if (a >= t1) break;
            if (b < t1) {
                after = seqs.find_wave(b, lane);
                after = after > s ? after : s + 1;
            }
            a = a > t0 ? a : t0;
            b = b < t1 ? b : t1;
            if (a >= b) continue;
        }
        for (int e = tid; e < E; e += kFwdBlock) hist[e] = 0;
        __syncthreads();
        float acc[VP] = {};
        constexpr int kStep = kFwdWaves * kEach;
        // a token's logits are on their way while the one before is summed, the
        // first ones' while the ids are counted
        auto tokens = [&](auto runs) {
            typedef Token<T, L, VP, decltype(runs)::value> Logits;
            Logits now, next;
            float x[VP], none[1];
            auto load = [&](int t, Logits &to) {
                const int mine = t + sub < b ? t + sub : b - 1;
                to.load(logits + mine * g.ld, at, E);
            };
            int t = a + wv * kEach;
            if (t < b) load(t, now);
            for (int i = a * g.k + tid; i < b * g.k; i += kFwdBlock) {
                const int id = g.ids[i];
                if (static_cast<uint32_t>(id) < static_cast<uint32_t>(E))
                    atomicAdd(&hist[id], 1);
            }
            for (; t < b; t += kStep) {
                if (t + kStep < b) load(t + kStep, next);
                now.get(at, E, x);
                float inv = scores<L, VP, SIGMOID, false>(x, none);
                if (t + sub >= b) inv = 0.f;
#pragma unroll
                for (int i = 0; i < VP; ++i) acc[i] = __builtin_fmaf(x[i], inv, acc[i]);
                now = next;
            }
        };
        if (E >= 4) tokens(std::true_type{});
        else tokens(std::false_type{});
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const float all = sum_across<L>(acc[i]);
            if (sub == 0) sums[wv][place_of_slot<L>(at, i)] = all;
        }
        __syncthreads();
        const int64_t slot = static_cast<int64_t>(WHOLE ? s : c + s) * (WHOLE ? E : padded(E));
        const float inv_n = b > a ? 1.0f / static_cast<float>(b - a) : 0.f;
        float term = 0.f;
        for (int e = tid; e < E; e += kFwdBlock) {
            const int at_place = E >= 4 ? place_of_expert<true>(e, E) : e;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kFwdWaves; ++w) v += sums[w][at_place];
            const int n = hist[e];
            if constexpr (WHOLE) {
                v *= inv_n;
                g.prob[slot + e] = v;
                g.counts[slot + e] = n;
                term += static_cast<float>(n) * v;
            } else {
                g.part[slot + e] = v;
                g.part_n[slot + e] = n;
            }
        }
        if constexpr (WHOLE) {
            __shared__ float terms[kFwdWaves];
            term = lanes_sum<64>(term);
            if (lane == 0) terms[wv] = term;
            __syncthreads();
            if (tid == 0) {
                float all = 0.f;
#pragma unroll
                for (int w = 0; w < kFwdWaves; ++w) all += terms[w];
                g.loss[s] = all * (static_cast<float>(E) / static_cast<float>(g.k)) * inv_n;
            }
        }
        __syncthreads();
    }
}

// Adds a sequence's rows of partial sums: wave w takes shares w, w + kEndWaves,
// ... and 256 experts at a time.
constexpr int kEndWaves = 16, kEndBlock = kEndWaves * 64;

__global__ __launch_bounds__(kEndBlock) void k_balance_end(BalanceArgs g) {
    __shared__ float sums[kEndWaves][256];
    __shared__ int counts[kEndWaves][256];
    __shared__ float terms[4];
    const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6, E = g.E;
    const int s = blockIdx.x;
    const Sequences seqs(g.offsets, g.T, g.n_seq, lane);
    const int a = seqs.begin_wave(s), b = seqs.begin_wave(s + 1), n = b > a ? b - a : 0;
    const int c0 = n ? a / g.chunk : 0, c1 = n ? (b - 1) / g.chunk + 1 : 0;
    const float inv_n = n ? 1.0f / static_cast<float>(n) : 0.f;
    float term = 0.f;
    for (int e0 = 0; e0 < E; e0 += 256) {
        float v[4] = {};
        int m[4] = {};
        // four experts of a lane, four shares at once
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        const int EP = padded(E), e = e0 + 4 * lane < EP ? e0 + 4 * lane : 0;
        for (int c = c0 + wv; c < c1; c += 4 * kEndWaves) {
            f32x4 p[4];
            i32x4 n4[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int cc = c + u * kEndWaves < c1 ? c + u * kEndWaves : c;
                const int64_t slot = static_cast<int64_t>(cc + s) * EP + e;
                p[u] = *reinterpret_cast<const f32x4 *>(g.part + slot);
                n4[u] = *reinterpret_cast<const i32x4 *>(g.part_n + slot);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c + u * kEndWaves < c1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] += p[u][i];
                        m[i] += n4[u][i];
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sums[wv][4 * lane + i] = v[i];
            counts[wv][4 * lane + i] = m[i];
        }
        __syncthreads();
        if (tid < 256 && e0 + tid < E) {
            float total = 0.f;
            int count = 0;
#pragma unroll
            for (int w = 0; w < kEndWaves; ++w) {
                total += sums[w][tid];
                count += counts[w][tid];
            }
            const int64_t o = static_cast<int64_t>(s) * E + e0 + tid;
            g.counts[o] = count;
            const float mean = total * inv_n;
            g.prob[o] = mean;
            term += static_cast<float>(count) * mean;
        }
        __syncthreads();
    }
    if (tid < 256) {
        term = lanes_sum<64>(term);
        if (lane == 0) terms[wv] = term;
    }
    __syncthreads();
    if (tid == 0)
        g.loss[s] = ((terms[0] + terms[1]) + (terms[2] + terms[3])) *
                    (static_cast<float>(E) / static_cast<float>(g.k)) * inv_n;
}

template <typename T, int L, int VP, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void k_balance_backward(BalanceBackArgs g, int chunk) {
    constexpr int kEach = 64 / L;
    const int lane = lane_id(), wv = threadIdx.x >> 6;
    const int at = lane & (L - 1), sub = lane / L, E = g.E;
    const Sequences seqs(g.offsets, g.T, g.n_seq, lane);
    const int t0 = blockIdx.x * chunk;
    const int t1 = g.T - t0 < chunk ? g.T : t0 + chunk;
    const T *logits = static_cast<const T *>(g.logits);
    T *out = static_cast<T *>(g.dlogits);
    auto tokens = [&](auto runs) {
        constexpr bool RUNS = decltype(runs)::value;
        int t = t0 + wv * kEach + sub;
        // this token's sequence; its counts times what its gradient is scaled with
        int s = 0, from = 0, to = -1;
        float cw[VP] = {};
        for (; t - sub < t1; t += kWaves * kEach) {
            const bool real = t < t1;
            const int mine = real ? t : t1 - 1;
            float x[VP], slope[VP];
            Token<T, L, VP, RUNS> token;
            token.load(logits + mine * g.ld, at, E);
            const bool look = real && t >= to;
            if (__any(look)) {
                if (g.n_seq < 64) {
                    // the tokens of the wave one by one, without a load
#pragma unroll
                    for (int u = 0; u < kEach; ++u) {
                        const int tu = __builtin_amdgcn_readfirstlane(t - sub) + u;
                        const int su = seqs.find_wave(tu, lane);
                        const bool past = su >= g.n_seq;
                        const int a = past ? g.T : seqs.begin_wave(su);
                        const int b = past ? g.T : seqs.begin_wave(su + 1);
                        if (look && sub == u) {
                            s = su;
                            from = a;
                            to = b;
                        }
                    }
                } else {
                    // the sequence of the wave's first token is most tokens'
                    const int tw = __builtin_amdgcn_readfirstlane(t - sub);
                    const int sw = seqs.find_wave(tw, lane);
                    const bool past = sw >= g.n_seq;
                    const int a = past ? g.T : seqs.begin(sw);
                    const int b = past ? g.T : seqs.begin(sw + 1);
                    if (look && t < b) {
                        s = sw;
                        from = a;
                        to = b;
                    } else if (look) {
                        s = seqs.find(t);
                        from = s < g.n_seq ? seqs.begin(s) : g.T;
                        to = s < g.n_seq ? seqs.begin(s + 1) : g.T;
                    }
                }
                // (behind the last sequence from and to are T)
                if (look && s < g.n_seq) {
                    const float n = static_cast<float>(to - from);
                    const float f = g.dloss[s] *
                        (static_cast<float>(E) / (static_cast<float>(g.k) * n)) / n;
                    const int32_t *counts = g.counts + static_cast<int64_t>(s) * E;
#pragma unroll
                    for (int c = 0; c < VP / 4; ++c) {
                        const int e = place_of_slot<L>(at, 4 * c);
                        typedef int32_t Four __attribute__((ext_vector_type(4), aligned(4)));
                        Four q = {};
                        if (RUNS) {
                            q = *reinterpret_cast<const Four *>(counts + run_begin<RUNS>(e, E));
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (e + i < E) q[i] = counts[e + i];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cw[4 * c + i] = own_slot<RUNS>(e, i, E) ? static_cast<float>(q[i]) * f
                                                                    : 0.f;
                    }
                }
            }
            const bool inside = real && t >= from && t < to;
            token.get(at, E, x);
            const float inv = scores<L, VP, SIGMOID, true>(x, slope);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                x[i] *= inv;
                dot = __builtin_fmaf(x[i], cw[i], dot);
            }
            dot = lanes_sum<L>(dot);
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                x[i] *= cw[i] - dot;
                if (SIGMOID) x[i] *= slope[i];
                if (!inside) x[i] = 0.f;
            }
            if (!real || (g.accumulate && !inside)) continue;
            T *row = out + t * g.ld_out;
#pragma unroll
            for (int c = 0; c < VP / 4; ++c) {
                const int e = place_of_slot<L>(at, 4 * c), begin = run_begin<RUNS>(e, E);
                if (e >= E) continue;
                const int n = RUNS ? 4 : E - e;
                float f[4];
                if (g.accumulate) load_run<4, false>(row + begin, n, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = (g.accumulate ? f[i] : 0.f) + x[4 * c + i];
                if (begin == e) {
                    store_run<4, true>(row + e, n, f);
                } else {
#pragma unroll
                    for (int i = 1; i < 4; ++i)
                        if (own_slot<RUNS>(e, i, E)) row[begin + i] = narrow<T>(f[i]);
                }
            }
        }
    };
    if (E >= 4) tokens(std::true_type{});
    else tokens(std::false_type{});
}

// The lanes and slots that hold E experts: f<L, VP>().
template <class F>
void with_lanes(int E, F f) {
    if (E <= 32) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
    else if (E <= 64) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
    else if (E <= 128) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 16>{});
    else if (E <= 256) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
    else if (E <= 512) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

template <typename T, bool SIGMOID>
void balance_any(const BalanceArgs &g, int shares, hipStream_t s) {
    with_lanes(g.E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, VP = decltype(v)::value;
        if (g.part)
            hipLaunchKernelGGL((k_balance<T, L, VP, SIGMOID, false>), dim3(shares),
                               dim3(kFwdBlock), 0, s, g);
        else
            hipLaunchKernelGGL((k_balance<T, L, VP, SIGMOID, true>), dim3(g.n_seq),
                               dim3(kFwdBlock), 0, s, g);
    });
}

template <typename T, bool SIGMOID>
void backward_any(const BalanceBackArgs &g, int chunk, int shares, hipStream_t s) {
    with_lanes(g.E, [&](auto l, auto v) {
        hipLaunchKernelGGL((k_balance_backward<T, decltype(l)::value, decltype(v)::value, SIGMOID>),
                           dim3(shares), dim3(kBlock), 0, s, g, chunk);
    });
}

}  // namespace

// Tokens that a workgroup passes over at once.
static int pass(int E) { return E <= 128 ? 64 : E <= 256 ? 32 : E <= 512 ? 16 : 8; }

// A share per CU, of one pass at least: a workgroup's start and end cost more than
// waves beside it hide (65536 tokens of 256 experts 26 us, two shares per CU 27.5,
// four 35; of at least 64 tokens 2221 tokens of 442 experts took 23 us, of one
// pass, 16 of them, 18).
int balance_chunk(int T, int E, int num_cu) {
    const int each = (T + num_cu - 1) / num_cu;
    return each <= pass(E) ? pass(E) : (each + 15) / 16 * 16;
}
// Batches of up to eight passes are left to a workgroup per sequence, without
// partial sums and the launch that adds them.
int64_t balance_slots(int T, int n_seq, int E, int num_cu) {
    if (T <= 8 * pass(E)) return 0;
    const int c = balance_chunk(T, E, num_cu);
    return (static_cast<int64_t>(T) + c - 1) / c + n_seq;
}

hipError_t launch_balance(ue_ctx &c, const BalanceArgs &a, hipStream_t s) {
    if (a.n_seq == 0) return hipSuccess;
    BalanceArgs g = a;
    g.chunk = balance_chunk(g.T, g.E, c.num_cu);
    const int shares = (g.T + g.chunk - 1) / g.chunk;
    if (g.bf16)
        g.sigmoid ? balance_any<uint16_t, true>(g, shares, s)
                  : balance_any<uint16_t, false>(g, shares, s);
    else
        g.sigmoid ? balance_any<float, true>(g, shares, s)
                  : balance_any<float, false>(g, shares, s);
    const hipError_t he = hipGetLastError();
    if (he != hipSuccess || !g.part) return he;
    tmark(&c, s);
    hipLaunchKernelGGL(k_balance_end, dim3(g.n_seq), dim3(kEndBlock), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const ue_ctx &c, const BalanceBackArgs &g,
                                   hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    // eight workgroups' shares per CU
    const int chunk = (g.T + 8 * c.num_cu - 1) / (8 * c.num_cu) < 16
                          ? 16 : (g.T + 8 * c.num_cu - 1) / (8 * c.num_cu);
    const int shares = (g.T + chunk - 1) / chunk;
    if (g.bf16)
        g.sigmoid ? backward_any<uint16_t, true>(g, chunk, shares, s)
                  : backward_any<uint16_t, false>(g, chunk, shares, s);
    else
        g.sigmoid ? backward_any<float, true>(g, chunk, shares, s)
                  : backward_any<float, false>(g, chunk, shares, s);
    return hipGetLastError();
}

}  // namespace ue
