// Sum of the experts' rows back to their tokens (ue_combine) and its gradients
// (ue_combine_backward).
//
//   out_t = add_t + sum_j w_tj y[inv_tj];  dy[inv_tj] = w_tj dout_t;
//   dw_tj = <dout_t, y[inv_tj]>
//
// Forward: the lanes of one segment of one token's row load that segment of up
// to kJoin of its rows at once before they add them, in order. Backward: those of
// an assignment go along its row, a token's side by side, so that dout comes from
// the caches for all but the first; a dot is added by lanes, then over them, in a
// fixed order. Rows take a wave's 64 lanes or, short ones, 16 or 32 of them.
//
// Bound: HBM. 16384 tokens x top-8 x 7168, bf16: forward 367 us (2.1 GB, 5.7
// TB/s), backward 730 us (4.0 GB, 5.5 TB/s). A workgroup per token whose waves
// shared out the segments took 880 backward; four segments ahead in place of two
// 965, one 724 (but 10.9 us in place of 9.8 for 1021 tokens x top-6 x 1002,
// fp32); dout past the caches too 794.
#include "ue_train.h"

namespace ue {
namespace {

constexpr int kJoin = 8;      // rows of a token in flight
constexpr int kEach = 8;      // elements of a lane, in runs of 16 bytes

// A lane's elements of the LANES lanes' segment of a row that begins at h: runs
// lie lane after lane. A run that the row's end would cut lies at that end
// instead, and its first few elements, `over` of them, are others' and left
// alone: so all lanes load without a branch, whatever the row's length. (With
// branches on a run's length, rows' loads waited for each other: 1021 tokens x
// top-6 x 1002, fp32, 23 us both ways, without 18; 25517 x top-5 x 166 89 and 77;
// 16 and 59 with rows through the caches.)
// SHORT: rows of less than a run, element by element.
template <typename T, int LANES, bool SHORT>
struct Segment {
    static constexpr int kRun = 16 / sizeof(T), kRuns = kEach / kRun;
    typedef typename Words<16>::type W;
    W v[kRuns];

    static __device__ __forceinline__ int over(int h, int lane, int c, int H) {
        const int o = h + (c * LANES + lane + 1) * kRun - H;
        return !SHORT && o > 0 ? o : 0;
    }
    template <bool ONCE>
    __device__ __forceinline__ void load(const T *row, int h, int lane, int H) {
#pragma unroll
        for (int c = 0; c < kRuns; ++c) {
            const int at = h + (c * LANES + lane) * kRun;
            if constexpr (!SHORT) {
                const W *p = reinterpret_cast<const W *>(row + (at < H - kRun ? at : H - kRun));
                v[c] = ONCE ? __builtin_nontemporal_load(p) : *p;
            } else {
                struct { T e[kRun]; } few = {};
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (at + i < H) few.e[i] = row[at + i];
                v[c] = __builtin_bit_cast(W, few);
            }
        }
    }
    __device__ __forceinline__ void get(float (&f)[kEach]) const {
        struct Elements { T e[kEach]; };
        const Elements e = __builtin_bit_cast(Elements, v);
#pragma unroll
        for (int i = 0; i < kEach; ++i) f[i] = widen<T>(e.e[i]);
    }
    // Others' elements as zeros.
    static __device__ __forceinline__ void own(int h, int lane, int H, float (&f)[kEach]) {
        if (H % (LANES * kEach) == 0) return;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i % kRun < over(h, lane, i / kRun, H)) f[i] = 0.f;
    }
    static __device__ __forceinline__ void store(T *row, int h, int lane, int H,
                                                 const float (&f)[kEach]) {
#pragma unroll
        for (int c = 0; c < kRuns; ++c) {
            const int at = h + (c * LANES + lane) * kRun, o = over(h, lane, c, H);
            if (at >= H) continue;
            float r[kRun];
#pragma unroll
            for (int i = 0; i < kRun; ++i) r[i] = f[c * kRun + i];
            if (o == 0) {
                store_run<kRun, true>(row + at, H - at, r);
            } else {
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (i >= o) row[at - o + i] = narrow<T>(r[i]);
            }
        }
    }
};

// LANES: of a row's segment. Rows shorter than a wave's 512 elements share it.
template <typename T, int LANES, bool SHORT, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_combine(CombineArgs g, FastDiv segs, uint32_t items) {
    constexpr int kItems = kBlock / LANES;
    uint32_t item = blockIdx.x * kItems + threadIdx.x / LANES;
    if (LANES == 64) item = __builtin_amdgcn_readfirstlane(item);
    if (item >= items) return;
    const int t = div_by(item, segs);
    const int h = (item - t * segs.d) * LANES * kEach, lane = threadIdx.x % LANES;
    const int64_t o = static_cast<int64_t>(t) * g.k;
    const T *y = static_cast<const T *>(g.y);
    typedef Segment<T, LANES, SHORT> Seg;
    float sum[kEach] = {};
    Seg first;
    if (g.add) first.template load<ONCE>(static_cast<const T *>(g.add) + t * g.ldadd, h, lane, g.H);
    for (int j0 = 0; j0 < g.k; j0 += kJoin) {
        Seg rows[kJoin];
        float w[kJoin];
        bool has[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int at = j0 + j < g.k ? j0 + j : 0, pos = g.inv[o + at];
            has[j] = j0 + j < g.k && static_cast<uint32_t>(pos) < static_cast<uint32_t>(g.rows);
            w[j] = g.weights ? g.weights[o + at] : 1.f;
            if (has[j]) rows[j].template load<ONCE>(y + pos * g.ldy, h, lane, g.H);
        }
        if (j0 == 0 && g.add) first.get(sum);
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            if (!has[j]) continue;
            float f[kEach];
            rows[j].get(f);
#pragma unroll
            for (int i = 0; i < kEach; ++i) sum[i] = __builtin_fmaf(w[j], f[i], sum[i]);
        }
    }
    Seg::store(static_cast<T *>(g.out) + t * g.ldo, h, lane, g.H, sum);
}

constexpr int kAhead = 2;     // segments in flight
constexpr int kBackBlock = 512;

// Zeros in a row of dy, by the lanes of one.
template <typename T, int LANES, bool SHORT>
__device__ __forceinline__ void zero_row(const CombineArgs &g, int64_t row, int lane) {
    const float none[kEach] = {};
    for (int h = 0; h < g.H; h += LANES * kEach)
        Segment<T, LANES, SHORT>::store(static_cast<T *>(g.dy) + row * g.lddy, h, lane, g.H, none);
}

// Rows of dy that no assignment names, where all are to be written: the first
// `clear` workgroups of the launch (a power of two) take rows clear apart (the
// unnamed ones are often the last), find the named ones of theirs and write zeros to
// the others, while the rest of the launch writes the named ones.
// A few assignments are all looked at by each of these workgroups. Of many, a launch
// ahead notes for each row an assignment that names it: what was noted is true if
// that assignment does, and a row that none names holds anything, so the notes need
// not be cleared. Calls of top-8, all rows named, us without and with this:
//    32768 rows of 512 bytes      8.9    8.9    looked at
//    32768 rows of 16 KB        220    220
//    32776 rows of 512 bytes      8.9   12.1    noted
//   131072 rows of 240 bytes     17.0   20.7    (each assignment looked at: 25)
//   131072 rows of 16 KB        865    873
//   524288 rows of 240 bytes     66     76      (each assignment looked at: 102)
// Zeros in all of dy ahead of the launch took 11 us for the first of these, 23, 1276
// and 87 for the last three.
constexpr int kLookAt = 1 << 15;           // assignments
constexpr int kClearBlocks = 256, kClearRows = 4096;

template <typename T, int LANES, bool SHORT>
__device__ __forceinline__ void clear_unnamed(const CombineArgs &g) {
    __shared__ uint32_t named[kClearRows / 32];
    const uint32_t mine = blockIdx.x, rows = g.rows, all = g.all;
    const uint32_t shift = __builtin_ctz(g.clear);
    auto mark = [&](uint32_t i) { atomicOr(&named[i >> 5], 1u << (i & 31)); };
    // (rows counted in steps of `clear`; more than kClearRows of them only with notes)
    const uint32_t steps = mine < rows ? ((rows - 1 - mine) >> shift) + 1 : 0;
    for (uint32_t from = 0; from < steps; from += kClearRows) {
        const uint32_t n = steps - from < kClearRows ? steps - from : kClearRows;
        if (threadIdx.x < kClearRows / 32) named[threadIdx.x] = 0;
        __syncthreads();
        if (g.named_by) {
            for (uint32_t i = threadIdx.x; i < n; i += kBackBlock) {
                const uint32_t row = ((from + i) << shift) + mine, by = g.named_by[row];
                if (by < all && static_cast<uint32_t>(g.inv[by]) == row) mark(i);
            }
        } else {
            typedef uint32_t Four __attribute__((ext_vector_type(4), aligned(4)));
            constexpr uint32_t kLoads = 4;
            const uint32_t fours = all / 4;
            auto look = [&](uint32_t row) {
                if (row < rows && (row & (g.clear - 1)) == mine) mark(row >> shift);
            };
            for (uint32_t a = threadIdx.x; a < fours; a += kLoads * kBackBlock) {
                Four row[kLoads];
#pragma unroll
                for (uint32_t u = 0; u < kLoads; ++u) {
                    const uint32_t at = a + u * kBackBlock;
                    row[u] = *reinterpret_cast<const Four *>(g.inv + 4 * (at < fours ? at : a));
                    if (at >= fours) row[u] = ~Four{};
                }
#pragma unroll
                for (uint32_t u = 0; u < kLoads; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) look(row[u][e]);
            }
            if (threadIdx.x < (all & 3)) look(g.inv[4 * fours + threadIdx.x]);
        }
        __syncthreads();
        const int lane = threadIdx.x % LANES;
        for (uint32_t i = threadIdx.x / LANES; i < n; i += kBackBlock / LANES)
            if (!(named[i >> 5] >> (i & 31) & 1))
                zero_row<T, LANES, SHORT>(g, ((from + i) << shift) + mine, lane);
        __syncthreads();
    }
}

__global__ __launch_bounds__(kBlock) void k_combine_note(CombineArgs g) {
    const uint32_t a = blockIdx.x * kBlock + threadIdx.x;
    if (a >= g.all) return;
    const uint32_t row = g.inv[a];
    if (row < static_cast<uint32_t>(g.rows)) g.named_by[row] = a;
}

// (four workgroups of rows of 64 lanes per CU, which 65 registers of fp32 rows
// would make three)
template <typename T, int LANES, bool SHORT, bool ONCE>
__global__ __launch_bounds__(kBackBlock, LANES == 64 ? 8 : 6) void k_combine_backward(
    CombineArgs g, FastDiv topk, uint32_t assignments) {
    constexpr int kItems = kBackBlock / LANES, kSeg = LANES * kEach;
    if (blockIdx.x < g.clear) {
        clear_unnamed<T, LANES, SHORT>(g);
        return;
    }
    uint32_t a = (blockIdx.x - g.clear) * kItems + threadIdx.x / LANES;
    if (LANES == 64) a = __builtin_amdgcn_readfirstlane(a);
    if (a >= assignments) return;                   // (whole rows of lanes)
    const int lane = threadIdx.x % LANES, t = div_by(a, topk);
    const T *dout = static_cast<const T *>(g.dout) + t * g.lddout;
    const int pos = g.inv[a];
    const float w = g.weights ? g.weights[a] : 1.f;
    float dot = 0.f;
    if (static_cast<uint32_t>(pos) < static_cast<uint32_t>(g.rows)) {
        const T *y = static_cast<const T *>(g.y) + pos * g.ldy;
        T *dy = static_cast<T *>(g.dy) + pos * g.lddy;
        typedef Segment<T, LANES, SHORT> Seg;
        for (int h0 = 0; h0 < g.H; h0 += kAhead * kSeg) {
            Seg d[kAhead], f[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * kSeg;
                if (h >= g.H) continue;
                d[u].template load<false>(dout, h, lane, g.H);
                if (g.dweights) f[u].template load<ONCE>(y, h, lane, g.H);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * kSeg;
                if (h >= g.H) continue;
                float dv[kEach];
                d[u].get(dv);
                if (g.dweights) {
                    float fv[kEach];
                    f[u].get(fv);
                    float mine[kEach];
#pragma unroll
                    for (int i = 0; i < kEach; ++i) mine[i] = dv[i];
                    Seg::own(h, lane, g.H, fv);
                    Seg::own(h, lane, g.H, mine);
#pragma unroll
                    for (int i = 0; i < kEach; ++i) dot = __builtin_fmaf(mine[i], fv[i], dot);
                }
                if (g.dy) {
#pragma unroll
                    for (int i = 0; i < kEach; ++i) dv[i] *= w;
                    Seg::store(dy, h, lane, g.H, dv);
                }
            }
        }
    }
    if (g.dweights) {
        dot = lanes_sum<LANES>(dot);
        if (lane == 0) g.dweights[a] = dot;
    }
}

// The lanes a row of H takes, and whether it is less than a run.
template <class F>
void with_row_lanes(const CombineArgs &g, F f) {
    typedef std::false_type No;
    if (g.H < (g.bf16 ? 8 : 4)) f(std::integral_constant<int, 16>{}, std::true_type{});
    else if (g.H <= 16 * kEach) f(std::integral_constant<int, 16>{}, No{});
    else if (g.H <= 32 * kEach) f(std::integral_constant<int, 32>{}, No{});
    else f(std::integral_constant<int, 64>{}, No{});
}

// A launch has fewer than 2^32 threads, of at most 64 for a row's segment.
constexpr int64_t kLaunchItems = int64_t(1) << 25;

// The arguments of the tokens from t on, n of them.
CombineArgs from_token(const CombineArgs &g, int64_t t, int64_t n) {
    CombineArgs p = g;
    const size_t es = g.bf16 ? 2 : 4;
    p.T = static_cast<int>(n);
    p.inv = g.inv + t * g.k;
    p.weights = g.weights ? g.weights + t * g.k : nullptr;
    p.add = g.add ? static_cast<const char *>(g.add) + t * g.ldadd * es : nullptr;
    p.out = g.out ? static_cast<char *>(g.out) + t * g.ldo * es : nullptr;
    p.dout = g.dout ? static_cast<const char *>(g.dout) + t * g.lddout * es : nullptr;
    p.dweights = g.dweights ? g.dweights + t * g.k : nullptr;
    return p;
}

}  // namespace

hipError_t launch_combine(const ue_ctx &, const CombineArgs &g, hipStream_t s) {
    hipError_t he = hipSuccess;
    with_row_lanes(g, [&](auto l, auto few) {
        constexpr bool kShort = decltype(few)::value;
        constexpr int kLanes = decltype(l)::value;
        const int segs = (g.H + kLanes * kEach - 1) / (kLanes * kEach);
        const int64_t tokens = kLaunchItems / segs;
        for (int64_t t = 0; t < g.T && he == hipSuccess; t += tokens) {
            const CombineArgs p = from_token(g, t, g.T - t < tokens ? g.T - t : tokens);
            const uint32_t items = static_cast<uint32_t>(p.T) * segs;
            const dim3 gr((items + kBlock / kLanes - 1) / (kBlock / kLanes));
            const int64_t bytes = static_cast<int64_t>(g.T) * g.k * g.H * (g.bf16 ? 2 : 4);
            with_rows(g.bf16, bytes, [&](auto type, auto once) {
                hipLaunchKernelGGL(
                    (k_combine<decltype(type), kLanes, kShort, decltype(once)::value>), gr,
                    dim3(kBlock), 0, s, p, fast_div(segs), items);
            });
            he = hipGetLastError();
        }
    });
    return he;
}

bool combine_notes(int T, int k, int rows) {
    return static_cast<int64_t>(T) * k > kLookAt || rows > kClearBlocks * kClearRows;
}

hipError_t launch_combine_backward(ue_ctx &c, const CombineArgs &a, bool every_row,
                                   hipStream_t s) {
    hipError_t he = hipSuccess;
    CombineArgs g = a;
    g.all = static_cast<uint32_t>(g.T) * g.k;
    g.clear = 0;
    if (every_row && g.rows > 0) {
        for (g.clear = 1; g.clear < kClearBlocks && g.clear * kBackBlock < static_cast<uint32_t>(g.rows);)
            g.clear *= 2;
        if (g.named_by && g.all > 0) {
            hipLaunchKernelGGL(k_combine_note, dim3((g.all + kBlock - 1) / kBlock), dim3(kBlock), 0, s,
                               g);
            he = hipGetLastError();
            tmark(&c, s);
        }
    }
    with_row_lanes(g, [&](auto l, auto few) {
        constexpr bool kShort = decltype(few)::value;
        constexpr int kLanes = decltype(l)::value, kItems = kBackBlock / kLanes;
        const int64_t tokens = kLaunchItems / g.k;
        // (no token is a launch all the same if rows are to be cleared)
        for (int64_t t = 0; (t < g.T || (t == 0 && g.clear)) && he == hipSuccess; t += tokens) {
            CombineArgs p = from_token(g, t, g.T - t < tokens ? g.T - t : tokens);
            if (t > 0) p.clear = 0;
            const uint32_t items = static_cast<uint32_t>(p.T) * g.k;
            const dim3 gr((items + kItems - 1) / kItems + p.clear);
            const int64_t bytes = static_cast<int64_t>(g.T) * g.k * g.H * (g.bf16 ? 2 : 4);
            with_rows(g.bf16, bytes, [&](auto type, auto once) {
                hipLaunchKernelGGL(
                    (k_combine_backward<decltype(type), kLanes, kShort, decltype(once)::value>),
                    gr, dim3(kBackBlock), 0, s, p, fast_div(g.k), items);
            });
            he = hipGetLastError();
        }
    });
    return he;
}

}  // namespace ue
