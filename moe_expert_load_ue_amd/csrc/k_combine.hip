// Sum of the experts' rows back to their tokens (ue_combine) and its gradients
// (ue_combine_backward).
//
//   out_t = add_t + sum_j w_tj y[inv_tj];  dy[inv_tj] = w_tj dout_t;
//   dw_tj = <dout_t, y[inv_tj]>
//
// Forward: a wave takes one segment of one token's row and loads that segment
// of up to kJoin of its rows at once before it adds them, in order. Backward: a
// wave per assignment, those of a token in one workgroup (of up to kJoin waves),
// so that dout comes from the cache for all but the first; a dot is added by
// lanes, then over them, in a fixed order. Places and weights are the same for a
// whole wave and so are read by scalar loads.
//
// Bound: HBM. 16384 tokens x top-8 x 7168, bf16: forward 372 us (2.1 GB, 5.7
// TB/s), backward 734 us (4.0 GB, 5.5 TB/s). A workgroup per token whose waves
// shared out the segments took 880 backward; four segments ahead in place of two
// 965, one 724 (but 10.9 us in place of 9.8 for 1021 tokens x top-6 x 1002,
// fp32); dout past the caches too 794.
#include "ue_train.h"

namespace ue {
namespace {

constexpr int kJoin = 8;      // rows of a token in flight
constexpr int kEach = 8;      // elements of a lane

// LANES: of a row's segment. Rows shorter than a wave's 512 elements share it.
template <typename T, int LANES>
__global__ __launch_bounds__(kBlock) void k_combine(CombineArgs g, FastDiv segs, uint32_t items) {
    constexpr int kItems = kBlock / LANES;
    uint32_t item = blockIdx.x * kItems + threadIdx.x / LANES;
    if (LANES == 64) item = __builtin_amdgcn_readfirstlane(item);
    if (item >= items) return;
    const int t = div_by(item, segs);
    const int h = (item - t * segs.d) * LANES * kEach + threadIdx.x % LANES * kEach;
    const int n = g.H - h;
    const int64_t o = static_cast<int64_t>(t) * g.k;
    const T *y = static_cast<const T *>(g.y) + h;
    float sum[kEach] = {};
    if (g.add) load8(static_cast<const T *>(g.add) + t * g.ldadd + h, n, sum);
    for (int j0 = 0; j0 < g.k; j0 += kJoin) {
        float f[kJoin][kEach], w[kJoin];
        bool has[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int at = j0 + j < g.k ? j0 + j : 0, pos = g.inv[o + at];
            has[j] = j0 + j < g.k && static_cast<uint32_t>(pos) < static_cast<uint32_t>(g.rows);
            w[j] = g.weights ? g.weights[o + at] : 1.f;
            if (has[j]) load8(y + pos * g.ldy, n, f[j]);
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            if (!has[j]) continue;
#pragma unroll
            for (int i = 0; i < kEach; ++i) sum[i] = __builtin_fmaf(w[j], f[j][i], sum[i]);
        }
    }
    store8(static_cast<T *>(g.out) + t * g.ldo + h, n, sum);
}

constexpr int kAhead = 2;     // segments in flight
constexpr int kBackBlock = 512;

template <typename T, int LANES>
__global__ __launch_bounds__(kBackBlock) void k_combine_backward(CombineArgs g, FastDiv topk,
                                                                 uint32_t assignments) {
    constexpr int kItems = kBackBlock / LANES, kSeg = LANES * kEach;
    uint32_t a = blockIdx.x * kItems + threadIdx.x / LANES;
    if (LANES == 64) a = __builtin_amdgcn_readfirstlane(a);
    if (a >= assignments) return;                   // (whole rows of lanes)
    const int lane = threadIdx.x % LANES, t = div_by(a, topk);
    const T *dout = static_cast<const T *>(g.dout) + t * g.lddout + lane * kEach;
    const int pos = g.inv[a];
    const float w = g.weights ? g.weights[a] : 1.f;
    float dot = 0.f;
    if (static_cast<uint32_t>(pos) < static_cast<uint32_t>(g.rows)) {
        const T *y = static_cast<const T *>(g.y) + pos * g.ldy + lane * kEach;
        T *dy = static_cast<T *>(g.dy) + pos * g.lddy + lane * kEach;
        const int n = g.H - lane * kEach;
        for (int h0 = 0; h0 < g.H; h0 += kAhead * kSeg) {
            float d[kAhead][kEach], f[kAhead][kEach];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * kSeg;
                if (h >= g.H) continue;
                load_run<kEach, false>(dout + h, n - h, d[u]);
                if (g.dweights) load8(y + h, n - h, f[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * kSeg;
                if (h >= g.H) continue;
                if (g.dweights) {
#pragma unroll
                    for (int i = 0; i < kEach; ++i) dot = __builtin_fmaf(d[u][i], f[u][i], dot);
                }
                if (g.dy) {
#pragma unroll
                    for (int i = 0; i < kEach; ++i) d[u][i] *= w;
                    store8(dy + h, n - h, d[u]);
                }
            }
        }
    }
    if (g.dweights) {
        dot = lanes_sum<LANES>(dot);
        if (lane == 0) g.dweights[a] = dot;
    }
}

// The lanes a row of H takes: f(lanes).
template <class F>
void with_row_lanes(int H, F f) {
    if (H <= 16 * kEach) f(std::integral_constant<int, 16>{});
    else if (H <= 32 * kEach) f(std::integral_constant<int, 32>{});
    else f(std::integral_constant<int, 64>{});
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
    with_row_lanes(g.H, [&](auto l) {
        constexpr int kLanes = decltype(l)::value;
        const int segs = (g.H + kLanes * kEach - 1) / (kLanes * kEach);
        const int64_t tokens = kLaunchItems / segs;
        for (int64_t t = 0; t < g.T && he == hipSuccess; t += tokens) {
            const CombineArgs p = from_token(g, t, g.T - t < tokens ? g.T - t : tokens);
            const uint32_t items = static_cast<uint32_t>(p.T) * segs;
            const dim3 gr((items + kBlock / kLanes - 1) / (kBlock / kLanes));
            if (g.bf16)
                hipLaunchKernelGGL((k_combine<uint16_t, kLanes>), gr, dim3(kBlock), 0, s, p,
                                   fast_div(segs), items);
            else
                hipLaunchKernelGGL((k_combine<float, kLanes>), gr, dim3(kBlock), 0, s, p,
                                   fast_div(segs), items);
            he = hipGetLastError();
        }
    });
    return he;
}

hipError_t launch_combine_backward(const ue_ctx &, const CombineArgs &g, hipStream_t s) {
    hipError_t he = hipSuccess;
    with_row_lanes(g.H, [&](auto l) {
        constexpr int kLanes = decltype(l)::value, kItems = kBackBlock / kLanes;
        const int64_t tokens = kLaunchItems / g.k;
        for (int64_t t = 0; t < g.T && he == hipSuccess; t += tokens) {
            const CombineArgs p = from_token(g, t, g.T - t < tokens ? g.T - t : tokens);
            const uint32_t items = static_cast<uint32_t>(p.T) * g.k;
            const dim3 gr((items + kItems - 1) / kItems);
            if (g.bf16)
                hipLaunchKernelGGL((k_combine_backward<uint16_t, kLanes>), gr, dim3(kBackBlock), 0,
                                   s, p, fast_div(g.k), items);
            else
                hipLaunchKernelGGL((k_combine_backward<float, kLanes>), gr, dim3(kBackBlock), 0, s,
                                   p, fast_div(g.k), items);
            he = hipGetLastError();
        }
    });
    return he;
}

}  // namespace ue
