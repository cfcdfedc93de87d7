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
constexpr int kSeg = 512;     // elements of a wave's segment: 8 a lane

// The lane's elements of a segment at p: 8 in a row (VEC), or every 64th. `n`:
// elements from p to the end of the row.
template <typename T, bool VEC, bool ONCE = true>
__device__ __forceinline__ void load_seg(const T *p, int n, float (&f)[8]) {
    const int lane = lane_id();
    if (VEC) {
        load8<T, ONCE>(p + lane * 8, true, n - lane * 8, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = lane + 64 * i < n ? widen<T>(p[lane + 64 * i]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_seg(T *p, int n, const float (&f)[8]) {
    const int lane = lane_id();
    if (VEC) {
        store8<T>(p + lane * 8, true, n - lane * 8, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 64 * i < n) p[lane + 64 * i] = narrow<T>(f[i]);
    }
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kBlock) void k_combine(CombineArgs g, FastDiv segs, uint32_t items) {
    const uint32_t item = __builtin_amdgcn_readfirstlane(
        blockIdx.x * kWaves + (threadIdx.x >> 6));
    if (item >= items) return;
    const int t = div_by(item, segs), h = (item - t * segs.d) * kSeg;
    const int n = g.H - h;
    const int64_t o = static_cast<int64_t>(t) * g.k;
    const T *y = static_cast<const T *>(g.y) + h;
    float sum[8] = {};
    if (g.add) load_seg<T, VEC>(static_cast<const T *>(g.add) + t * g.ldadd + h, n, sum);
    for (int j0 = 0; j0 < g.k; j0 += kJoin) {
        float f[kJoin][8], w[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int pos = j0 + j < g.k ? g.inv[o + j0 + j] : -1;
            w[j] = 0.f;
            if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(g.rows)) continue;
            w[j] = g.weights ? g.weights[o + j0 + j] : 1.f;
            load_seg<T, VEC>(y + pos * g.ldy, n, f[j]);
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int pos = j0 + j < g.k ? g.inv[o + j0 + j] : -1;
            if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(g.rows)) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], f[j][i], sum[i]);
        }
    }
    store_seg<T, VEC>(static_cast<T *>(g.out) + t * g.ldo + h, n, sum);
}

constexpr int kAhead = 2;     // segments in flight

template <typename T, bool VEC>
__global__ __launch_bounds__(kJoin * 64) void k_combine_backward(CombineArgs g, int t_first) {
    const int lane = lane_id(), waves = blockDim.x >> 6;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = t_first + blockIdx.x;
    const int64_t o = static_cast<int64_t>(t) * g.k;
    const T *dout = static_cast<const T *>(g.dout) + t * g.lddout;
    for (int j = wv; j < g.k; j += waves) {
        const int pos = g.inv[o + j];
        const float w = g.weights ? g.weights[o + j] : 1.f;
        float dot = 0.f;
        if (static_cast<uint32_t>(pos) < static_cast<uint32_t>(g.rows)) {
            const T *y = static_cast<const T *>(g.y) + pos * g.ldy;
            T *dy = static_cast<T *>(g.dy) + pos * g.lddy;
            for (int h0 = 0; h0 < g.H; h0 += kAhead * kSeg) {
                float d[kAhead][8], f[kAhead][8];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int h = h0 + u * kSeg;
                    if (h >= g.H) continue;
                    load_seg<T, VEC, false>(dout + h, g.H - h, d[u]);
                    if (g.dweights) load_seg<T, VEC>(y + h, g.H - h, f[u]);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int h = h0 + u * kSeg;
                    if (h >= g.H) continue;
                    if (g.dweights) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(d[u][i], f[u][i], dot);
                    }
                    if (g.dy) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[u][i] *= w;
                        store_seg<T, VEC>(dy + h, g.H - h, d[u]);
                    }
                }
            }
        }
        if (g.dweights) {
            dot = lanes_sum<64>(dot);
            if (lane == 0) g.dweights[o + j] = dot;
        }
    }
}

}  // namespace

hipError_t launch_combine(const ue_ctx &, const CombineArgs &g, hipStream_t s) {
    const int segs = (g.H + kSeg - 1) / kSeg;
    // (a launch has fewer than 2^32 threads)
    const int64_t tokens = (int64_t(1) << 25) / segs;
    const size_t es = g.bf16 ? 2 : 4;
    for (int64_t t = 0; t < g.T; t += tokens) {
        CombineArgs p = g;
        p.T = static_cast<int>(g.T - t < tokens ? g.T - t : tokens);
        p.inv = g.inv + t * g.k;
        p.weights = g.weights ? g.weights + t * g.k : nullptr;
        p.add = g.add ? static_cast<const char *>(g.add) + t * g.ldadd * es : nullptr;
        p.out = static_cast<char *>(g.out) + t * g.ldo * es;
        const uint32_t items = static_cast<uint32_t>(p.T) * segs;
        const dim3 gr((items + kWaves - 1) / kWaves), bl(kBlock);
        const FastDiv d = fast_div(segs);
        if (g.bf16) {
            if (g.vec) hipLaunchKernelGGL((k_combine<uint16_t, true>), gr, bl, 0, s, p, d, items);
            else hipLaunchKernelGGL((k_combine<uint16_t, false>), gr, bl, 0, s, p, d, items);
        } else {
            if (g.vec) hipLaunchKernelGGL((k_combine<float, true>), gr, bl, 0, s, p, d, items);
            else hipLaunchKernelGGL((k_combine<float, false>), gr, bl, 0, s, p, d, items);
        }
        const hipError_t he = hipGetLastError();
        if (he != hipSuccess) return he;
    }
    return hipSuccess;
}

hipError_t launch_combine_backward(const ue_ctx &, const CombineArgs &g, hipStream_t s) {
    constexpr int kTokens = 1 << 22;         // of a launch: fewer than 2^32 threads
    for (int t = 0; t < g.T; t += kTokens) {
        const dim3 gr(g.T - t < kTokens ? g.T - t : kTokens), bl(64 * (g.k < kJoin ? g.k : kJoin));
        if (g.bf16) {
            if (g.vec) hipLaunchKernelGGL((k_combine_backward<uint16_t, true>), gr, bl, 0, s, g, t);
            else hipLaunchKernelGGL((k_combine_backward<uint16_t, false>), gr, bl, 0, s, g, t);
        } else {
            if (g.vec) hipLaunchKernelGGL((k_combine_backward<float, true>), gr, bl, 0, s, g, t);
            else hipLaunchKernelGGL((k_combine_backward<float, false>), gr, bl, 0, s, g, t);
        }
        const hipError_t he = hipGetLastError();
        if (he != hipSuccess) return he;
        if (g.T - t <= kTokens) break;       // (t + kTokens may pass 31 bits)
    }
    return hipSuccess;
}

}  // namespace ue
