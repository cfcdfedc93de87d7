// Gradients of the matrices of row groups (ue_weight_grad):
//   out[g, n, k] (+)= sum over the rows m of group g of dy[m, n] x[r(m), k]
//
// A workgroup makes a 64 x 64 tile of one group's matrix, one thread 4 x 4 of
// it, sixteen rows at a time through LDS in fp32.
#include "ue_train.h"

namespace ue {
namespace {

constexpr int kTile = 64, kRows = 16;

__global__ __launch_bounds__(kBlock) void k_wgrad(WgradArgs g, int tiles_n, int tiles_k) {
    __shared__ float a[kRows][kTile], b[kRows][kTile];
    const int tid = threadIdx.x;
    int id = blockIdx.x;
    const int tk = id % tiles_k;
    id /= tiles_k;
    const int tn = id % tiles_n, grp = id / tiles_n;
    int lo = 0, hi = g.M;
    if (g.offsets) {
        lo = g.offsets[grp];
        hi = g.offsets[grp + 1];
        lo = lo < 0 ? 0 : lo > g.M ? g.M : lo;
        hi = hi < lo ? lo : hi > g.M ? g.M : hi;
    }
    const int n0 = tn * kTile, k0 = tk * kTile;
    const int r = tid >> 4, c4 = (tid & 15) * 4;      // what this thread loads
    const int tr = (tid >> 4) * 4, tc = (tid & 15) * 4;
    float acc[4][4] = {};
    for (int m0 = lo; m0 < hi; m0 += kRows) {
        const int m = m0 + r;
        int row = -1;
        if (m < hi) {
            row = m;
            if (g.index) {
                row = g.index[m];
                row = row < 0 ? -1 : row / g.index_div;
            }
            if (row >= g.x_rows) row = -1;
        }
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + c4 + i, k = k0 + c4 + i;
            a[r][c4 + i] = m < hi && n < g.N ? bf16_to_f32(g.dy[m * g.lddy + n]) : 0.f;
            float v = 0.f;
            if (row >= 0 && k < g.K) {
                if (g.x_scale)
                    v = static_cast<float>(static_cast<const int8_t *>(g.x)[row * g.ldx + k]) *
                        scale_step(g.x_scale[row * g.lds + k / UE_PACK_BLOCK]);
                else
                    v = bf16_to_f32(static_cast<const uint16_t *>(g.x)[row * g.ldx + k]);
            }
            b[r][c4 + i] = v;
        }
        __syncthreads();
        for (int q = 0; q < kRows; ++q)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_fmaf(a[q][tr + i], b[q][tc + j], acc[i][j]);
        __syncthreads();
    }
    float *out = g.out + grp * g.out_stride;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tr + i, k = k0 + tc + j;
            if (n >= g.N || k >= g.K) continue;
            float *p = out + n * g.ldo + k;
            *p = g.accumulate ? *p + acc[i][j] : acc[i][j];
        }
}

constexpr int64_t kLaunchThreads = 0xFFFFFFFFll;

}  // namespace

int wgrad_parts(int, int, int, int, bool, int) { return 1; }

hipError_t launch_wgrad(ue_ctx &, const WgradArgs &g, hipStream_t s, bool &too_large) {
    const int64_t tn = (g.N + kTile - 1) / kTile, tk = (g.K + kTile - 1) / kTile;
    too_large = tn * tk > kLaunchThreads || tn * tk * g.G * kBlock > kLaunchThreads;
    if (too_large || tn * tk * g.G == 0) return hipSuccess;
    hipLaunchKernelGGL(k_wgrad, dim3(static_cast<uint32_t>(tn * tk * g.G)), dim3(kBlock), 0, s,
                       g, static_cast<int>(tn), static_cast<int>(tk));
    return hipGetLastError();
}

}  // namespace ue
