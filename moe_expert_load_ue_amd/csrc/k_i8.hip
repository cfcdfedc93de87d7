// Products in 8-bit integers with one scale per row of activations and one
// per channel of the matrix (ue_matmul_i8):
//   out[m, n] = a_scale[r] w_scale[g, n] sum_k a[r, k] w[g, n, k]
// with g the group of row m and r its row of activations. The integer sums
// are exact (32 bits), so the result is rounded only by the two scales and
// the output type. Gated: the matrix holds N gate channels, then N up
// channels, and out = silu(gate) up.
//
// A workgroup makes a tile of rows times channels. Both operands come
// through LDS by direct loads, 128 bytes of every row at a time, two stages:
// the next stage's loads are issued before this stage's products. A stage
// holds rows of 8 16-byte pieces; piece c of row r sits at c ^ (r & 7), so
// that the 16 rows an operand read touches fall on different banks (the
// direct load writes LDS in lane order, so the lanes' addresses carry the
// swizzle).
//
// The matrix is the instruction's first operand and the activations its
// second: a lane then holds channels of one row. The matrix's rows are laid
// in LDS so that row 4 q + i of fragment f is channel 4 F q + 4 f + i of the
// wave's F fragments: lane group q then holds 4 F consecutive channels.
#include "ue_gate.h"

namespace ue {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;               // bytes of K per stage

// Rows [lo, hi) of group `tile` of the launch's row tiles: group g has
// ceil(rows / BM) tiles, groups in order. Offsets are clamped to [0, M], so
// that no table can send a tile outside. False: no such tile.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const I8Args &g, int tile, int BM,
                                          int *sh, int &group, int &lo,
                                          int &hi) {
    if (!g.offsets) {
        group = 0;
        lo = tile * BM;
        hi = g.M;
        return lo < g.M;
    }
    const int tid = threadIdx.x;
    const int per = (g.G + THREADS - 1) / THREADS;
    const int first = tid * per;
    auto bounds = [&](int i, int &a, int &b) {
        a = g.offsets[i];
        b = g.offsets[i + 1];
        a = a < 0 ? 0 : a > g.M ? g.M : a;
        b = b < a ? a : b > g.M ? g.M : b;
    };
    int n = 0;
    for (int i = first; i < first + per && i < g.G; ++i) {
        int a, b;
        bounds(i, a, b);
        n += (b - a + BM - 1) / BM;
    }
    // tiles before this thread's groups
    const int incl = wave_inclusive_sum(n);
    if (tid == 0) sh[16] = -1;
    if (lane_id() == 63) sh[tid >> 6] = incl;
    __syncthreads();
    int before = incl - n;
    for (int w = 0; w < (tid >> 6); ++w) before += sh[w];
    if (tile >= before && tile < before + n) {
        int t = tile - before;
        for (int i = first;; ++i) {
            int a, b;
            bounds(i, a, b);
            const int nt = (b - a + BM - 1) / BM;
            if (t < nt) {
                sh[16] = i;
                sh[17] = a + t * BM;
                sh[18] = b;
                break;
            }
            t -= nt;
        }
    }
    __syncthreads();
    group = sh[16];
    lo = sh[17];
    hi = sh[18];
    return group >= 0;
}

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) {
    *p = f32_to_bf16(v);
}

// FM, FN: 16-row fragments of activations and of the matrix per wave;
// WM, WN: waves along each.
template <int FM, int FN, int WM, int WN, bool GATED, typename OUT>
__global__ __launch_bounds__(WM *WN * 64) void k_matmul_i8(I8Args g) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int BM = WM * FM * 16, BN = WN * FN * 16;   // rows in LDS
    constexpr int kOut = GATED ? BN / 2 : BN;             // channels out
    constexpr int kChunks = (BM + BN) / 8 / (WM * WN);    // of 8 rows, a wave
    static_assert((BM + BN) / 8 % (WM * WN) == 0, "whole chunks per wave");
    extern __shared__ __align__(16) char lds[];
    __shared__ int sh[20];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int ncol = (g.N + kOut - 1) / kOut;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    const int n0 = (id % ncol) * kOut;
    int group, m0, m_end;
    if (!find_tile<kThreads>(g, id / ncol, BM, sh, group, m0, m_end)) return;
    const int mat = g.expert_of ? g.expert_of[group] : group;
    if (static_cast<uint32_t>(mat) >= static_cast<uint32_t>(g.n_mats)) return;

    // the row of activations of output row m (-1: none)
    auto act_row = [&](int m) {
        if (!g.index) return m;
        const int i = g.index[m];
        if (i < 0) return -1;
        const int r = i / g.index_div;
        return r < g.a_rows ? r : -1;
    };
    // global address of this lane's piece of each chunk it loads
    const int8_t *src[kChunks];
    const int piece = (lane & 7) ^ (lane >> 3);     // row & 7 = lane >> 3
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int r = (wv * kChunks + c) * 8 + (lane >> 3);
        if (r < BM) {
            int m = m0 + r;
            m = m < m_end ? m : m_end - 1;
            const int a = act_row(m);
            src[c] = g.a + static_cast<int64_t>(a < 0 ? 0 : a) * g.lda;
        } else {
            // row b of the tile's matrix: row l of fragment j of wave w's
            // block takes channel 4 F (l >> 2) + 4 j + (l & 3) of the block
            // (gated: fragments alternate gate, up of the same channels)
            const int b = r - BM, w = b / (FN * 16);
            const int j = (b >> 4) % FN, l = b & 15;
            int n;
            if (GATED) {
                constexpr int P = FN / 2;
                n = n0 + w * P * 16 + 4 * P * (l >> 2) + 4 * (j >> 1) + (l & 3);
                n = n < g.N ? n : g.N - 1;
                n += (j & 1) ? g.N : 0;
            } else {
                n = n0 + w * FN * 16 + 4 * FN * (l >> 2) + 4 * j + (l & 3);
                n = n < g.N ? n : g.N - 1;
            }
            src[c] = g.w + mat * g.w_stride + static_cast<int64_t>(n) * g.ldw;
        }
    }
    const int kbytes = (g.K + 15) & ~15;
    auto load_stage = [&](int buf, int k0) {
        // pieces past the row's end are read from its start: the last
        // stage's products mask them
        int k = k0 + piece * 16;
        k = k < kbytes ? k : 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            char *dst = lds + buf * (BM + BN) * kStep +
                        (wv * kChunks + c) * 8 * kStep;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(src[c] + k),
                (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
        }
    };

    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int wm = wv / WN, wn = wv % WN;
    const int q = lane >> 4, l16 = lane & 15;
    // rows of this lane's operand reads
    const int arow = wm * FM * 16 + l16;
    const int brow = wn * FN * 16 + l16;
    auto products = [&](int buf, int k0, bool mask) {
        const char *A = lds + buf * (BM + BN) * kStep;
        const char *B = A + BM * kStep;
#pragma unroll
        for (int h = 0; h < kStep / 64; ++h) {
            const int c = h * 4 + q;
            i32x4 a[FM], b[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                a[i] = *reinterpret_cast<const i32x4 *>(
                    A + (arow + i * 16) * kStep + ((c ^ (arow & 7)) << 4));
            }
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = *reinterpret_cast<const i32x4 *>(
                    B + (brow + j * 16) * kStep + ((c ^ (brow & 7)) << 4));
            if (mask) {
                // zero activations past K (integers: what they meet in the
                // matrix then does not matter)
                const int left = g.K - (k0 + c * 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int nb = left - 4 * w;
                    const uint32_t keep =
                        nb >= 4 ? 0xFFFFFFFFu
                                : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        a[i][w] &= static_cast<int>(keep);
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        b[j], a[i], acc[i][j], 0, 0, 0);
        }
    };

    const int steps = (g.K + kStep - 1) / kStep;
    load_stage(0, 0);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) load_stage((s + 1) & 1, (s + 1) * kStep);
        products(s & 1, s * kStep, (s + 1) * kStep > g.K);
        __syncthreads();
    }

    const float *ws = g.w_scale + mat * g.ws_stride;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + arow + i * 16;
        if (m >= m_end) continue;
        const int ar = act_row(m);
        const float as = ar < 0 ? 0.f : g.a_scale[ar];
        OUT *out = static_cast<OUT *>(g.out) + static_cast<int64_t>(m) * g.ldo;
        if (GATED) {
            constexpr int P = FN / 2;
            const int base = n0 + wn * FN * 8 + 4 * P * q;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = base + 4 * p + e;
                    if (n >= g.N) continue;
                    const float gt = static_cast<float>(acc[i][2 * p][e]) * as * ws[n];
                    const float up = static_cast<float>(acc[i][2 * p + 1][e]) * as * ws[g.N + n];
                    store_out(out + n, gt / (1.0f + expf(-gt)) * up);
                }
        } else {
            const int base = n0 + wn * FN * 16 + 4 * FN * q;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = base + 4 * j + e;
                    if (n >= g.N) continue;
                    store_out(out + n, static_cast<float>(acc[i][j][e]) * as * ws[n]);
                }
        }
    }
}

template <int FM, int FN, int WM, int WN>
hipError_t tiled(const I8Args &g, hipStream_t s) {
    constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
    const int kout = g.gated ? BN / 2 : BN;
    const int64_t ncol = (g.N + kout - 1) / kout;
    int64_t mt = (static_cast<int64_t>(g.M) + BM - 1) / BM;
    if (g.offsets) mt += g.G;       // each group's last tile may be partial
    const int64_t grid = ncol * mt;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const size_t lds = 2 * (BM + BN) * kStep;
    const dim3 gr(static_cast<uint32_t>(grid)), bl(WM * WN * 64);
#define UE_I8_LAUNCH(GATED, OUT)                                               \
    hipLaunchKernelGGL((k_matmul_i8<FM, FN, WM, WN, GATED, OUT>), gr, bl, lds, \
                       s, g)
    if (g.gated) {
        if (g.out_f32) UE_I8_LAUNCH(true, float);
        else UE_I8_LAUNCH(true, uint16_t);
    } else {
        if (g.out_f32) UE_I8_LAUNCH(false, float);
        else UE_I8_LAUNCH(false, uint16_t);
    }
#undef UE_I8_LAUNCH
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_i8(const ue_ctx &c, const I8Args &g, hipStream_t s) {
    if (g.M == 0 || g.N == 0) return hipSuccess;
    return tiled<4, 4, 2, 2>(g, s);
}

}  // namespace ue
