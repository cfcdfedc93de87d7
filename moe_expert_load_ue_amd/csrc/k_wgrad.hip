// Gradients of the matrices of row groups (ue_weight_grad):
//   out[g, n, k] (+)= sum over the rows m of group g of dy[m, n] x[r(m), k]
//
// A workgroup makes a tile of one group's matrix. Both operands lie row by row,
// with the sum going down the rows, while a matrix instruction wants each lane's
// eight terms side by side. So rows go to LDS as they are, in bf16, and come
// out transposed: a transposing LDS read gives each of 16 lanes one column of
// four rows. A stage is kRows rows; dy comes by direct loads two stages ahead,
// . Which four rows a lane's terms
// come from does not matter as long as both operands take the same.
//
// Rows in LDS are units of 16 columns (32 bytes); unit u of row r sits at
// u ^ (r mod units), so that the four rows a transposing read touches fall on
// different banks.
#include "ue_train.h"

#include <type_traits>

namespace ue {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 16;                // columns of a unit: 32 bytes in LDS

// Sixteen columns of a row as bf16.
struct Unit { u32x4 lo, hi; };

// Four int8 times a power of two as bf16: the product's low half is zero.
__device__ __forceinline__ void widen_packed(uint32_t v, float step, uint32_t &a, uint32_t &b) {
    const float f0 = static_cast<float>(static_cast<int8_t>(v)) * step;
    const float f1 = static_cast<float>(static_cast<int8_t>(v >> 8)) * step;
    const float f2 = static_cast<float>(static_cast<int8_t>(v >> 16)) * step;
    const float f3 = static_cast<float>(static_cast<int8_t>(v >> 24)) * step;
    a = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
    b = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
}
__device__ __forceinline__ Unit widen_unit(u32x4 q, float step) {
    Unit u;
    uint32_t a, b;
    widen_packed(q[0], step, a, b);
    u.lo[0] = a;
    u.lo[1] = b;
    widen_packed(q[1], step, a, b);
    u.lo[2] = a;
    u.lo[3] = b;
    widen_packed(q[2], step, a, b);
    u.hi[0] = a;
    u.hi[1] = b;
    widen_packed(q[3], step, a, b);
    u.hi[2] = a;
    u.hi[3] = b;
    return u;
}

// The first `n` of 16 bf16 at p (zeros past them); whole pieces by 16-byte loads
// at any 2-byte alignment.
__device__ __forceinline__ Unit load_unit(const uint16_t *p, int n) {
    struct __attribute__((packed, aligned(2))) Piece { u32x4 v; };
    Unit u{};
    if (n >= 8) u.lo = reinterpret_cast<const Piece *>(p)->v;
    if (n >= 16) u.hi = reinterpret_cast<const Piece *>(p + 8)->v;
    if (n > 0 && n < 16 && n != 8) {
        const int from = n > 8 ? 8 : 0;
        u32x4 t{};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (from + i < n)
                t[i / 2] |= static_cast<uint32_t>(p[from + i]) << (16 * (i & 1));
        if (from) u.hi = t;
        else u.lo = t;
    }
    return u;
}

// FN, FK: 32-column fragments of dy and of x per wave; WN, WK: waves along each;
// ROWS: rows of a stage. WHOLE: rows are 16-byte aligned and multiples of 8
// columns (packed x always is), so that pieces are whole or nobody's.
//
// While a stage's products run, the next one's rows are in registers or on
// their way to LDS, and the one after that is on its way to registers.
template <int FN, int FK, int WN, int WK, int ROWS, bool WHOLE, bool PACKED>
__global__ __launch_bounds__(WN *WK * 64, FN * FK > 8 ? 1 : 2) void k_wgrad(
    WgradArgs g, FastDiv div, int tiles_n, int tiles_k) {
    constexpr int kThreads = WN * WK * 64;
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32;
    constexpr int UN = BN / kUnit, UK = BK / kUnit;          // units of a row
    constexpr int kDyBytes = ROWS * BN * 2, kStage = kDyBytes + ROWS * BK * 2;
    constexpr int kUnitsX = ROWS * UK / kThreads;            // units of a thread
    constexpr int kUnitsDy = ROWS * UN / kThreads;
    static_assert(kUnitsX * kThreads == ROWS * UK && kUnitsDy * kThreads == ROWS * UN,
                  "whole units per thread");
    static_assert(ROWS % 16 == 0 && UN % 8 == 0 && UK % 8 == 0);
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);

    // tiles of a group side by side, four along n to every one along k
    constexpr int kBlockN = 4;
    const int per = tiles_n * tiles_k;
    const int id = xcd_order(blockIdx.x, per * g.G);
    const int grp = id / per, in_grp = id - grp * per;
    const int blk = in_grp / (kBlockN * tiles_k), in = in_grp - blk * kBlockN * tiles_k;
    const int bn = tiles_n - blk * kBlockN < kBlockN ? tiles_n - blk * kBlockN : kBlockN;
    const int n0 = (blk * kBlockN + in % bn) * BN, k0 = in / bn * BK;
    int lo = 0, hi = g.M;
    if (g.offsets) {
        lo = g.offsets[grp];
        hi = g.offsets[grp + 1];
        lo = lo < 0 ? 0 : lo > g.M ? g.M : lo;
        hi = hi < lo ? lo : hi > g.M ? g.M : hi;
    }
    const int steps = (hi - lo + ROWS - 1) / ROWS;

    // ---- loads: rows past the group's last are read again as the last one and
    // put down as zeros; pieces past the last column are read from the first
    // (results of columns that nobody stores) ----
    Unit dyr[kUnitsDy];
    auto fetch_dy = [&](int st) {
#pragma unroll
        for (int c = 0; c < kUnitsDy; ++c) {
            const int i = c * kThreads + tid, n = n0 + i % UN * kUnit;
            int m = lo + st * ROWS + i / UN;
            m = m < hi ? m : hi - 1;
            const uint16_t *row = g.dy + m * g.lddy;
            if constexpr (WHOLE) {
                dyr[c].lo = *reinterpret_cast<const u32x4 *>(row + (n < g.N ? n : 0));
                dyr[c].hi = *reinterpret_cast<const u32x4 *>(row + (n + 8 < g.N ? n + 8 : 0));
            } else {
                dyr[c] = load_unit(row + n, g.N - n);
            }
        }
    };
    auto put = [&](char *base, int units, int i, const Unit &u) {
        const int r = i / units, at = (i % units) ^ (r & (units - 1));
        u32x4 *to = reinterpret_cast<u32x4 *>(base + (r * units + at) * 32);
        to[0] = u.lo;
        to[1] = u.hi;
    };
    auto put_dy = [&](int st) {
        const bool last = lo + (st + 1) * ROWS > hi;
#pragma unroll
        for (int c = 0; c < kUnitsDy; ++c) {
            const int i = c * kThreads + tid;
            Unit u = dyr[c];
            if (last && lo + st * ROWS + i / UN >= hi) u = Unit{};
            put(lds + (st & 1) * kStage, UN, i, u);
        }
    };
    // x: the index of a row a stage before its units
    int index[kUnitsX];
    auto fetch_index = [&](int st) {
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) {
            int m = lo + st * ROWS + (c * kThreads + tid) / UK;
            m = m < hi ? m : hi - 1;
            index[c] = g.index ? g.index[m] : m;
        }
    };
    struct Raw { u32x4 q; uint32_t s; };
    Raw xq[PACKED ? kUnitsX : 1];
    Unit xu[PACKED ? 1 : kUnitsX];
    bool live[kUnitsX];
    auto fetch_x = [&](int st) {
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) {
            const int i = c * kThreads + tid, k = k0 + i % UK * kUnit;
            int r = index[c] < 0 ? -1 : static_cast<int>(div_by(index[c], div));
            live[c] = r >= 0 && r < g.x_rows && lo + st * ROWS + i / UK < hi;
            r = live[c] ? r : 0;
            if constexpr (PACKED) {
                // (rows are readable up to a multiple of 16)
                const int at = k < g.K ? k : 0;
                xq[c].q = *reinterpret_cast<const u32x4 *>(
                    static_cast<const int8_t *>(g.x) + r * g.ldx + at);
                xq[c].s = g.x_scale[r * g.lds + at / UE_PACK_BLOCK];
            } else {
                const uint16_t *row = static_cast<const uint16_t *>(g.x) + r * g.ldx;
                if constexpr (WHOLE) {
                    xu[c].lo = *reinterpret_cast<const u32x4 *>(row + (k < g.K ? k : 0));
                    xu[c].hi = *reinterpret_cast<const u32x4 *>(row + (k + 8 < g.K ? k + 8 : 0));
                } else {
                    xu[c] = load_unit(row + k, g.K - k);
                }
            }
        }
    };
    auto put_x = [&](int st) {
        char *const base = lds + (st & 1) * kStage + kDyBytes;
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) {
            if constexpr (PACKED)
                put(base, UK, c * kThreads + tid,
                    widen_unit(xq[c].q, live[c] ? scale_step(xq[c].s) : 0.f));
            else
                put(base, UK, c * kThreads + tid, live[c] ? xu[c] : Unit{});
        }
    };

    // ---- products ----
    f32x16 acc[FN][FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j) acc[i][j] = f32x16{};
    const int wn = wv / WK, wk = wv % WK;
    // where this lane reads: four rows of one unit per 16 lanes; half of a
    // wave's lanes take rows 0-7 of sixteen, half 8-15, in two reads
    const int q = lane >> 4, sub = lane & 15;
    int ra[FN][2], rb[FK][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r = 8 * (q >> 1) + 4 * t + (sub >> 2);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int u = wn * FN * 2 + i * 2 + (q & 1);
            ra[i][t] = (r * UN + (u ^ (r & (UN - 1)))) * 32 + (sub & 3) * 8;
        }
#pragma unroll
        for (int j = 0; j < FK; ++j) {
            const int u = wk * FK * 2 + j * 2 + (q & 1);
            rb[j][t] = kDyBytes + (r * UK + (u ^ (r & (UK - 1)))) * 32 + (sub & 3) * 8;
        }
    }
    auto read = [&](const char *p, int a, int b) {
        typedef __attribute__((address_space(3))) s16x4 *P;
        const s16x4 l = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + a));
        const s16x4 h = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + b));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(l, h, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto products = [&](int st) {
        const char *base = lds + (st & 1) * kStage;
#pragma unroll
        for (int ks = 0; ks < ROWS / 16; ++ks) {
            bf16x8 a[FN], b[FK];
#pragma unroll
            for (int j = 0; j < FK; ++j)
                b[j] = read(base + ks * 16 * BK * 2, rb[j][0], rb[j][1]);
#pragma unroll
            for (int i = 0; i < FN; ++i)
                a[i] = read(base + ks * 16 * BN * 2, ra[i][0], ra[i][1]);
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FK; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    };

    // ---- stages ----
    if (steps > 0) {
        fetch_index(0);
        fetch_x(0);
        fetch_dy(0);
        fetch_index(1);
        put_x(0);
        put_dy(0);
        fetch_x(1);
        fetch_dy(1);
        fetch_index(2);
        for (int st = 0; st < steps; ++st) {
            // this stage has been put down, and the other buffer is read
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            // (past the last stage: rows read again, put where nobody reads)
            put_x(st + 1);
            put_dy(st + 1);
            fetch_x(st + 2);
            fetch_dy(st + 2);
            fetch_index(st + 3);
            products(st);
        }
    }

    // ---- results: lane l holds column l mod 32, rows 8 (r / 4) + 4 (l / 32) +
    // r mod 4 of each fragment ----
    float *out = g.out + grp * g.out_stride;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int n = n0 + (wn * FN + i) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
            if (n >= g.N) continue;
#pragma unroll
            for (int j = 0; j < FK; ++j) {
                const int k = k0 + (wk * FK + j) * 32 + (lane & 31);
                if (k >= g.K) continue;
                float *p = out + n * g.ldo + k;
                *p = g.accumulate ? *p + acc[i][j][r] : acc[i][j][r];
            }
        }
}

constexpr int64_t kLaunchThreads = 0xFFFFFFFFll;

template <int FN, int FK, int WN, int WK, int ROWS, bool WHOLE, bool PACKED>
hipError_t wgrad_as(const WgradArgs &g, hipStream_t s, bool &too_large) {
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32, kThreads = WN * WK * 64;
    constexpr int kLds = 2 * ROWS * (BN + BK) * 2;
    const int64_t tn = (g.N + BN - 1) / BN, tk = (g.K + BK - 1) / BK;
    too_large = tn * tk * g.G > kLaunchThreads / kThreads;
    if (too_large) return hipSuccess;
    const auto kernel = k_wgrad<FN, FK, WN, WK, ROWS, WHOLE, PACKED>;
    if (kLds > 65536) {
        const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                  hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (he != hipSuccess) return he;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(tn * tk * g.G)), dim3(kThreads), kLds,
                       s, g, fast_div(g.index ? g.index_div : 1), static_cast<int>(tn),
                       static_cast<int>(tk));
    return hipGetLastError();
}

template <int FN, int FK, int WN, int WK, int ROWS>
hipError_t wgrad_any(const WgradArgs &g, hipStream_t s, bool &too_large) {
    const bool whole = g.vec_dy && g.N % 8 == 0 && (g.x_scale || (g.vec_x && g.K % 8 == 0));
    if (g.x_scale)
        return whole ? wgrad_as<FN, FK, WN, WK, ROWS, true, true>(g, s, too_large)
                     : wgrad_as<FN, FK, WN, WK, ROWS, false, true>(g, s, too_large);
    return whole ? wgrad_as<FN, FK, WN, WK, ROWS, true, false>(g, s, too_large)
                 : wgrad_as<FN, FK, WN, WK, ROWS, false, false>(g, s, too_large);
}

}  // namespace

int wgrad_parts(int, int, int, int, bool, int) { return 1; }

hipError_t launch_wgrad(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    too_large = false;
    if (g.N == 0 || g.K == 0 || g.G == 0) return hipSuccess;
    const int64_t large = static_cast<int64_t>((g.N + 255) / 256) * ((g.K + 255) / 256) * g.G;
    if (large >= c.num_cu) return wgrad_any<4, 2, 2, 4, 32>(g, s, too_large);
    return wgrad_any<2, 2, 2, 2, 32>(g, s, too_large);
}

}  // namespace ue
