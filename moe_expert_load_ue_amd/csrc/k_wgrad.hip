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

// The two low int8 of v times a power of two as bf16: the products' low halves
// are zero.
__device__ __forceinline__ uint32_t widen_pair(uint32_t v, float step) {
    const float f0 = static_cast<float>(static_cast<int8_t>(v)) * step;
    const float f1 = static_cast<float>(static_cast<int8_t>(v >> 8)) * step;
    return __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
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

// FN, FK: 32-column fragments of dy and of x per wave; WN, WK: waves along each.
// WHOLE: rows are 16-byte aligned and multiples of 8 columns (packed x always
// is), so that pieces are whole or nobody's.
//
// A stage is four steps of 16 rows. A step's operands are read from LDS during
// the step before; the next stage is put down during the second and third step,
// and each of its registers is at once filled with the stage after that. So by
// the end of the third step this stage has been read and the next one is in
// LDS: one barrier there.
constexpr int kStep = 16, kSteps = 4, kRows = kStep * kSteps;

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED, bool INDEXED>
__global__ __launch_bounds__(WN *WK * 64, 2) void k_wgrad(
    WgradArgs g, FastDiv div, int tiles_n, int tiles_k) {
    constexpr int kThreads = WN * WK * 64;
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32;
    constexpr int UN = BN / kUnit, UK = BK / kUnit;          // units of a row
    constexpr int kDyBytes = kRows * BN * 2, kXBytes = kRows * BK * 2;
    constexpr int kUnitsX = kRows * UK / kThreads;           // units of a thread
    constexpr int kUnitsDy = kRows * UN / kThreads;
    constexpr int kGapX = kThreads / UK, kGapDy = kThreads / UN;   // rows between them
    static_assert(kUnitsX * kThreads == kRows * UK && kUnitsDy * kThreads == kRows * UN,
                  "whole units per thread");
    static_assert((UN == 8 || UN == 16) && (UK == 8 || UK == 16));
    // both stages of dy, then both of x: a stage is an offset that fits the
    // instructions'
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
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int steps = (hi - lo + kRows - 1) / kRows;
    // first row of a stage (past the last one: the last one's, read again and
    // put where nobody reads it)
    auto first_of = [&](int st) { return lo + (st < steps ? st : steps - 1) * kRows; };

    // ---- loads: rows past the group's last are read again as the last one and
    // put down as zeros; pieces past the last column are read as others
    // (results of columns that nobody stores) ----
    const int dy_row = tid / UN, dy_n = n0 + tid % UN * kUnit;
    const uint32_t dy_at = dy_n < g.N ? dy_n * 2 : 0;
    const uint32_t dy_up = dy_n + 8 < g.N ? 16 : 0;
    Unit dyr[kUnitsDy];
    auto fetch_dy = [&](int st, int c) {
        const int m0 = first_of(st), left = hi - m0;
        const char *base = reinterpret_cast<const char *>(g.dy + m0 * g.lddy);
        int r = c * kGapDy + dy_row;
        if (left < kRows) r = r < left ? r : left - 1;
        const uint32_t at = r * static_cast<uint32_t>(g.lddy * 2);
        if constexpr (WHOLE) {
            dyr[c].lo = *reinterpret_cast<const u32x4 *>(base + (at + dy_at));
            dyr[c].hi = *reinterpret_cast<const u32x4 *>(base + (at + dy_at + dy_up));
        } else {
            dyr[c] = load_unit(reinterpret_cast<const uint16_t *>(base + at) + dy_n, g.N - dy_n);
        }
    };
    // LDS places of a row's units: the units' first halves side by side, then
    // the second ones (16 lanes that put down a row meet all 64 banks), unit u at
    // u ^ 2 (r mod 4), so that the four rows of two units that 32 lanes read meet
    // all banks too
    auto place = [](int units, int r, int u, int half) {
        const int p = u ^ (2 * (r & 3));
        return units == 16 ? (r * 32 + half * 16 + (p ^ (half * 8))) * 16
                           : (r * 16 + (half ^ (r & 1)) * 8 + p) * 16;
    };
    auto put = [&](char *base, int units, int r, int u, const Unit &v) {
        *reinterpret_cast<u32x4 *>(base + place(units, r, u, 0)) = v.lo;
        *reinterpret_cast<u32x4 *>(base + place(units, r, u, 1)) = v.hi;
    };
    auto put_dy = [&](int st, int buf, int c) {
        const int left = hi - lo - st * kRows, r = c * kGapDy + dy_row;
        if (left < kRows && r >= left) dyr[c] = Unit{};
        put(lds + buf * kDyBytes, UN, r, tid % UN, dyr[c]);
    };
    // x: the index of a row a stage before its units
    const int x_row = tid / UK, x_k = k0 + tid % UK * kUnit;
    const int x_at = x_k < g.K ? x_k : 0;
    const int x_up = x_k + 8 < g.K ? 8 : 0;
    int index[kUnitsX] = {};
    auto fetch_index = [&](int st, int c) {
        const int m0 = first_of(st), left = hi - m0;
        int r = c * kGapX + x_row;
        if (left < kRows) r = r < left ? r : left - 1;
        if constexpr (INDEXED) index[c] = (g.index + m0)[r];
    };
    struct Raw { u32x4 q; uint32_t s; };
    Raw xq[PACKED ? kUnitsX : 1];
    Unit xu[PACKED ? 1 : kUnitsX];
    bool live[kUnitsX];
    auto fetch_x = [&](int st, int c) {
        const int m = lo + st * kRows + c * kGapX + x_row;
        const int i = INDEXED ? index[c] : m;
        const uint32_t r = INDEXED ? div_by(i, div) : i;
        live[c] = i >= 0 && r < static_cast<uint32_t>(g.x_rows) && m < hi;
        const uint64_t row = live[c] ? r : 0;
        if constexpr (PACKED) {
            // (rows are readable up to a multiple of 16)
            xq[c].q = *reinterpret_cast<const u32x4 *>(
                static_cast<const int8_t *>(g.x) + (row * static_cast<uint32_t>(g.ldx) + x_at));
            xq[c].s = g.x_scale[row * static_cast<uint32_t>(g.lds) + x_at / UE_PACK_BLOCK];
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(g.x) + row * static_cast<uint32_t>(g.ldx);
            if constexpr (WHOLE) {
                xu[c].lo = *reinterpret_cast<const u32x4 *>(p + x_at);
                xu[c].hi = *reinterpret_cast<const u32x4 *>(p + x_at + x_up);
            } else {
                xu[c] = load_unit(p + x_k, g.K - x_k);
            }
        }
    };
    // A unit is made ready in kParts parts: two columns each, or at once.
    constexpr int kParts = 8;
    Unit ready;
    auto ready_x = [&](int c, int part) {
        uint32_t v;
        if constexpr (PACKED) {
            // (or the compiler takes bytes out of a load as soon as it is issued)
            if (part == 0) asm volatile("" : "+v"(xq[c].q), "+v"(xq[c].s));
            const float step = live[c] ? scale_step(xq[c].s) : 0.f;
            v = widen_pair(xq[c].q[part / 2] >> (16 * (part & 1)), step);
        } else {
            v = live[c] ? (part < 4 ? xu[c].lo[part & 3] : xu[c].hi[part & 3]) : 0u;
        }
        if (part < 4) ready.lo[part & 3] = v;
        else ready.hi[part & 3] = v;
    };
    auto put_x = [&](int buf, int c) {
        put(lds + 2 * kDyBytes + buf * kXBytes, UK, c * kGapX + x_row, tid % UK, ready);
    };

    // ---- products ----
    f32x16 acc[FN][FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j) acc[i][j] = f32x16{};
    const int wn = wv / WK, wk = wv % WK;
    // where this lane reads: four rows of one unit per 16 lanes; half of a
    // wave's lanes take rows 0-7 of a step, half 8-15, in two reads
    const int q = lane >> 4, sub = lane & 15;
    const int r0 = 8 * (q >> 1) + (sub >> 2);
    const char *ra[FN], *rb[FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
        ra[i] = lds + place(UN, r0, (wn * FN + i) * 2 + (q & 1), (sub >> 1) & 1) + (sub & 1) * 8;
#pragma unroll
    for (int j = 0; j < FK; ++j)
        rb[j] = lds + 2 * kDyBytes +
                place(UK, r0, (wk * FK + j) * 2 + (q & 1), (sub >> 1) & 1) + (sub & 1) * 8;
    struct Operands { s16x4 a[FN][2], b[FK][2]; };
    constexpr int kReads = 2 * (FN + FK);
    auto read = [&](Operands &o, int buf, int step, int t) {
        typedef __attribute__((address_space(3))) s16x4 *P;
        // x's fragments first, every dy fragment meets them
        if (t < 2 * FK) {
            const int off = buf * kXBytes + (step * kStep + t % 2 * 4) * BK * 2;
            o.b[t / 2][t % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(rb[t / 2] + off));
        } else {
            const int i = t / 2 - FK, off = buf * kDyBytes + (step * kStep + t % 2 * 4) * BN * 2;
            o.a[i][t % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(ra[i] + off));
        }
    };
    auto joined = [](const s16x4 (&v)[2]) {
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // The products of one step: work(p) stands behind the p-th matrix
    // instruction. A wave issues in order, and what stands between matrix
    // instructions runs beside them.
    constexpr int kAll = FN * FK;
    auto products = [&](const Operands &o, auto work) {
#pragma unroll
        for (int p = 0; p < kAll; ++p) {
            const int i = p / FK, j = p % FK;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(joined(o.a[i]), joined(o.b[j]),
                                                                acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            work(p);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the p-th share of a step's operand reads
    auto reads = [&](Operands &o, int buf, int step, int p) {
#pragma unroll
        for (int t = p * kReads / kAll; t < (p + 1) * kReads / kAll; ++t) read(o, buf, step, t);
    };
    Operands o0, o1;
    auto stage = [&](int st, auto buffer) {
        constexpr int buf = decltype(buffer)::value, other = 1 - buf;
        // units of x that are made ready behind the instructions of step n
        auto x_step = [&](int n, int p) {
#pragma unroll
            for (int c = n; c < kUnitsX; c += 2) {
#pragma unroll
                for (int part = p * kParts / kAll; part < (p + 1) * kParts / kAll; ++part)
                    ready_x(c, part);
                if (p + 1 == kAll) {
                    put_x(other, c);
                    fetch_x(st + 2, c);
                    fetch_index(st + 3, c);
                }
            }
        };
        products(o0, [&](int p) {
            reads(o1, buf, 1, p);
            x_step(0, p);
        });
        products(o1, [&](int p) {
            reads(o0, buf, 2, p);
            x_step(1, p);
        });
        products(o0, [&](int p) {
            reads(o1, buf, 3, p);
#pragma unroll
            for (int c = p * kUnitsDy / kAll; c < (p + 1) * kUnitsDy / kAll; ++c) {
                put_dy(st + 1, other, c);
                fetch_dy(st + 2, c);
            }
        });
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        products(o1, [&](int p) { reads(o0, other, 0, p); });
    };
    static_assert(kUnitsX <= 2, "a unit a step");
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;

    // ---- stages ----
    if (steps > 0) {
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) fetch_index(0, c);
#pragma unroll
        for (int c = 0; c < kUnitsDy; ++c) fetch_dy(0, c);
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) {
            fetch_x(0, c);
            fetch_index(1, c);
        }
#pragma unroll
        for (int c = 0; c < kUnitsDy; ++c) {
            put_dy(0, 0, c);
            fetch_dy(1, c);
        }
#pragma unroll
        for (int c = 0; c < kUnitsX; ++c) {
#pragma unroll
            for (int part = 0; part < kParts; ++part) ready_x(c, part);
            put_x(0, c);
            fetch_x(1, c);
            fetch_index(2, c);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int t = 0; t < kReads; ++t) read(o0, 0, 0, t);
        for (int st = 0; st < steps; st += 2) {
            stage(st, Even{});
            if (st + 1 < steps) stage(st + 1, Odd{});
        }
    }

    // ---- results: lane l holds column l mod 32, rows 8 (r / 4) + 4 (l / 32) +
    // r mod 4 of each fragment: whole lines of 128 bytes per store ----
    const int nb = n0 + wn * FN * 32 + 4 * (lane >> 5), kb = k0 + wk * FK * 32 + (lane & 31);
    float *const out = g.out + grp * g.out_stride + nb * g.ldo + kb;
    auto results = [&](auto inside, auto add) {
        constexpr bool kInside = decltype(inside)::value, kAdd = decltype(add)::value;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
                auto each = [&](auto f) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = h + e, n = i * 32 + 8 * (r / 4) + r % 4;
#pragma unroll
                        for (int j = 0; j < FK; ++j)
                            if (kInside || (nb + n < g.N && kb + j * 32 < g.K))
                                f(out + n * g.ldo + j * 32, e, j, acc[i][j][r]);
                    }
                };
                float old[8][FK];
                if (kAdd) each([&](float *p, int e, int j, float) { old[e][j] = *p; });
                each([&](float *p, int e, int j, float v) { *p = kAdd ? old[e][j] + v : v; });
            }
    };
    typedef std::true_type Yes;
    typedef std::false_type No;
    if (n0 + BN <= g.N && k0 + BK <= g.K) {
        if (g.accumulate) results(Yes{}, Yes{});
        else results(Yes{}, No{});
    } else {
        if (g.accumulate) results(No{}, Yes{});
        else results(No{}, No{});
    }
}

constexpr int64_t kLaunchThreads = 0xFFFFFFFFll;

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED, bool INDEXED>
hipError_t wgrad_as(const WgradArgs &g, hipStream_t s, bool &too_large) {
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32, kThreads = WN * WK * 64;
    constexpr int kLds = 2 * kRows * (BN + BK) * 2;
    const int64_t tn = (g.N + BN - 1) / BN, tk = (g.K + BK - 1) / BK;
    too_large = tn * tk * g.G > kLaunchThreads / kThreads;
    if (too_large) return hipSuccess;
    const auto kernel = k_wgrad<FN, FK, WN, WK, WHOLE, PACKED, INDEXED>;
    if (kLds > 65536) {
        const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                  hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (he != hipSuccess) return he;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(tn * tk * g.G)), dim3(kThreads), kLds,
                       s, g, fast_div(INDEXED ? g.index_div : 1), static_cast<int>(tn),
                       static_cast<int>(tk));
    return hipGetLastError();
}

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED>
hipError_t wgrad_rows(const WgradArgs &g, hipStream_t s, bool &too_large) {
    return g.index ? wgrad_as<FN, FK, WN, WK, WHOLE, PACKED, true>(g, s, too_large)
                   : wgrad_as<FN, FK, WN, WK, WHOLE, PACKED, false>(g, s, too_large);
}

template <int FN, int FK, int WN, int WK>
hipError_t wgrad_any(const WgradArgs &g, hipStream_t s, bool &too_large) {
    const bool whole = g.vec_dy && g.N % 8 == 0 && (g.x_scale || (g.vec_x && g.K % 8 == 0));
    if (g.x_scale)
        return whole ? wgrad_rows<FN, FK, WN, WK, true, true>(g, s, too_large)
                     : wgrad_rows<FN, FK, WN, WK, false, true>(g, s, too_large);
    return whole ? wgrad_rows<FN, FK, WN, WK, true, false>(g, s, too_large)
                 : wgrad_rows<FN, FK, WN, WK, false, false>(g, s, too_large);
}

}  // namespace

int wgrad_parts(int, int, int, int, bool, int) { return 1; }

hipError_t launch_wgrad(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    too_large = false;
    if (g.N == 0 || g.K == 0 || g.G == 0) return hipSuccess;
    const int64_t large = static_cast<int64_t>((g.N + 255) / 256) * ((g.K + 255) / 256) * g.G;
    if (large >= c.num_cu) return wgrad_any<4, 2, 2, 4>(g, s, too_large);
    return wgrad_any<2, 2, 2, 2>(g, s, too_large);
}

}  // namespace ue
