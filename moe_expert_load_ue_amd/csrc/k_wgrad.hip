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
// A workgroup walks tiles, and the stages of all of them are one stream: while a
// stage's products run, the next one's rows go to LDS, those of the one after
// are on their way to registers, and the row numbers of the third too, whichever
// tiles they are of. So the first stages of a tile are there when the results of
// the one before have been stored. (A workgroup per tile, with nothing under its
// first loads and its stores, took 870 us for 72 groups of 2048x4096 with 455
// rows each; its stores alone 500, all but the stores 737.)
//
// A stage is four steps of 16 rows. A step's operands are read from LDS during
// the step before, and the next stage is put down during the first three. So by
// the end of the third step this stage has been read and the next one is in
// LDS: one barrier there.
constexpr int kStep = 16;

// A stage of a tile: rows m0 .. of the group, `left` of them in the group still
// (0: none, for a group without rows, or behind the last tile).
struct Stage {
    int m0, left, grp, n0, k0;
    bool real;
};

template <int FN, int FK, int WN, int WK, int STEPS, bool WHOLE, bool PACKED, bool INDEXED>
__global__ __launch_bounds__(WN *WK * 64, 2) void k_wgrad(
    WgradArgs g, FastDiv div, int tiles_n, int tiles_k) {
    constexpr int kThreads = WN * WK * 64, kRows = STEPS * kStep;
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32;
    constexpr int UN = BN / kUnit, UK = BK / kUnit;          // units of a row
    constexpr int kDyBytes = kRows * BN * 2, kXBytes = kRows * BK * 2;
    constexpr int kGapX = kThreads / UK, kGapDy = kThreads / UN;
    // units of a thread, of rows kGap apart
    constexpr int kUnitsX = kRows / kGapX, kUnitsDy = kRows / kGapDy;
    static_assert(kUnitsX >= 1 && kUnitsX <= 2 && kUnitsDy >= 1 && kUnitsDy <= 2);
    static_assert((UN == 8 || UN == 16) && (UK == 8 || UK == 16));
    // both stages of dy, then both of x
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- the stream of stages: tiles in launch order, those of a group side by
    // side along n first, so that an XCD (every eighth workgroup) keeps to some
    // columns of dy and every XCD has a share of every group ----
    const int per = tiles_n * tiles_k, total = per * g.G * g.parts;
    auto begin_tile = [&](int id) {
        Stage s;
        s.grp = id / per;
        const int in = id - s.grp * per;
        s.n0 = in % tiles_n * BN;
        s.k0 = in / tiles_n * BK;
        const int part = s.grp / g.G, grp = s.grp - part * g.G;
        int lo = 0, hi = g.M;
        if (g.offsets) {
            lo = g.offsets[grp];
            hi = g.offsets[grp + 1];
            lo = lo < 0 ? 0 : lo > g.M ? g.M : lo;
            hi = hi < lo ? lo : hi > g.M ? g.M : hi;
        }
        if (g.parts > 1) {
            // whole stages, but for the group's end
            const int len = ((hi - lo) / g.parts + kRows) / kRows * kRows;
            lo = (hi - lo) / len >= part ? lo + part * len : hi;
            hi = hi - lo > len ? lo + len : hi;
        }
        s.left = __builtin_amdgcn_readfirstlane(hi - lo);
        // (rows that are not there are read as some other row)
        s.m0 = __builtin_amdgcn_readfirstlane(lo < g.M ? lo : g.M - 1);
        s.real = true;
        return s;
    };
    int id = blockIdx.x;
    auto next_stage = [&](Stage &s) {
        if (s.left > kRows) {
            s.m0 += kRows;
            s.left -= kRows;
        } else if (id + static_cast<int>(gridDim.x) < total) {
            id += gridDim.x;
            s = begin_tile(id);
        } else {
            s.left = 0;
            s.real = false;
        }
    };
    // row r of a stage; past the last one, that one
    auto row_in = [](const Stage &s, int r) {
        return s.left >= kRows ? r : r < s.left ? r : s.left > 0 ? s.left - 1 : 0;
    };

    // ---- loads: two units of dy and of x per thread, a half at a time. Rows
    // that are not the stage's are put down as zeros; whole units are read with
    // the second half, when the first has been put down too; pieces past the last column
    // are read as others (results of columns that nobody stores) ----
    const int dy_row = tid / UN, dy_col = tid % UN * kUnit;
    const int x_row = tid / UK, x_col = tid % UK * kUnit;
    Unit dyr[kUnitsDy];
    auto fetch_dy = [&](const Stage &s, int c, int half) {
        const char *base = reinterpret_cast<const char *>(g.dy + s.m0 * g.lddy);
        const uint32_t at = row_in(s, c * kGapDy + dy_row) * static_cast<uint32_t>(g.lddy * 2);
        const int n = s.n0 + dy_col;
        if constexpr (WHOLE) {
            const int h = n + half * 8;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(base + (at + (h < g.N ? h * 2 : 0)));
            if (half) dyr[c].hi = v;
            else dyr[c].lo = v;
        } else if (half) {
            dyr[c] = load_unit(reinterpret_cast<const uint16_t *>(base + at) + n, g.N - n);
        }
    };
    int index[kUnitsX] = {};
    auto fetch_index = [&](const Stage &s, int c) {
        if constexpr (INDEXED) index[c] = (g.index + s.m0)[row_in(s, c * kGapX + x_row)];
    };
    struct Raw { u32x4 q; uint32_t s; };
    Raw xq[PACKED ? kUnitsX : 1];
    Unit xu[PACKED ? 1 : kUnitsX];
    bool live[kUnitsX];
    uint32_t x_of[kUnitsX];
    auto fetch_x = [&](const Stage &s, int c, int half) {
        if (half == 0) {
            const int r = c * kGapX + x_row, i = INDEXED ? index[c] : s.m0 + r;
            const uint32_t row = INDEXED ? div_by(i, div) : i;
            live[c] = i >= 0 && row < static_cast<uint32_t>(g.x_rows) && r < s.left;
            x_of[c] = live[c] ? row : 0;
        }
        const uint64_t row = x_of[c];
        const int k = s.k0 + x_col;
        if constexpr (PACKED) {
            // (rows are readable up to a multiple of 16)
            const int at = k < g.K ? k : 0;
            if (half) xq[c].s = g.x_scale[row * static_cast<uint32_t>(g.lds) + at / UE_PACK_BLOCK];
            else xq[c].q = *reinterpret_cast<const u32x4 *>(
                static_cast<const int8_t *>(g.x) + (row * static_cast<uint32_t>(g.ldx) + at));
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(g.x) + row * static_cast<uint32_t>(g.ldx);
            if constexpr (WHOLE) {
                const int h = k + half * 8;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(p + (h < g.K ? h : 0));
                if (half) xu[c].hi = v;
                else xu[c].lo = v;
            } else if (half) {
                xu[c] = load_unit(p + k, g.K - k);
            }
        }
    };

    // ---- LDS: the first halves of a row's units side by side, then the second
    // ones (16 lanes that put down a row meet all 64 banks), unit u at
    // u ^ 2 (r mod 4), so that the four rows of two units that 32 lanes read meet
    // all banks too ----
    auto place = [](int units, int r, int u, int half) {
        const int p = u ^ (2 * (r & 3));
        return units == 16 ? (r * 32 + half * 16 + (p ^ (half * 8))) * 16
                           : (r * 16 + (half ^ (r & 1)) * 8 + p) * 16;
    };
    typedef __attribute__((address_space(3))) char *Lds;
    const Lds base = (Lds)lds;
    // where units go, of dy and of x (the second one kGap rows on); which buffer
    // alternates: `flip` times the buffers' size is added to all places
    Lds wd[2], wx[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        wd[half] = base + place(UN, dy_row, tid % UN, half);
        wx[half] = base + 2 * kDyBytes + place(UK, x_row, tid % UK, half);
    }
    static_assert(kGapDy % 4 == 0 && kGapX % 4 == 0, "the same place in the row");
    auto put = [](Lds to, const u32x4 &v) {
        *(__attribute__((address_space(3))) u32x4 *)to = v;
    };
    auto put_dy = [&](const Stage &s, int c, int half) {
        u32x4 v = half ? dyr[c].hi : dyr[c].lo;
        if (s.left < kRows && c * kGapDy + dy_row >= s.left) v = u32x4{};
        put(wd[half] + c * kGapDy * BN * 2, v);
    };
    // A unit of x is made ready in kParts parts, two columns each.
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
    auto put_x = [&](int c, int half) {
        put(wx[half] + c * kGapX * BK * 2, half ? ready.hi : ready.lo);
    };

    // ---- products ----
    f32x16 acc[FN][FK];
    const int wn = wv / WK, wk = wv % WK;
    // where this lane reads: four rows of one unit per 16 lanes; half of a
    // wave's lanes take rows 0-7 of a step, half 8-15, in two reads
    const int q = lane >> 4, sub = lane & 15;
    const int r0 = 8 * (q >> 1) + (sub >> 2);
    Lds ra[FN], rb[FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
        ra[i] = base + place(UN, r0, (wn * FN + i) * 2 + (q & 1), (sub >> 1) & 1) + (sub & 1) * 8;
#pragma unroll
    for (int j = 0; j < FK; ++j)
        rb[j] = base + 2 * kDyBytes +
                place(UK, r0, (wk * FK + j) * 2 + (q & 1), (sub >> 1) & 1) + (sub & 1) * 8;
    struct Operands { s16x4 a[FN][2], b[FK][2]; };
    constexpr int kReads = 2 * (FN + FK), kAll = FN * FK;
    auto read = [&](Operands &o, int step, int t) {
        typedef __attribute__((address_space(3))) s16x4 *P;
        // x's fragments first, every dy fragment meets them
        if (t < 2 * FK)
            o.b[t / 2][t % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (P)(rb[t / 2] + (step * kStep + t % 2 * 4) * BK * 2));
        else
            o.a[t / 2 - FK][t % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (P)(ra[t / 2 - FK] + (step * kStep + t % 2 * 4) * BN * 2));
    };
    auto joined = [](const s16x4 (&v)[2]) {
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    int delta_dy = kDyBytes, delta_x = kXBytes;      // to the other buffer
    auto flip_puts = [&] {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            wd[half] += delta_dy;
            wx[half] += delta_x;
        }
    };
    auto flip_reads = [&] {
#pragma unroll
        for (int i = 0; i < FN; ++i) ra[i] += delta_dy;
#pragma unroll
        for (int j = 0; j < FK; ++j) rb[j] += delta_x;
    };
    // Stages: of the products, of what is put down, of units on their way, and
    // of row numbers.
    Stage now, put_of, fetch_of, index_of;
    // What stands at 32 places of a stage: a unit is made ready and put down and
    // its registers filled again, a load or a store at a time. Loads are waited
    // for in their order, so each is used after about as many others.
    auto at_place = [&](int at) {
        constexpr int x1 = kUnitsX - 1, dy1 = kUnitsDy - 1;
        if (at < kParts) ready_x(0, at);
        else if (kUnitsX > 1 && at < 2 * kParts) ready_x(x1, at - kParts);
        switch (at) {
            case 1: put_dy(put_of, 0, 0); break;
            case 2: fetch_dy(fetch_of, 0, 0); break;
            case 4: put_x(0, 0); break;
            case 5: put_dy(put_of, 0, 1); break;
            case 6: fetch_dy(fetch_of, 0, 1); break;
            case 7: put_x(0, 1); break;
            case 8: fetch_x(fetch_of, 0, 0); break;
            case 9: fetch_x(fetch_of, 0, 1); fetch_index(index_of, 0); break;
            default: break;
        }
        if (kUnitsDy > 1) switch (at) {
            case 9: put_dy(put_of, dy1, 0); break;
            case 10: fetch_dy(fetch_of, dy1, 0); break;
            case 13: put_dy(put_of, dy1, 1); break;
            case 14: fetch_dy(fetch_of, dy1, 1); break;
            default: break;
        }
        if (kUnitsX > 1) switch (at) {
            case 12: put_x(x1, 0); break;
            case 15: put_x(x1, 1); break;
            case 16: fetch_x(fetch_of, x1, 0); break;
            case 17: fetch_x(fetch_of, x1, 1); fetch_index(index_of, x1); break;
            default: break;
        }
    };
    constexpr int kEach = 32 / (STEPS * kAll);
    static_assert(kEach * STEPS * kAll == 32 && (STEPS == 2 || STEPS == 4));
    // The products of one step on `use`, while the operands of `step` are read
    // into `load`. A wave issues in order, and what stands between matrix
    // instructions runs beside them.
    auto products = [&](int nth, const Operands &use, Operands &load, int step) {
#pragma unroll
        for (int p = 0; p < kAll; ++p) {
            const int i = p / FK, j = p % FK;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(joined(use.a[i]), joined(use.b[j]),
                                                                acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = p * kReads / kAll; t < (p + 1) * kReads / kAll; ++t) read(load, step, t);
#pragma unroll
            for (int e = 0; e < kEach; ++e) at_place((nth * kAll + p) * kEach + e);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FK; ++j) acc[i][j] = f32x16{};
    };

    // ---- results: lane l holds column l mod 32, rows 8 (r / 4) + 4 (l / 32) +
    // r mod 4 of each fragment: whole lines of 128 bytes per store, which nobody
    // reads soon (past the caches 870 us, through them 1030, of the size above) ----
    auto results = [&](const Stage &s) {
        const int nb = s.n0 + wn * FN * 32 + 4 * (lane >> 5);
        const int kb = s.k0 + wk * FK * 32 + (lane & 31);
        // (kept from the compiler, which would hold every row's offset in
        // registers all along)
        int64_t ldo = g.ldo;
        asm volatile("" : "+s"(ldo));
        float *const out = g.out + s.grp * g.out_stride + nb * ldo + kb;
        auto store = [&](auto inside, auto add) {
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
                                    f(out + n * ldo + j * 32, e, j, acc[i][j][r]);
                        }
                    };
                    float old[8][FK];
                    if (kAdd) each([&](float *p, int e, int j, float) { old[e][j] = *p; });
                    each([&](float *p, int e, int j, float v) {
                        __builtin_nontemporal_store(kAdd ? old[e][j] + v : v, p);
                    });
                }
        };
        typedef std::true_type Yes;
        typedef std::false_type No;
        if (s.n0 + BN <= g.N && s.k0 + BK <= g.K) {
            if (g.accumulate) store(Yes{}, Yes{});
            else store(Yes{}, No{});
        } else {
            if (g.accumulate) store(No{}, Yes{});
            else store(No{}, No{});
        }
    };

    // ---- the first stages ----
    now = begin_tile(id);
    put_of = now;
    next_stage(put_of);
    fetch_of = put_of;
    next_stage(fetch_of);
    index_of = fetch_of;
    next_stage(index_of);
#pragma unroll
    for (int c = 0; c < kUnitsX; ++c) fetch_index(now, c);
#pragma unroll
    for (int c = 0; c < 2 * kUnitsDy; ++c) fetch_dy(now, c / 2, c % 2);
#pragma unroll
    for (int c = 0; c < 2 * kUnitsX; ++c) fetch_x(now, c / 2, c % 2);
#pragma unroll
    for (int c = 0; c < kUnitsX; ++c) fetch_index(put_of, c);
#pragma unroll
    for (int c = 0; c < 2 * kUnitsDy; ++c) {
        put_dy(now, c / 2, c % 2);
        fetch_dy(put_of, c / 2, c % 2);
    }
#pragma unroll
    for (int c = 0; c < kUnitsX; ++c) {
#pragma unroll
        for (int part = 0; part < kParts; ++part) ready_x(c, part);
        put_x(c, 0);
        put_x(c, 1);
        fetch_x(put_of, c, 0);
        fetch_x(put_of, c, 1);
        fetch_index(fetch_of, c);
        // (a byte that is known to be one from here on would be cut to it in the
        // loop, at a place that waits for it too soon)
        if constexpr (PACKED) asm volatile("" : "+v"(xq[c].s));
    }
    flip_puts();
    clear();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    Operands o0, o1;
#pragma unroll
    for (int t = 0; t < kReads; ++t) read(o0, 0, t);

    while (now.real) {
        products(0, o0, o1, 1);
        if constexpr (STEPS == 4) {
            products(1, o1, o0, 2);
            products(2, o0, o1, 3);
        }
        // this stage has been read by every wave, the next one been put down
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        flip_reads();
        delta_dy = -delta_dy;
        delta_x = -delta_x;
        flip_puts();
        products(STEPS - 1, o1, o0, 0);
        if (now.left <= kRows) {
            results(now);
            clear();
        }
        now = put_of;
        put_of = fetch_of;
        fetch_of = index_of;
        next_stage(index_of);
    }
}

// ---- which tile ----
enum WgradTile { kTile256, kTile256x128, kTile128 };

int64_t tiles_of(int N, int K, int bn, int bk) {
    return static_cast<int64_t>((N + bn - 1) / bn) * ((K + bk - 1) / bk);
}
constexpr int kPartRows = 256, kMaxParts = 64;

WgradTile wgrad_tile(int M, int N, int K, int64_t G, int num_cu) {
#ifdef FORCE_TILE
    return FORCE_TILE;
#endif
    if (tiles_of(N, K, 256, 256) * G >= num_cu) return kTile256;
    return kTile128;
}

// Matrices of groups without any rows at all.
__global__ __launch_bounds__(kBlock) void k_wgrad_zero(WgradArgs g) {
    const int64_t rows = static_cast<int64_t>(g.G) * g.N;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float *out = g.out + r / g.N * g.out_stride + r % g.N * g.ldo;
        for (int k = threadIdx.x; k < g.K; k += kBlock) out[k] = 0.f;
    }
}

// The parts of split sums, added in order.
__global__ __launch_bounds__(kBlock) void k_wgrad_join(WgradArgs g) {
    const int64_t rows = static_cast<int64_t>(g.G) * g.N, all = rows * g.K;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float *out = g.out + r / g.N * g.out_stride + r % g.N * g.ldo;
        const float *part = g.part + r * g.K;
        for (int k = threadIdx.x; k < g.K; k += kBlock) {
            float v = g.accumulate ? out[k] : 0.f;
            for (int p = 0; p < g.parts; ++p) v += part[p * all + k];
            out[k] = v;
        }
    }
}

template <int FN, int FK, int WN, int WK, int STEPS, bool WHOLE, bool PACKED, bool INDEXED>
hipError_t wgrad_as(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32, kThreads = WN * WK * 64;
    constexpr int kLds = 2 * STEPS * kStep * (BN + BK) * 2;
    // as many workgroups as fit at once: two waves per SIMD
    constexpr int kPerCu = 512 / kThreads;
    const int64_t tn = (g.N + BN - 1) / BN, tk = (g.K + BK - 1) / BK, total = tn * tk * g.G * g.parts;
    too_large = total > 0x7FFFFFFF - kPerCu * c.num_cu;
    if (too_large) return hipSuccess;
    const auto kernel = k_wgrad<FN, FK, WN, WK, STEPS, WHOLE, PACKED, INDEXED>;
    if (kLds > 65536) {
        const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                  hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (he != hipSuccess) return he;
    }
    const int64_t grid = total < kPerCu * c.num_cu ? total : kPerCu * c.num_cu;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid)), dim3(kThreads), kLds, s, g,
                       fast_div(INDEXED ? g.index_div : 1), static_cast<int>(tn),
                       static_cast<int>(tk));
    return hipGetLastError();
}

template <int FN, int FK, int WN, int WK, int STEPS, bool WHOLE, bool PACKED>
hipError_t wgrad_rows(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    return g.index ? wgrad_as<FN, FK, WN, WK, STEPS, WHOLE, PACKED, true>(c, g, s, too_large)
                   : wgrad_as<FN, FK, WN, WK, STEPS, WHOLE, PACKED, false>(c, g, s, too_large);
}

template <int FN, int FK, int WN, int WK, int STEPS>
hipError_t wgrad_any(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    const bool whole = g.vec_dy && g.N % 8 == 0 && (g.x_scale || (g.vec_x && g.K % 8 == 0));
    if (g.x_scale)
        return whole ? wgrad_rows<FN, FK, WN, WK, STEPS, true, true>(c, g, s, too_large)
                     : wgrad_rows<FN, FK, WN, WK, STEPS, false, true>(c, g, s, too_large);
    return whole ? wgrad_rows<FN, FK, WN, WK, STEPS, true, false>(c, g, s, too_large)
                 : wgrad_rows<FN, FK, WN, WK, STEPS, false, false>(c, g, s, too_large);
}

hipError_t wgrad_tiles(ue_ctx &c, const WgradArgs &g, hipStream_t s, bool &too_large) {
    switch (wgrad_tile(g.M, g.N, g.K, static_cast<int64_t>(g.G) * g.parts, c.num_cu)) {
        case kTile256: return wgrad_any<4, 2, 2, 4, 4>(c, g, s, too_large);
        case kTile256x128: return wgrad_any<4, 2, 2, 2, 2>(c, g, s, too_large);
        default: return wgrad_any<2, 2, 2, 2, 4>(c, g, s, too_large);
    }
}

}  // namespace

int wgrad_parts(int M, int N, int K, int G, bool, int num_cu) {
    const int64_t tiles = tiles_of(N, K, 128, 128) * G;
    const int64_t slots = 2 * num_cu, rows = M / G;
    int64_t parts = slots / tiles;
    if (parts > rows / kPartRows) parts = rows / kPartRows;
    if (parts > kMaxParts) parts = kMaxParts;
    return parts > 1 ? static_cast<int>(parts) : 1;
}

hipError_t launch_wgrad(ue_ctx &c, const WgradArgs &a, hipStream_t s, bool &too_large) {
    too_large = false;
    if (a.N == 0 || a.K == 0 || a.G == 0) return hipSuccess;
    WgradArgs g = a;
    const int64_t rows = static_cast<int64_t>(g.G) * g.N, most = 64 * c.num_cu;
    const dim3 per_row(static_cast<uint32_t>(rows < most ? rows : most));
    if (g.M == 0) {
        if (g.accumulate) return hipSuccess;
        hipLaunchKernelGGL(k_wgrad_zero, per_row, dim3(kBlock), 0, s, g);
        return hipGetLastError();
    }
    if (g.parts == 1) return wgrad_tiles(c, g, s, too_large);
    g.out = g.part;
    g.ldo = g.K;
    g.out_stride = static_cast<int64_t>(g.N) * g.K;
    g.accumulate = false;
    const hipError_t he = wgrad_tiles(c, g, s, too_large);
    if (he != hipSuccess || too_large) return he;
    hipLaunchKernelGGL(k_wgrad_join, per_row, dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace ue
