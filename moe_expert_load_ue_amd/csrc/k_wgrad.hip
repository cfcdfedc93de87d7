// Gradients of the matrices of row groups (ue_weight_grad):
//   out[g, n, k] (+)= sum over the rows m of group g of dy[m, n] x[r(m), k]
//
// A workgroup makes tiles of the groups' matrices. Both operands lie row by row,
// with the sum going down the rows, while a matrix instruction wants each lane's
// eight terms side by side. So rows go to LDS as they are, in bf16, and come
// out transposed: a transposing LDS read gives each of 16 lanes one column of
// four rows. A stage is kRows rows, which come to registers, packed x is widened
// on the way down to LDS. Which four rows a lane's terms come from does not
// matter as long as both operands take the same.
//
// Rows in LDS are units of 16 columns (32 bytes), placed so that neither what is
// put down nor what is read back transposed meets a bank twice (no conflicts
// counted).
//
// Bound: not the products alone. One group of 8192 x 4096 x 7168, packed x, takes
// 465-475 us (1.02 PFLOP/s; bf16 x 451-456) at 1.97 GHz of 2.4, with the matrix units
// busy 46% of the cycles (five groups 51%): a stage takes 3900 cycles, of which the
// matrix instructions need 2048 and LDS 1290. Without its loads it takes 388 us,
// without what it puts down in LDS either 312: bringing rows to LDS through
// registers is a third of the time, and 120 of a wave's 215 vector instructions of a
// stage are addresses. Changes that took waiting away left the time alone: loads
// used a whole stage after they are issued in place of half of one (465-473 us, bf16
// x 458-470), workgroups started apart from each other (466-483). The clock falls
// under load, but power has not been measured, and the library's product of the same
// operand layout reaches 1180 TFLOP/s on the device. Four waves of 128 x 128 spilled (3.7 ms); tiles
// of 256 x 128 on four waves, two workgroups per CU, 575 us against 483; rows
// straight to LDS wait for each other, since the compiler puts a wait for all of
// them ahead of every LDS read.
#include "ue_train.h"

#include <atomic>
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

// Rows at any 2-byte alignment are read in pieces of eight elements all the
// same, past their end too (results of columns that nobody stores); but a piece
// that would pass the end of the whole matrix is read back from that end, and
// moved to its place when it is put down.
__device__ __forceinline__ u32x4 load_piece(const void *p) {
    struct __attribute__((packed, aligned(2))) Piece { u32x4 v; };
    return static_cast<const Piece *>(p)->v;
}
__device__ __forceinline__ u32x4 moved_down(u32x4 v, int elements) {
    uint64_t lo = static_cast<uint64_t>(v[1]) << 32 | v[0];
    uint64_t hi = static_cast<uint64_t>(v[3]) << 32 | v[2];
    const int bits = 16 * elements;
    if (bits >= 64) {
        lo = hi >> (bits & 63);
        hi = 0;
    } else if (bits > 0) {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
    }
    return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                 static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
}
constexpr int kPiece = 8;

// FN, FK: 32-column fragments of dy and of x per wave; WN, WK: waves along each.
// WHOLE: rows are 16-byte aligned and multiples of 8 columns (packed x always
// is), so that pieces are whole or nobody's.
//
// A workgroup walks tiles, and the stages of all of them are one stream: while a
// stage's products run, the next one's rows go to LDS, those of the one after
// are on their way to registers, and the row numbers of the third too, whichever
// tiles they are of. So the first stages of a tile are there when the results of
// the one before have been stored. (72 groups of 2048x4096 with 455 rows each on
// average take 780 us where they are even and 825-860 where their rows differ as
// routing's do; 752 at the least. A workgroup per tile, with nothing under its first
// loads and its stores, took 870 where this took 794. The stores alone take 500.)
//
// A stage is four steps of 16 rows. A step's operands are read from LDS during
// the step before, and the next stage is put down during the first three. So by
// the end of the third step this stage has been read and the next one is in
// LDS: one barrier there.
constexpr int kStep = 16, kSteps = 4, kRows = kStep * kSteps;

// A stage of a tile: rows m0 .. of the group, `left` of them in the group still
// (0: none, for a group without rows, or behind the last tile).
struct Stage {
    int m0, left, grp, n0, k0;
    bool real;
};

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED, bool INDEXED>
__global__ __launch_bounds__(WN *WK * 64, FN * FK > 8 ? 1 : 2) void k_wgrad(
    WgradArgs g, FastDiv div, int tiles_n, int tiles_k) {
    constexpr int kThreads = WN * WK * 64;
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32;
    constexpr int UN = BN / kUnit, UK = BK / kUnit;          // units of a row
    constexpr int kDyBytes = kRows * BN * 2, kXBytes = kRows * BK * 2;
    constexpr int kGapX = kThreads / UK, kGapDy = kThreads / UN;
    constexpr int kUnits = kRows / kGapX;        // of a thread, kGap rows apart
    static_assert(kGapX * kUnits == kRows && kGapDy * kUnits == kRows);
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
    // Stages: of the products, of what is put down, of units on their way, and
    // of row numbers.
    Stage now, put_of, fetch_of, index_of;
    // row r of a stage; past the last one, that one
    auto row_in = [](const Stage &s, int r) {
        return s.left >= kRows ? r : r < s.left ? r : s.left > 0 ? s.left - 1 : 0;
    };

    // ---- loads: units of dy and of x, a half at a time. Rows that are not the
    // stage's are put down as zeros; pieces past the last column are read as others
    // (results of columns that nobody stores) ----
    const int dy_row = tid / UN, dy_col = tid % UN * kUnit;
    const int x_row = tid / UK, x_col = tid % UK * kUnit;
    Unit dyr[kUnits];
    auto fetch_dy = [&](const Stage &s, int c, int half) {
        // (a piece before the stage's first row: what is read back from the end
        // may begin there, and offsets are unsigned)
        const int64_t first = s.m0 * g.lddy - (WHOLE ? 0 : kPiece);
        const uint32_t at = row_in(s, c * kGapDy + dy_row) * static_cast<uint32_t>(g.lddy);
        const int n = s.n0 + dy_col + half * kPiece;
        uint32_t from = at + (n < g.N ? n : 0);
        const uint16_t *p = g.dy + first;
        u32x4 v;
        if constexpr (WHOLE) {
            v = *reinterpret_cast<const u32x4 *>(p + from);
        } else {
            const int64_t last = (g.M - 1) * g.lddy + g.N - kPiece - first;
            const uint32_t most = last < 0x7FFFFFFF ? static_cast<uint32_t>(last) : 0x7FFFFFFFu;
            from += kPiece;
            v = load_piece(p + (from < most ? from : most));
        }
        if (half) dyr[c].hi = v;
        else dyr[c].lo = v;
    };
    int index[kUnits] = {};
    auto fetch_index = [&](const Stage &s, int c) {
        if constexpr (INDEXED) index[c] = (g.index + s.m0)[row_in(s, c * kGapX + x_row)];
    };
    struct Raw { u32x4 q; uint32_t s; };
    Raw xq[PACKED ? kUnits : 1];
    Unit xu[PACKED ? 1 : kUnits];
    bool live[kUnits];
    uint32_t x_of[kUnits];
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
            const int h = k + half * kPiece;
            u32x4 v;
            if constexpr (WHOLE) {
                v = *reinterpret_cast<const u32x4 *>(p + (h < g.K ? h : 0));
            } else {
                p += h < g.K ? h : 0;
                const uint16_t *last = static_cast<const uint16_t *>(g.x) +
                                       (g.x_rows - 1) * g.ldx + g.K - kPiece;
                v = load_piece(p < last ? p : last);
            }
            if (half) xu[c].hi = v;
            else xu[c].lo = v;
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
        if constexpr (!WHOLE) {
            if (s.m0 + kRows + kPiece > g.M) {
                const int n = s.n0 + dy_col + half * kPiece;
                const int64_t over = (s.m0 + row_in(s, c * kGapDy + dy_row) + 1 - g.M) * g.lddy +
                                     (n < g.N ? n : 0) + kPiece - g.N;
                if (over > 0) v = moved_down(v, static_cast<int>(over));
            }
        }
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
            if constexpr (!WHOLE) {
                // (x_of and the stage are still those of this unit)
                if (part % 4 == 0 && x_of[c] + kPiece >= static_cast<uint32_t>(g.x_rows)) {
                    const int k = put_of.k0 + x_col + part / 4 * kPiece;
                    const int64_t over = (static_cast<int64_t>(x_of[c]) + 1 - g.x_rows) * g.ldx +
                                         (k < g.K ? k : 0) + kPiece - g.K;
                    if (over > 0) {
                        u32x4 &u = part ? xu[c].hi : xu[c].lo;
                        u = moved_down(u, static_cast<int>(over));
                    }
                }
            }
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
    // What stands at the places of a stage, 16 for each unit: a unit is made ready
    // and put down and its registers filled again, a load or a store at a time.
    // Loads are waited for in their order, so each is used after about as many
    // others. All units have been put down by the middle of the stage.
    auto at_place = [&](int at) {
        const int c = at / kParts, r = at % kParts;
        if (c < kUnits) {
            ready_x(c, r);
            switch (r) {
                case 1: put_dy(put_of, c, 0); break;
                case 2: fetch_dy(fetch_of, c, 0); break;
                case 4: put_x(c, 0); break;
                case 5: put_dy(put_of, c, 1); break;
                case 6: fetch_dy(fetch_of, c, 1); break;
                case 7: put_x(c, 1); break;
                default: break;
            }
        }
        if (c > 0 && c <= kUnits) {
            if (r == 0) fetch_x(fetch_of, c - 1, 0);
            if (r == 1) {
                fetch_x(fetch_of, c - 1, 1);
                fetch_index(index_of, c - 1);
            }
        }
    };
    constexpr int kEach = 2 * kParts * kUnits / (kSteps * kAll);
    static_assert(kEach * kSteps * kAll == 2 * kParts * kUnits);
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
    // reads soon (past the caches 870 us, through them 1030, of the size above when
    // a workgroup made one tile) ----
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

    // ---- the first stages: the first one is put down, two more are on their
    // way ----
    put_of = begin_tile(id);
    fetch_of = put_of;
    next_stage(fetch_of);
    index_of = fetch_of;
    next_stage(index_of);
#pragma unroll
    for (int c = 0; c < kUnits; ++c) fetch_index(put_of, c);
#pragma unroll
    for (int c = 0; c < 2 * kUnits; ++c) fetch_dy(put_of, c / 2, c % 2);
#pragma unroll
    for (int c = 0; c < 2 * kUnits; ++c) fetch_x(put_of, c / 2, c % 2);
#pragma unroll
    for (int c = 0; c < kUnits; ++c) fetch_index(fetch_of, c);
#pragma unroll
    for (int c = 0; c < 2 * kUnits; ++c) {
        put_dy(put_of, c / 2, c % 2);
        fetch_dy(fetch_of, c / 2, c % 2);
    }
#pragma unroll
    for (int c = 0; c < kUnits; ++c) {
#pragma unroll
        for (int part = 0; part < kParts; ++part) ready_x(c, part);
        put_x(c, 0);
        put_x(c, 1);
        fetch_x(fetch_of, c, 0);
        fetch_x(fetch_of, c, 1);
        fetch_index(index_of, c);
        // (a byte that is known to be one from here on would be cut to it in the
        // loop, at a place that waits for it too soon)
        if constexpr (PACKED) asm volatile("" : "+v"(xq[c].s));
    }
    now = put_of;
    put_of = fetch_of;
    fetch_of = index_of;
    next_stage(index_of);
    flip_puts();
    clear();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    Operands o0, o1;
#pragma unroll
    for (int t = 0; t < kReads; ++t) read(o0, 0, t);

    while (now.real) {
        products(0, o0, o1, 1);
        products(1, o1, o0, 2);
        products(2, o0, o1, 3);
        // this stage has been read by every wave, the next one been put down
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        flip_reads();
        delta_dy = -delta_dy;
        delta_x = -delta_x;
        flip_puts();
        products(3, o1, o0, 0);
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

// Tiles of 256 x 256 on eight waves, one workgroup per CU, or of 128 x 128 on
// four, two per CU. By what each measured (us, packed x, groups of uneven length;
// mean rows x N x K):
//                            256    128
//    72 of  455x2048x4096     794   1119
//     5 of 1638x4096x7168     593    682
//    64 of  256x1024x2048     119    158
//     8 of  256x1024x2048      22     26
//     8 of  748x 316x3650      46     57   (240 tiles of 256)
//     3 of 4000x 760x3640     155    136   (135)
//     4 of 2048x1024x2048      87     67   (128)
//     8 of  600x 480x 352      30     23   (32)
//          32768x 128x 256      50     41   (in parts)
// So the large ones when they make work for three CUs of four. Added to what out
// holds (written), even groups: 5 of 1638x4096x7168 607 us (518), 72 of 455x2048x4096
// 1169 (780), 64 of 256x1024x2048 241 (125): one more read of out, with nothing
// under its loads.
enum WgradTile { kTile256, kTile128 };

int64_t tiles_of(int N, int K, int b) {
    return static_cast<int64_t>((N + b - 1) / b) * ((K + b - 1) / b);
}
WgradTile wgrad_tile(int N, int K, int64_t G, int num_cu) {
    return tiles_of(N, K, 256) * G >= num_cu * 3 / 4 ? kTile256 : kTile128;
}
constexpr int per_cu(int tile) { return tile == 256 ? 1 : 2; }      // workgroups

// Matrices too small to be read in pieces.
bool wgrad_tiny(const WgradArgs &g) {
    auto tiny = [](int64_t rows, int64_t ld, int cols) { return (rows - 1) * ld + cols < kPiece; };
    return tiny(g.M, g.lddy, g.N) || (!g.x_scale && tiny(g.x_rows, g.ldx, g.K));
}
// A part has at least kPartRows rows (on average), so that what it writes and
// reads again, 128 KB for a tile of 128, is less than the rows it saves others.
constexpr int kPartRows = 256, kMaxParts = 64;

// Matrices of groups without any rows at all.
__global__ __launch_bounds__(kBlock) void k_wgrad_zero(WgradArgs g) {
    const int64_t rows = static_cast<int64_t>(g.G) * g.N;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float *out = g.out + r / g.N * g.out_stride + r % g.N * g.ldo;
        for (int k = threadIdx.x; k < g.K; k += kBlock) out[k] = 0.f;
    }
}

// Those too small to be read in pieces: a thread per result.
__global__ __launch_bounds__(kBlock) void k_wgrad_tiny(WgradArgs g) {
    const int64_t each = static_cast<int64_t>(g.N) * g.K, all = each * g.G;
    for (int64_t i = blockIdx.x * kBlock + threadIdx.x; i < all; i += gridDim.x * kBlock) {
        const int grp = static_cast<int>(i / each), k = static_cast<int>(i % g.K);
        const int n = static_cast<int>(i / g.K % g.N);
        int lo = 0, hi = g.M;
        if (g.offsets) {
            lo = g.offsets[grp];
            hi = g.offsets[grp + 1];
            lo = lo < 0 ? 0 : lo > g.M ? g.M : lo;
            hi = hi < lo ? lo : hi > g.M ? g.M : hi;
        }
        float sum = 0.f;
        for (int m = lo; m < hi; ++m) {
            int r = m;
            if (g.index) r = g.index[m] < 0 ? -1 : g.index[m] / g.index_div;
            float v = 0.f;
            if (r >= 0 && r < g.x_rows)
                v = g.x_scale ? static_cast<float>(static_cast<const int8_t *>(g.x)[r * g.ldx + k]) *
                                    scale_step(g.x_scale[r * g.lds + k / UE_PACK_BLOCK])
                              : bf16_to_f32(static_cast<const uint16_t *>(g.x)[r * g.ldx + k]);
            sum = __builtin_fmaf(bf16_to_f32(g.dy[m * g.lddy + n]), v, sum);
        }
        float *p = g.out + grp * g.out_stride + n * g.ldo + k;
        *p = g.accumulate ? *p + sum : sum;
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

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED, bool INDEXED>
hipError_t wgrad_as(ue_ctx &c, const WgradArgs &g, hipStream_t s) {
    constexpr int BN = WN * FN * 32, BK = WK * FK * 32, kThreads = WN * WK * 64;
    constexpr int kLds = 2 * kRows * (BN + BK) * 2;
    // as many workgroups as fit at once: two waves per SIMD
    constexpr int kPerCu = 512 / kThreads;
    static_assert(BN == BK && kPerCu == per_cu(BN));
    const int64_t tn = (g.N + BN - 1) / BN, tk = (g.K + BK - 1) / BK, total = tn * tk * g.G * g.parts;
    const auto kernel = k_wgrad<FN, FK, WN, WK, WHOLE, PACKED, INDEXED>;
    if (kLds > 65536) {
        // once per kernel and device (a grant is the device's); one that fails is
        // asked for again by the next call
        static std::atomic<uint64_t> granted{0};
        const uint64_t bit = 1ull << (c.device & 63);
        if (c.device > 63 || !(granted.load(std::memory_order_relaxed) & bit)) {
            const hipError_t he = hipFuncSetAttribute(
                reinterpret_cast<const void *>(kernel),
                hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
            if (he != hipSuccess) return he;
            granted.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    const int64_t grid = total < kPerCu * c.num_cu ? total : kPerCu * c.num_cu;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid)), dim3(kThreads), kLds, s, g,
                       fast_div(INDEXED ? g.index_div : 1), static_cast<int>(tn),
                       static_cast<int>(tk));
    return hipGetLastError();
}

template <int FN, int FK, int WN, int WK, bool WHOLE, bool PACKED>
hipError_t wgrad_rows(ue_ctx &c, const WgradArgs &g, hipStream_t s) {
    return g.index ? wgrad_as<FN, FK, WN, WK, WHOLE, PACKED, true>(c, g, s)
                   : wgrad_as<FN, FK, WN, WK, WHOLE, PACKED, false>(c, g, s);
}

template <int FN, int FK, int WN, int WK>
hipError_t wgrad_any(ue_ctx &c, const WgradArgs &g, hipStream_t s) {
    const bool whole = g.vec_dy && g.N % 8 == 0 && (g.x_scale || (g.vec_x && g.K % 8 == 0));
    if (g.x_scale)
        return whole ? wgrad_rows<FN, FK, WN, WK, true, true>(c, g, s)
                     : wgrad_rows<FN, FK, WN, WK, false, true>(c, g, s);
    return whole ? wgrad_rows<FN, FK, WN, WK, true, false>(c, g, s)
                 : wgrad_rows<FN, FK, WN, WK, false, false>(c, g, s);
}

hipError_t wgrad_tiles(ue_ctx &c, const WgradArgs &g, hipStream_t s) {
    if (wgrad_tile(g.N, g.K, static_cast<int64_t>(g.G) * g.parts, c.num_cu) == kTile256)
        return wgrad_any<4, 2, 2, 4>(c, g, s);
    return wgrad_any<2, 2, 2, 2>(c, g, s);
}

}  // namespace

// As many as give every CU two tiles of 128.
int wgrad_parts(int M, int N, int K, int G, int num_cu) {
    const int64_t tiles = tiles_of(N, K, 128) * G;
    const int64_t slots = 2 * num_cu, rows = M / G;
    int64_t parts = slots / tiles;
    if (parts > rows / kPartRows) parts = rows / kPartRows;
    if (parts > kMaxParts) parts = kMaxParts;
    return parts > 1 ? static_cast<int>(parts) : 1;
}

bool wgrad_too_large(const WgradArgs &g, int num_cu) {
    if (g.M == 0 || wgrad_tiny(g)) return false;
    const int64_t mats = static_cast<int64_t>(g.G) * g.parts;
    const int tile = wgrad_tile(g.N, g.K, mats, num_cu) == kTile256 ? 256 : 128;
    // (a workgroup's next tile is a launch's workgroups on)
    return tiles_of(g.N, g.K, tile) * mats > 0x7FFFFFFF - per_cu(tile) * num_cu;
}

hipError_t launch_wgrad(ue_ctx &c, const WgradArgs &a, hipStream_t s) {
    if (a.N == 0 || a.K == 0 || a.G == 0) return hipSuccess;
    WgradArgs g = a;
    const int64_t rows = static_cast<int64_t>(g.G) * g.N, most = 64 * c.num_cu;
    const dim3 per_row(static_cast<uint32_t>(rows < most ? rows : most));
    if (g.M == 0) {
        if (g.accumulate) return hipSuccess;
        hipLaunchKernelGGL(k_wgrad_zero, per_row, dim3(kBlock), 0, s, g);
        return hipGetLastError();
    }
    if (wgrad_tiny(g)) {
        const int64_t blocks = (rows * g.K + kBlock - 1) / kBlock;
        hipLaunchKernelGGL(k_wgrad_tiny, dim3(static_cast<uint32_t>(blocks < most ? blocks : most)),
                           dim3(kBlock), 0, s, a);
        return hipGetLastError();
    }
    if (g.parts == 1) return wgrad_tiles(c, g, s);
    g.out = g.part;
    g.ldo = g.K;
    g.out_stride = static_cast<int64_t>(g.N) * g.K;
    g.accumulate = false;
    const hipError_t he = wgrad_tiles(c, g, s);
    if (he != hipSuccess) return he;
    tmark(&c, s);
    hipLaunchKernelGGL(k_wgrad_join, per_row, dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace ue
