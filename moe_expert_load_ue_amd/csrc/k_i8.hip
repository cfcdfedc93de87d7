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
//
// Bound: for large products the matrix units at the clock that the power
// limit leaves them. 8192x7168x4096: 196-225 us (2.1-2.5 POP/s) on random data,
// 166 on zeros, which draw less power; the library's product, without scales,
// in turn with it 204-235 and 141. Matrix units busy 64% of the cycles, no LDS
// bank conflicts. With groups, the last row tile of each (23% of the rows of
// 256-row tiles are empty at 263-939 rows a group, 13% of 128-row tiles) and
// the rounds of tiles over the CUs: gated 32768x4096x2048 in 72 uneven groups
// 403 us (128-row tiles), and with 256-row tiles 306 in 64 even groups, 250 in
// four, 238 without groups.
#include <type_traits>

#include "ue_rows.h"
#include "ue_tiles.h"

namespace ue {
namespace {

constexpr int kStep = 128;               // bytes of K per stage

// Waits until at most N of this wave's loads are on their way and its LDS
// reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// The tile of a workgroup: rows [lo, hi) of a group, channels from n0.
struct Tile {
    int mat, lo, hi, col;               // mat: the matrix its group uses
};

// Group g has ceil(rows / BM) row tiles, groups in order; offsets are clamped
// to [0, M], so that no table can send a tile outside. The launch has room
// for any table; how many tiles there are is counted here, and only those are
// dealt to the XCDs. Tiles go in blocks of kBlockM row tiles by all column
// tiles, row tiles first, each XCD a contiguous run: the tiles an XCD has at
// once then share both operands' rows in its L2. False: no tile left.
constexpr int kBlockM = 4;
template <int THREADS>
__device__ __forceinline__ bool find_tile(const I8Args &g, int BM, int ncol,
                                          int *sh, Tile &t) {
    const int tid = threadIdx.x;
    const int per = (g.G + THREADS - 1) / THREADS;
    const int first = tid * per;
    auto bounds = [&](int i, int &a, int &b) {
        a = g.offsets[i];
        b = g.offsets[i + 1];
        a = a < 0 ? 0 : a > g.M ? g.M : a;
        b = b < a ? a : b > g.M ? g.M : b;
    };
    int n = 0, before = 0, rows = (g.M + BM - 1) / BM, a1 = 0, b1 = 0, mat = first;
    if (g.offsets) {
        // (the common case of a group per thread reads everything at once)
        if (first < g.G) {
            if (g.expert_of) mat = g.expert_of[first];
            bounds(first, a1, b1);
            n = (b1 - a1 + BM - 1) / BM;
        }
        for (int i = first + 1; i < first + per && i < g.G; ++i) {
            int a, b;
            bounds(i, a, b);
            n += (b - a + BM - 1) / BM;
        }
        // tiles before this thread's groups, and of all
        const int incl = wave_inclusive_sum(n);
        if (lane_id() == 63) sh[tid >> 6] = incl;
        __syncthreads();
        before = incl - n;
        rows = 0;
        for (int w = 0; w < THREADS / 64; ++w) {
            before += w < (tid >> 6) ? sh[w] : 0;
            rows += sh[w];
        }
    }
    // (a table whose groups overlap may ask for more tiles than there is room)
    const int room = gridDim.x / ncol;
    rows = rows < room ? rows : room;
    if (static_cast<int>(blockIdx.x) >= rows * ncol) return false;
    const int id = xcd_order(blockIdx.x, rows * ncol);
    const int blk = id / (kBlockM * ncol), in = id - blk * kBlockM * ncol;
    const int bm = rows - blk * kBlockM < kBlockM ? rows - blk * kBlockM : kBlockM;
    t.col = in / bm;
    const int tile = blk * kBlockM + in % bm;
    if (!g.offsets) {
        t.mat = 0;
        t.lo = tile * BM;
        t.hi = g.M;
        return true;
    }
    if (tile >= before && tile < before + n) {
        int left = tile - before, i = first, a = a1, b = b1;
        for (int nt; left >= (nt = (b - a + BM - 1) / BM); left -= nt) {
            ++i;
            bounds(i, a, b);
        }
        sh[16] = i == first ? mat : g.expert_of ? g.expert_of[i] : i;
        sh[17] = a + left * BM;
        sh[18] = b;
    }
    __syncthreads();
    t.mat = sh[16];
    t.lo = sh[17];
    t.hi = sh[18];
    return true;
}

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) {
    *p = f32_to_bf16(v);
}

// N consecutive results: 16 bytes at a time (or all of them, if that is
// less) when `whole`, else those of the first `left` one by one.
template <int N, typename OUT>
__device__ __forceinline__ void store_run(OUT *p, const float (&v)[N], bool whole,
                                          int left) {
    constexpr int kBytes = N * static_cast<int>(sizeof(OUT));
    constexpr int kEach = kBytes < 16 ? N : 16 / static_cast<int>(sizeof(OUT));
    if (whole) {
        struct alignas(kBytes < 16 ? kBytes : 16) Pack { OUT o[kEach]; };
#pragma unroll
        for (int c = 0; c < N; c += kEach) {
            Pack k;
#pragma unroll
            for (int e = 0; e < kEach; ++e) store_out(&k.o[e], v[c + e]);
            *reinterpret_cast<Pack *>(p + c) = k;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) store_out(p + e, v[e]);
    }
}

// The row of activations of output row m (-1: none).
__device__ __forceinline__ int act_row(const I8Args &g, int m) {
    if (!g.index) return m;
    const int i = g.index[m];
    if (i < 0) return -1;
    const int r = i / g.index_div;
    return r < g.a_rows ? r : -1;
}

// FM, FN: 16-row fragments of activations and of the matrix per wave;
// WM, WN: waves along each; NS: stages in LDS.
//
// A stage is two halves of 64 bytes of K. While a half's products run, the
// operands of the next half are on their way from LDS. At the end of a
// stage's first half its second half has been read, so the stage's LDS is
// free: one barrier there tells that every wave is done with it and that the
// next stage has landed, and the stage NS ahead is loaded into it.
template <int FM, int FN, int WM, int WN, int NS, bool GATED, typename OUT,
          typename OFF>
__global__ __launch_bounds__(WM *WN * 64, FM * FN > 32 ? 1 : 2) void k_matmul_i8(I8Args g) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int BM = WM * FM * 16, BN = WN * FN * 16;   // rows in LDS
    constexpr int kOut = GATED ? BN / 2 : BN;             // channels out
    constexpr int kChunks = (BM + BN) / 8 / (WM * WN);    // of 8 rows, a wave
    constexpr int kStage = (BM + BN) * kStep;
    static_assert((BM + BN) / 8 % (WM * WN) == 0, "whole chunks per wave");
    extern __shared__ __align__(16) char lds[];
    __shared__ int sh[20];
    __shared__ float tile_scale[BM + BN];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);

    Tile tile;
    if (!find_tile<kThreads>(g, BM, (g.N + kOut - 1) / kOut, sh, tile)) return;
    const int m0 = __builtin_amdgcn_readfirstlane(tile.lo);
    const int m_end = __builtin_amdgcn_readfirstlane(tile.hi);
    const int n0 = tile.col * kOut;
    const int mat = __builtin_amdgcn_readfirstlane(tile.mat);
    if (static_cast<uint32_t>(mat) >= static_cast<uint32_t>(g.n_mats)) return;

    // offset of this lane's piece of each chunk it loads, from the matrix or
    // the activations (without an index, from the tile's first row)
    const int8_t *const abase = g.index ? g.a : g.a + static_cast<int64_t>(m0) * g.lda;
    const int8_t *const wbase = g.w + mat * g.w_stride;
    OFF src[kChunks];
    const int piece = (lane & 7) ^ (lane >> 3);     // row & 7 = lane >> 3
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int r = (wv * kChunks + c) * 8 + (lane >> 3);
        if (r < BM) {
            int m = m0 + r;
            m = m < m_end ? m : m_end - 1;
            const int a = g.index ? act_row(g, m) : m - m0;
            src[c] = static_cast<OFF>(a < 0 ? 0 : a) * static_cast<OFF>(g.lda);
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
            src[c] = static_cast<OFF>(n) * static_cast<OFF>(g.ldw);
        }
        src[c] += piece * 16;
    }
    const int kbytes = (g.K + 15) & ~15;
    const int steps = (g.K + kStep - 1) / kStep;
    // one chunk of the stage at k0, into the LDS of stage `buf`
    auto load_chunk = [&](int c, int buf, int k0) {
        // pieces past the row's end are read from its start: the last
        // stage's products mask them
        const OFF k = static_cast<OFF>(k0 + piece * 16 < kbytes ? k0 : -piece * 16);
        const int8_t *from = ((wv * kChunks + c) * 8 < BM ? abase : wbase) +
                             static_cast<OFF>(src[c] + k);
        char *to = lds + buf * kStage + (wv * kChunks + c) * 8 * kStep;
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void *)from,
            (__attribute__((address_space(3))) void *)to, 16, 0, 0);
    };

    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int wm = wv / WN, wn = wv % WN;
    const int q = lane >> 4, l16 = lane & 15;
    // rows of this lane's operand reads, and its pieces of the two halves
    const int arow = wm * FM * 16 + l16;
    const int brow = wn * FN * 16 + l16;
    const char *la = lds + arow * kStep, *lb = lds + (BM + brow) * kStep;
    struct Half { i32x4 a[FM], b[FN]; };
    // operand read t of half h: the matrix's fragments, then the activations'
    auto read_part = [&](Half &f, int t, int buf, int h) {
        const int at = buf * kStage + (((h * 4 + q) ^ (l16 & 7)) << 4);
        if (t < FN)
            f.b[t] = *reinterpret_cast<const i32x4 *>(lb + at + t * 16 * kStep);
        else
            f.a[t - FN] = *reinterpret_cast<const i32x4 *>(la + at + (t - FN) * 16 * kStep);
    };
    // The products of one half, with `tasks` calls of work(t) spread between
    // them: a wave issues in order, so loads issued in one go would hold the
    // matrix instructions behind them until the memory pipes have taken them
    // all.
    auto products = [&](Half &f, auto tasks, auto work) {
        constexpr int kTasks = decltype(tasks)::value, kAll = FM * FN;
        int done = 0;
#pragma unroll
        for (int p = 0; p < kAll; ++p) {
#pragma unroll
            for (; done < kTasks && done * kAll < p * kTasks; ++done) work(done);
            __builtin_amdgcn_sched_barrier(0);
            const int i = p / FN, j = p % FN;
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                f.b[j], f.a[i], acc[i][j], 0, 0, 0);
        }
#pragma unroll
        for (; done < kTasks; ++done) work(done);
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kReads = FM + FN;
    typedef std::integral_constant<int, kReads> Reads;
    typedef std::integral_constant<int, kReads + kChunks> ReadsAndLoads;
    typedef std::integral_constant<int, 0> None;

    // The scales of the tile's rows and channels (gated: the gate channels',
    // then the up channels'), on their way before the stages: in order, so
    // that no wait is for them. They go to LDS behind the last products.
    constexpr int kScales = (BM + BN + kThreads - 1) / kThreads;
    float scale[kScales];
    const float *ws = g.w_scale + mat * g.ws_stride;
#pragma unroll
    for (int c = 0; c < kScales; ++c) {
        const int i = c * kThreads + tid, j = i - BM;
        if (i < BM) {
            const int ar = m0 + i < m_end ? act_row(g, m0 + i) : -1;
            scale[c] = ar < 0 ? 0.f : g.a_scale[ar];
        } else {
            const int n = n0 + j % kOut;
            scale[c] = ws[(n < g.N ? n : g.N - 1) + (j < kOut || !GATED ? 0 : g.N)];
        }
    }
    for (int s = 0; s < NS && s < steps; ++s)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) load_chunk(c, s, s * kStep);
    // every stage but the first may still be on its way
    if (steps >= NS) wait_loads<(NS - 1) * kChunks>();
    else wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    Half f0, f1;
#pragma unroll
    for (int t = 0; t < kReads; ++t) read_part(f0, t, 0, 0);
    int buf = 0, st = 0;
    // all stages but the last NS load ahead, the next ones only use what was
    // loaded, the last one masks what lies past K
    auto stage = [&](auto loads) {
        constexpr bool kLoads = decltype(loads)::value;
        products(f0, Reads{}, [&](int t) { read_part(f1, t, buf, 1); });
        wait_loads<kLoads ? (NS - 2) * kChunks : 0>();
        __builtin_amdgcn_s_barrier();
        const int old = buf;
        buf = buf + 1 == NS ? 0 : buf + 1;
        if constexpr (kLoads)
            products(f1, ReadsAndLoads{}, [&](int t) {
                if (t < kReads) read_part(f0, t, buf, 0);
                else load_chunk(t - kReads, old, (st + NS) * kStep);
            });
        else
            products(f1, Reads{}, [&](int t) { read_part(f0, t, buf, 0); });
    };
    for (; st + NS < steps; ++st) stage(std::true_type{});
    for (; st + 1 < steps; ++st) stage(std::false_type{});
#pragma unroll
    for (int t = 0; t < kReads; ++t) read_part(f1, t, buf, 1);
    auto mask_half = [&](Half &f, int k0) {
        const int left = g.K - (k0 + q * 16);
#pragma unroll
        for (int i = 0; i < FM; ++i)
            f.a[i] = __builtin_bit_cast(
                i32x4, keep_bytes(__builtin_bit_cast(u32x4, f.a[i]), left));
    };
    mask_half(f0, st * kStep);
    mask_half(f1, st * kStep + 64);
    products(f0, None{}, [](int) {});
    products(f1, None{}, [](int) {});

#pragma unroll
    for (int c = 0; c < kScales; ++c)
        if (c * kThreads + tid < BM + BN) tile_scale[c * kThreads + tid] = scale[c];
    __syncthreads();
    const float *row_scale = tile_scale, *col_scale = tile_scale + BM;
    constexpr int kRun = GATED ? FN * 2 : FN * 4;   // channels a lane holds
    const int at = wn * kRun * 4 + kRun * q, nb = n0 + at;
    float sw[kRun], su[kRun];
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
        sw[e] = col_scale[at + e];
        if (GATED) su[e] = col_scale[kOut + at + e];
    }
    const bool whole = g.vec_out && nb + kRun <= g.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + arow + i * 16;
        if (m >= m_end) continue;
        const float sa = row_scale[arow + i * 16];
        float v[kRun];
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            if (GATED) {
                const float gt = static_cast<float>(acc[i][e / 4 * 2][e % 4]) * sa * sw[e];
                const float up = static_cast<float>(acc[i][e / 4 * 2 + 1][e % 4]) * sa * su[e];
                v[e] = silu_of(gt) * up;
            } else {
                v[e] = static_cast<float>(acc[i][e / 4][e % 4]) * sa * sw[e];
            }
        }
        store_run<kRun>(static_cast<OUT *>(g.out) + static_cast<int64_t>(m) * g.ldo + nb,
                        v, whole, g.N - nb);
    }
}

// Up to 16 rows: the matrix's bytes bound the product. 16 channels (and their
// 16 up channels) per workgroup, K split over its waves, each streaming its
// part of the matrix from HBM straight into its operand registers (ue_rows.h).
// One row, 7168x4096: 6.6 us (29.4 MB, 4.4 TB/s; an empty launch takes 2).
constexpr int kRowWaves = 8;

template <int FOLD, bool GATED, typename OUT>
__global__ __launch_bounds__(kRowWaves * 64) void k_rows_i8(I8Args g) {
    constexpr int NW = GATED ? 2 : 1;
    typedef RowStream<I8Rows, NW, FOLD, 1, 1> S;
    __shared__ i32x4 part[kRowWaves][NW][S::kAcc][64];
    const int tid = threadIdx.x, lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16, group = blockIdx.y;
    int lo = 0, hi = g.M;
    if (g.offsets) {
        lo = g.offsets[group];
        hi = g.offsets[group + 1];
        lo = lo < 0 ? 0 : lo > g.M ? g.M : lo;
        hi = hi < lo ? lo : hi > g.M ? g.M : hi;
    }
    if (lo >= hi) return;
    const int mat = g.expert_of ? g.expert_of[group] : group;
    if (static_cast<uint32_t>(mat) >= static_cast<uint32_t>(g.n_mats)) return;
    // (hi - lo <= M <= the tokens FOLD holds)
    const int m = lo + S::token(0), row = act_row(g, m < hi ? m : hi - 1);
    const char *w[NW], *x[1] = {reinterpret_cast<const char *>(g.a)};
    uint32_t wo[S::LD], xo[1] = {static_cast<uint32_t>(row < 0 ? 0 : row) *
                                 static_cast<uint32_t>(g.lda)};
#pragma unroll
    for (int c = 0; c < NW; ++c)
        w[c] = reinterpret_cast<const char *>(
            g.w + mat * g.w_stride + static_cast<int64_t>(c) * g.N * g.ldw);
#pragma unroll
    for (int j = 0; j < S::LD; ++j) {
        const int n = n0 + S::row(j) < g.N ? n0 + S::row(j) : g.N - 1;
        wo[j] = static_cast<uint32_t>(n) * static_cast<uint32_t>(g.ldw);
    }
    // this wave's part of K, in whole windows
    const int windows = (g.K + S::kWindow - 1) / S::kWindow;
    const int per = (windows + kRowWaves - 1) / kRowWaves;
    const int w0 = wv * per, w1 = w0 + per < windows ? w0 + per : windows;
    i32x4 acc[NW][S::kAcc] = {};
    S::run(w, wo, x, xo, w0 * S::kWindow, w1 * S::kWindow, g.K, acc);
#pragma unroll
    for (int c = 0; c < NW; ++c)
#pragma unroll
        for (int r = 0; r < S::kAcc; ++r) part[wv][c][r][lane] = acc[c][r];
    __syncthreads();
    const int *sums = reinterpret_cast<const int *>(part);
    const float *ws = g.w_scale + mat * g.ws_stride;
    for (int i = tid; i < 16 * (hi - lo); i += kRowWaves * 64) {
        const int nn = i & 15, t = i >> 4, n = n0 + nn;
        if (n >= g.N) continue;
        int v[NW] = {};
#pragma unroll
        for (int c = 0; c < NW; ++c)
            for (int u = 0; u < kRowWaves; ++u)
#pragma unroll
                for (int b = 0; b < S::kParts; ++b) {
                    int a, at;
                    S::where(nn, t, b, a, at);
                    v[c] += sums[((u * NW + c) * S::kAcc + a) * 256 + at];
                }
        const int ar = act_row(g, lo + t);
        const float sa = ar < 0 ? 0.f : g.a_scale[ar];
        float y = static_cast<float>(v[0]) * sa * ws[n];
        if constexpr (GATED) {
            const float up = static_cast<float>(v[1]) * sa * ws[g.N + n];
            y = silu_of(y) * up;
        }
        store_out(static_cast<OUT *>(g.out) + static_cast<int64_t>(lo + t) * g.ldo + n, y);
    }
}

template <int FOLD, bool GATED, typename OUT>
hipError_t rows_as(const I8Args &g, hipStream_t s) {
    static_assert(i8_tile(kI8Rows).bn == 16 && i8_tile(kI8Rows).threads == kRowWaves * 64);
    hipLaunchKernelGGL((k_rows_i8<FOLD, GATED, OUT>), dim3((g.N + 15) / 16, g.G),
                       dim3(kRowWaves * 64), 0, s, g);
    return hipGetLastError();
}

template <int FOLD>
hipError_t rows(const I8Args &g, hipStream_t s) {
    if (g.gated)
        return g.out_f32 ? rows_as<FOLD, true, float>(g, s)
                         : rows_as<FOLD, true, uint16_t>(g, s);
    return g.out_f32 ? rows_as<FOLD, false, float>(g, s)
                     : rows_as<FOLD, false, uint16_t>(g, s);
}

template <I8Kernel KIND, int FM, int FN, int WM, int WN, int NS, bool GATED,
          typename OUT, typename OFF>
hipError_t tiled_as(ue_ctx &c, const I8Args &g, int64_t workgroups, hipStream_t s) {
    constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
    static_assert(i8_tile(KIND).bm == BM && i8_tile(KIND).bn == BN &&
                  i8_tile(KIND).threads == WM * WN * 64);
    static_assert(KIND * 4 + 3 < 32, "a bit for every kernel");
    constexpr int kLds = NS * (BM + BN) * kStep;
    const auto kernel = k_matmul_i8<FM, FN, WM, WN, NS, GATED, OUT, OFF>;
    if constexpr (kLds > 65536) {
        // once per kernel and context (a grant is the device's, and a context
        // belongs to one): the need is a constant. One that fails is asked for
        // again by the next call.
        const uint32_t bit = 1u << (KIND * 4 + GATED * 2 + (sizeof(OUT) == 4));
        if (!(c.i8_granted & bit)) {
            const hipError_t he = hipFuncSetAttribute(
                reinterpret_cast<const void *>(kernel),
                hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
            if (he != hipSuccess) return he;
            c.i8_granted |= bit;
        }
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(workgroups)),
                       dim3(WM * WN * 64), kLds, s, g);
    return hipGetLastError();
}

template <I8Kernel KIND, int FM, int FN, int WM, int WN, int NS, typename OFF = uint32_t>
hipError_t tiled(ue_ctx &c, const I8Args &g, int64_t n, hipStream_t s) {
    if (g.gated)
        return g.out_f32 ? tiled_as<KIND, FM, FN, WM, WN, NS, true, float, OFF>(c, g, n, s)
                         : tiled_as<KIND, FM, FN, WM, WN, NS, true, uint16_t, OFF>(c, g, n, s);
    return g.out_f32 ? tiled_as<KIND, FM, FN, WM, WN, NS, false, float, OFF>(c, g, n, s)
                     : tiled_as<KIND, FM, FN, WM, WN, NS, false, uint16_t, OFF>(c, g, n, s);
}

}  // namespace

hipError_t launch_matmul_i8(ue_ctx &c, const I8Args &g, hipStream_t s,
                            bool &too_large) {
    too_large = false;
    if (g.M == 0 || g.N == 0) return hipSuccess;
    // offsets of an indexed row past 32 bits: one kernel has them in 64
    const int64_t reach = static_cast<int64_t>(g.index ? g.a_rows : g.M) * g.lda;
    const I8Size z{g.M, g.N, g.K, g.G, g.gated, g.offsets != nullptr,
                   g.index && reach > 0xFFFFFFFFll, c.num_cu};
    const I8Kernel kind = i8_kernel(z);
    const int64_t n = i8_workgroups(kind, z);
    if (n * i8_tile(kind).threads > kLaunchThreads) {
        too_large = true;
        return hipSuccess;
    }
    switch (kind) {
        case kI8Rows:
            return g.M <= 4 ? rows<4>(g, s) : g.M <= 8 ? rows<2>(g, s) : rows<1>(g, s);
        case kI8Wide: return tiled<kI8Wide, 2, 2, 2, 2, 4, uint64_t>(c, g, n, s);
        case kI8Tall: return tiled<kI8Tall, 8, 4, 2, 4, 2>(c, g, n, s);
        case kI8Deep: return tiled<kI8Deep, 4, 4, 2, 4, 3>(c, g, n, s);
        case kI8Mid: return tiled<kI8Mid, 4, 2, 2, 4, 2>(c, g, n, s);
        case kI8Small: return tiled<kI8Small, 2, 2, 2, 2, 4>(c, g, n, s);
        case kI8Least: break;
    }
    return tiled<kI8Least, 1, 2, 2, 2, 6>(c, g, n, s);
}

}  // namespace ue
