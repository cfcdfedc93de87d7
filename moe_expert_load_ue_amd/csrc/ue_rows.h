// Streaming product of one wave: 16 rows of a matrix, read once from HBM
// straight into operand registers, against up to 64 rows of activations
// (tokens). Shared by the few-token layer and the 8-bit row kernel, whose time
// is the matrix's bytes.
//
// A matrix instruction takes 16 rows by 64 bytes of K, lane l the 16 bytes
// of row l mod 16 at piece g = l div 16. Loaded that way a wave touches 64
// bytes of 16 rows at a time, and such reads reach 4.9-5.6 TB/s here; loads of
// 128 bytes of 8 rows, or 256 bytes of 4, reach 6.8-6.9 (470 MB, rows of 14
// KiB, nontemporal). So a load takes LD = 2 or 4 pieces' worth of 16 / LD rows:
// lane l the row l mod (16 / LD) and the piece g + 4 b, b = (l mod 16) div
// (16 / LD). Two ways to multiply that:
// - FOLD = LD, for at most 16 / LD tokens: the load is an operand as it is.
//   Instruction row m and column c then hold different parts b of K, and only
//   results with equal parts mean anything: those of token t and row r are at
//   (b 16 / LD + r, b 16 / LD + t), and their sum over b is the product. The
//   tokens' operand is loaded the same way, once for the LD loads of a matrix.
// - FOLD = 1, for tiles of 16 tokens: two loads (LD = 2) swap the halves of
//   their rows of 16 lanes, one lane move per register, which gives operands
//   of 16 rows by each 64 bytes.
#pragma once

#include "ue_gate.h"

namespace ue {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Zeroes the bytes of a 16-byte piece from `left` on.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, int left) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int nb = left - 4 * w;
        v[w] &= nb >= 4 ? 0xFFFFFFFFu : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
    }
    return v;
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 w, u32x4 x, f32x4 c) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}

// Four int8 as bf16 (exact: 8 bits fit the significand).
__device__ __forceinline__ u32x2 widen4(uint32_t v) {
    const float f0 = static_cast<float>(static_cast<int8_t>(v));
    const float f1 = static_cast<float>(static_cast<int8_t>(v >> 8));
    const float f2 = static_cast<float>(static_cast<int8_t>(v >> 16));
    const float f3 = static_cast<float>(static_cast<int8_t>(v >> 24));
    // the low halves are zero: take the high ones
    return u32x2{__builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0),
                                       0x07060302u),
                 __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2),
                                       0x07060302u)};
}

// Kinds of operands. kEl: elements of the matrix in a 16-byte piece; kX:
// 16-byte pieces of activations that meet it.
struct Bf16Rows {            // bf16 matrix, bf16 activations
    static constexpr int kEl = 8, kX = 1, kXBytes = 2;
    typedef f32x4 Acc;
    static __device__ __forceinline__ void mul(u32x4 w, const u32x4 (&x)[1],
                                               Acc &acc) {
        acc = mfma_bf16(w, x[0], acc);
    }
};
struct WideRows {            // int8 matrix widened to bf16, bf16 activations
    static constexpr int kEl = 16, kX = 2, kXBytes = 2;
    typedef f32x4 Acc;
    static __device__ __forceinline__ void mul(u32x4 w, const u32x4 (&x)[2],
                                               Acc &acc) {
        const u32x2 a = widen4(w.x), b = widen4(w.y);
        const u32x2 c = widen4(w.z), d = widen4(w.w);
        acc = mfma_bf16(u32x4{a.x, a.y, b.x, b.y}, x[0], acc);
        acc = mfma_bf16(u32x4{c.x, c.y, d.x, d.y}, x[1], acc);
    }
};
struct I8Rows {              // int8 matrix, int8 activations
    static constexpr int kEl = 16, kX = 1, kXBytes = 1;
    typedef i32x4 Acc;
    static __device__ __forceinline__ void mul(u32x4 w, const u32x4 (&x)[1],
                                               Acc &acc) {
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            __builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x[0]), acc,
            0, 0, 0);
    }
};

// NW matrices; FOLD as above; RT tiles of 16 tokens (1 when folded); P parts
// each activation is the sum of; NJ: loads of a window that are made, so that
// the pass covers NJ 16 / LD rows (folded only; 0: all, 16 rows).
template <class Kind, int NW, int FOLD, int RT, int P, int NJ = 0>
struct RowStream {
    static_assert(FOLD == 1 || RT == 1, "folded products have one tile");
    static_assert(FOLD > 1 || NJ == 0, "two loads make the unfolded operands");
    static constexpr int kFold = FOLD == 1 ? 2 : FOLD;
    static constexpr int LD = NJ ? NJ : kFold;        // loads of a window
    static constexpr int kRows = 16 / kFold;          // rows of a load
    static constexpr int kAllRows = kRows * LD;       // rows of the pass
    static constexpr int kWindow = 4 * kFold * Kind::kEl;   // elements of K
    static constexpr int kTokens = FOLD == 1 ? 16 * RT : kRows;
    static constexpr int kAcc = FOLD == 1 ? RT : LD;  // results per matrix
    static constexpr int kXLoads = (FOLD == 1 ? 2 * RT : 1) * P * Kind::kX;
    // windows loaded together, within 80 registers (128 are a quarter of a
    // SIMD's)
    static constexpr int kRegs = 4 * (NW * LD + kXLoads);
    static constexpr int kAhead = kRegs > 40 ? 1 : kRegs < 20 ? 4 : 80 / kRegs;
    typedef typename Kind::Acc Acc;

    // The matrix row (of the pass) this lane reads in load j.
    static __device__ __forceinline__ int row(int j) {
        return j * kRows + (lane_id() & (kRows - 1));
    }
    // The token this lane holds: of tile r, or of the one folded tile.
    static __device__ __forceinline__ int token(int r) {
        return FOLD == 1 ? r * 16 + (lane_id() & 15) : (lane_id() & (kRows - 1));
    }

    // Matrix n's first row is at w[n], this lane's row of load j wo[j] bytes
    // on; part p of the activations at x[p], its token's row of tile r xo[r]
    // bytes on (bases are uniform: the offsets take 32 bits). K in [k0, k1),
    // k0 and k1 whole windows but for K itself; what lies past K is read from
    // the row's start and multiplied by zeros. (K a multiple of a piece for the bf16 kinds; for I8Rows any,
    // and rows readable to the end of their last piece.)
    static __device__ __forceinline__ void run(const char *const (&w)[NW],
                                               const uint32_t (&wo)[LD],
                                               const char *const (&x)[P],
                                               const uint32_t (&xo)[RT],
                                               int k0, int k1, int K,
                                               Acc (&acc)[NW][kAcc]) {
        constexpr int kEl = Kind::kEl, kX = Kind::kX;
        constexpr int kWBytes = 16 / kEl;      // of an element of the matrix
        const int g = lane_id() >> 4, l16 = lane_id() & 15;
        const int piece = g + 4 * (l16 / kRows);
        constexpr int kHalves = FOLD == 1 ? 2 : 1;
        const u32x4 zero = {0, 0, 0, 0};
        for (int k = k0; k < k1; k += kWindow * kAhead) {
            u32x4 wf[kAhead][NW][LD], xf[kAhead][RT][P][kHalves][kX];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int win = k + u * kWindow;
                const int at = win + piece * kEl;
                const uint32_t kw = win < k1 && at < K ? at : 0;
#pragma unroll
                for (int n = 0; n < NW; ++n)
#pragma unroll
                    for (int j = 0; j < LD; ++j)
                        wf[u][n][j] = __builtin_nontemporal_load(
                            reinterpret_cast<const u32x4 *>(
                                w[n] + (wo[j] + kw * kWBytes)));
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const int ax = FOLD == 1 ? win + (g + 4 * h) * kEl : at;
                    const uint32_t kx = win < k1 && ax < K ? ax : 0;
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int p = 0; p < P; ++p)
#pragma unroll
                            for (int i = 0; i < kX; ++i)
                                xf[u][r][p][h][i] = *reinterpret_cast<const u32x4 *>(
                                    x[p] + (xo[r] + kx * Kind::kXBytes + 16 * i));
                }
            }
            // (left alone, the compiler sinks the loads to their uses)
            __builtin_amdgcn_sched_barrier(0);
            if (k + kWindow * kAhead > k1 || k + kWindow * kAhead > K) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int win = k + u * kWindow;
                    const bool in = win < k1 && win + piece * kEl < K;
#pragma unroll
                    for (int n = 0; n < NW; ++n)
#pragma unroll
                        for (int j = 0; j < LD; ++j)
                            if (!in) wf[u][n][j] = zero;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        const int ax = FOLD == 1 ? win + (g + 4 * h) * kEl
                                                 : win + piece * kEl;
                        // whole pieces, but for 8-bit activations
                        const int left = win < k1 ? (K - ax) * Kind::kXBytes * kX : 0;
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int p = 0; p < P; ++p)
#pragma unroll
                                for (int i = 0; i < kX; ++i) {
                                    u32x4 &v = xf[u][r][p][h][i];
                                    if (Kind::kXBytes == 1) v = keep_bytes(v, left);
                                    else if (left <= 0) v = zero;
                                }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    if constexpr (FOLD > 1) {
#pragma unroll
                        for (int j = 0; j < LD; ++j)
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                Kind::mul(wf[u][n][j], xf[u][0][p][0], acc[n][j]);
                    } else {
                        u32x4 &a = wf[u][n][0], &b = wf[u][n][1];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            // a: rows 0-7, pieces g (lanes 0-7 of each row of
                            // 16) and g + 4; b: rows 8-15. Swap a's upper
                            // lanes with b's lower ones (row_ror:8 into half
                            // of the banks).
                            const uint32_t av = a[d], bv = b[d];
                            a[d] = __builtin_amdgcn_update_dpp(av, bv, 0x128, 0xF, 0xC, false);
                            b[d] = __builtin_amdgcn_update_dpp(bv, av, 0x128, 0xF, 0x3, false);
                        }
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int p = 0; p < P; ++p) {
                                Kind::mul(a, xf[u][r][p][0], acc[n][r]);
                                Kind::mul(b, xf[u][r][p][1], acc[n][r]);
                            }
                    }
                }
        }
    }

    // Where the result of matrix row n and token t lies, part b of kParts:
    // accumulator and index into its 64 lanes' four values.
    static constexpr int kParts = FOLD;
    static __device__ __forceinline__ void where(int n, int t, int b, int &a,
                                                 int &i) {
        if (FOLD == 1) {
            a = t >> 4;
            i = ((n >> 2) * 16 + (t & 15)) * 4 + (n & 3);
        } else {
            a = n / kRows;
            const int m = b * kRows + n % kRows;
            i = ((m >> 2) * 16 + b * kRows + t) * 4 + (m & 3);
        }
    }
};

}  // namespace ue
