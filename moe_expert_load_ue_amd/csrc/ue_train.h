// Internal declarations of the expert layer's training step: kernel arguments,
// launchers, packed rows, sums over the lanes that share a token.
#pragma once

#include "ue_gate.h"

#include <type_traits>

namespace ue {

// A launcher that starts several kernels one after another marks the end of each
// but the last (tmark); a kernel in several launches, for more rows than one's
// threads reach, is one.

struct BalanceArgs {
    const void *logits;         // [T] rows of E, ld elements apart
    int64_t ld;
    bool bf16, sigmoid;
    int E, k, T, n_seq;
    const int32_t *ids;
    const int32_t *offsets;     // [n_seq + 1] or null (one sequence)
    int32_t *counts;
    float *prob, *loss;
    int chunk;                  // tokens of a workgroup's share
    float *part;                // [slots][E up to 4 n] sums of p; slot: chunk + sequence;
                                // null: a workgroup per sequence, no partial sums
    int32_t *part_n;            // likewise: assignments
};
struct BalanceBackArgs {
    const void *logits;
    int64_t ld;
    bool bf16, sigmoid, accumulate;
    int E, k, T, n_seq;
    const int32_t *offsets, *counts;
    const float *dloss;
    void *dlogits;
    int64_t ld_out;
};
// Tokens of a workgroup's share, and the slots of partial sums that T tokens in
// n_seq sequences need (0: none are made).
int balance_chunk(int T, int E, int num_cu);
int64_t balance_slots(int T, int n_seq, int E, int num_cu);
hipError_t launch_balance(ue_ctx &c, const BalanceArgs &g, hipStream_t s);
hipError_t launch_balance_backward(const ue_ctx &c, const BalanceBackArgs &g,
                                   hipStream_t s);

// Rows and their packed form.
struct PackArgs {
    const void *x;
    void *out;                  // unpacking: where the values go
    int64_t ldx;
    bool bf16;
    int M, K;
    int8_t *q;
    const int8_t *q_in;
    int64_t ldq;
    uint8_t *scale;
    const uint8_t *scale_in;
    int64_t lds;
};
hipError_t launch_pack(const ue_ctx &c, const PackArgs &g, hipStream_t s);
hipError_t launch_unpack(const ue_ctx &c, const PackArgs &g, hipStream_t s);

struct GatedArgs {
    const void *gu;             // forward: [M] rows of 2 I
    const void *dh;             // backward: [M] rows of I
    int64_t ldin;
    bool bf16;
    int M, I;
    void *h;                    // may be null backward
    int64_t ldh;
    void *dgu;
    int64_t lddgu;
    int8_t *q;                  // may be null forward
    const int8_t *q_in;
    int64_t ldq;
    uint8_t *scale;
    const uint8_t *scale_in;
    int64_t lds;
};
hipError_t launch_gated(const ue_ctx &c, const GatedArgs &g, hipStream_t s);
hipError_t launch_gated_backward(const ue_ctx &c, const GatedArgs &g, hipStream_t s);

struct CombineArgs {
    const void *y;              // [rows] rows of H
    int64_t ldy;
    int rows;
    bool bf16;
    const int32_t *inv;
    const float *weights;       // or null (ones)
    int T, k, H;
    const void *add;            // or null
    int64_t ldadd;
    void *out;                  // forward
    int64_t ldo;
    const void *dout;           // backward
    int64_t lddout;
    void *dy;                   // or null
    int64_t lddy;
    float *dweights;            // or null
    uint32_t *named_by;         // [rows] notes of who names a row, or null
    uint32_t clear, all;        // set at launch: workgroups that clear rows of dy, and
                                // all assignments
};
hipError_t launch_combine(const ue_ctx &c, const CombineArgs &g, hipStream_t s);
// Whether rows that no assignment names are found with notes (4 bytes a row).
bool combine_notes(int T, int k, int rows);
// every_row: rows of dy that no assignment names are written too, with zeros.
hipError_t launch_combine_backward(ue_ctx &c, const CombineArgs &g, bool every_row,
                                   hipStream_t s);

struct WgradArgs {
    const uint16_t *dy;
    int64_t lddy;
    const void *x;
    int64_t ldx;
    const uint8_t *x_scale;
    int64_t lds;
    int x_rows;
    const int32_t *offsets;     // [G + 1] or null
    int G;
    const int32_t *index;       // [M] or null
    int index_div;
    int M, N, K;
    bool accumulate, vec_dy, vec_x;            // rows in 16-byte pieces
    float *out;
    int64_t ldo, out_stride;
    float *part;                // [parts][G][N][K] of a split sum, or null
    int parts;
};
// More tiles than the workgroups of a launch number with 31 bits.
bool wgrad_too_large(const WgradArgs &g, int num_cu);
hipError_t launch_wgrad(ue_ctx &c, const WgradArgs &g, hipStream_t s);
// Parts each group's rows are split into (1: no workspace).
int wgrad_parts(int M, int N, int K, int G, int num_cu);

// What a call reads is not kept in the caches where it is more than half of what
// the last of them holds (256 MB; the rest is for what the call writes): the sum of
// 25517 tokens' top-5 rows of 166, fp32, 85 MB, both ways 59 us through the caches
// and 77 past them, gated activation of 32768 rows of 2048, 268 MB, both ways 198
// and 193, 16384 tokens' top-8 rows of 7168, 1.9 GB, 1168 and 1100.
// f(type of the rows, past the caches).
template <class F>
void with_rows(bool bf16, int64_t bytes_read, F f) {
    const bool once = bytes_read > (int64_t(128) << 20);
    if (bf16) once ? f(uint16_t{}, std::true_type{}) : f(uint16_t{}, std::false_type{});
    else once ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
}

// ---------------------------------------------------------------------
// device helpers

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) { return bf16_to_f32(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) { return f32_to_bf16(v); }

// N elements, or those of them before `n`, at p, in loads and stores of up to 16
// bytes whatever p's alignment (the device takes any). ONCE: past the caches, as
// results go (gated activation of 32768 rows of 2048 with its backward pass 258 us
// with results through the caches, 198 past them; not the packed rows that
// ue_pack_rows makes, which a product reads next), and what a call reads where it is
// large (`with_rows`).
template <int BYTES>
struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(BYTES / 4), aligned(2)));
};
template <int N, bool ONCE, typename T>
__device__ __forceinline__ void load_run(const T *p, int n, float (&f)[N]) {
    constexpr int kBytes = N * sizeof(T), kPiece = kBytes < 16 ? kBytes : 16;
    typedef typename Words<kPiece>::type W;
    if (n >= N) {
        struct Pack { W v[kBytes / kPiece]; } k;
#pragma unroll
        for (int c = 0; c < kBytes / kPiece; ++c) {
            const W *at = reinterpret_cast<const W *>(p) + c;
            k.v[c] = ONCE ? __builtin_nontemporal_load(at) : *at;
        }
        struct Elements { T v[N]; };
        const Elements e = __builtin_bit_cast(Elements, k);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = widen<T>(e.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = i < n ? widen<T>(p[i]) : 0.f;
    }
}
template <int N, bool ONCE, typename T>
__device__ __forceinline__ void store_run(T *p, int n, const float (&f)[N]) {
    constexpr int kBytes = N * sizeof(T), kPiece = kBytes < 16 ? kBytes : 16;
    typedef typename Words<kPiece>::type W;
    if (n >= N) {
        struct Elements { T v[N]; } e;
#pragma unroll
        for (int i = 0; i < N; ++i) e.v[i] = narrow<T>(f[i]);
        struct Pack { W v[kBytes / kPiece]; };
        const Pack k = __builtin_bit_cast(Pack, e);
#pragma unroll
        for (int c = 0; c < kBytes / kPiece; ++c) {
            W *at = reinterpret_cast<W *>(p) + c;
            if (ONCE) __builtin_nontemporal_store(k.v[c], at);
            else *at = k.v[c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = narrow<T>(f[i]);
    }
}
template <bool ONCE, typename T>
__device__ __forceinline__ void load8(const T *p, int n, float (&f)[8]) {
    load_run<8, ONCE>(p, n, f);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float (&f)[8]) {
    store_run<8, true>(p, n, f);
}

// The power of two of a block whose largest magnitude has these bits, biased
// by 127: its exponent less 6, one more above 127/64 of its power of two, and
// at least 1 (so that it and its inverse are normal numbers); at most 248, whose
// 127-fold is still a float (64 times the next one is 2^128); 255 for a block that
// holds an infinity or a NaN.
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    uint32_t e = (top + 0x1FFFFu) >> 23;
    e = e < 254u ? e : 254u;
    return e > 7u ? e - 6u : 1u;
}
// 2^e, infinity for 255 (which q = 0 turns into the block's NaNs).
__device__ __forceinline__ float scale_step(uint32_t s) { return __uint_as_float(s << 23); }
// 2^-e, 0 for 255.
__device__ __forceinline__ float scale_inverse(uint32_t s) {
    return s >= 254u ? 0.f : __uint_as_float((254u - s) << 23);
}

// Largest of four lanes' values (the lanes of one block).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t o = __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false);
    v = o > v ? o : v;
    o = __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false);
    return o > v ? o : v;
}

// Eight elements of this lane's part of a block (four lanes) as integers;
// returns the block's scale.
__device__ __forceinline__ uint32_t pack8(const float (&f)[8], uint64_t &q) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(f[i]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
    }
    const uint32_t s = block_scale(quad_max(top));
    const float inv = scale_inverse(s);
    union { int8_t b[8]; uint64_t w; } u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (up to 128 steps where they are the largest)
        const float r = __builtin_amdgcn_fmed3f(rintf(f[i] * inv), -127.f, 127.f);
        u.b[i] = static_cast<int8_t>(s == 255u ? 0 : static_cast<int>(r));
    }
    q = u.w;
    return s;
}
__device__ __forceinline__ void unpack8(uint64_t q, uint32_t s, float (&f)[8]) {
    const float step = scale_step(s);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = static_cast<float>(static_cast<int8_t>(q >> (8 * i))) * step;
}

// Quotients of numbers below 2^31 by a divisor fixed on the host: a high
// product, a sum and a shift.
struct FastDiv {
    uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint32_t m = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    return FastDiv{d, m, l};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
    return (__umulhi(n, f.mul) + n) >> f.shift;
}

template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(
        __float_as_uint(v), __float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// Of lane i's value and that of lane i + 16 (i + 32), or i - 16 (i - 32): both, in
// either order. (Swaps of vector registers: through LDS's permutes the balance
// loss of 65536 tokens of 256 experts took 29 us in place of 27, forward.)
struct Both { float a, b; };
__device__ __forceinline__ Both across16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v),
                                                    false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Both across32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v),
                                                    false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
// Sum over the lanes with the same lane % L.
template <int L>
__device__ __forceinline__ float sum_across(float v) {
    static_assert(L == 8 || L == 16 || L == 32 || L == 64);
    if (L <= 8) v += lane_move<0x128>(v);            // by 8 round a row of 16
    if (L <= 16) { const Both o = across16(v); v = o.a + o.b; }
    if (L <= 32) { const Both o = across32(v); v = o.a + o.b; }
    return v;
}

// Sum and maximum over L consecutive lanes, the same in each: inside a row of
// 16 by lane moves (pairs, halves of four, mirrored eights and sixteens),
// beyond it by exchange.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    if (L > 1) v += lane_move<0xB1>(v);
    if (L > 2) v += lane_move<0x4E>(v);
    if (L > 4) v += lane_move<0x141>(v);
    if (L > 8) v += lane_move<0x140>(v);
    if (L > 16) { const Both o = across16(v); v = o.a + o.b; }
    if (L > 32) { const Both o = across32(v); v = o.a + o.b; }
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    if (L > 1) v = fmaxf(v, lane_move<0xB1>(v));
    if (L > 2) v = fmaxf(v, lane_move<0x4E>(v));
    if (L > 4) v = fmaxf(v, lane_move<0x141>(v));
    if (L > 8) v = fmaxf(v, lane_move<0x140>(v));
    if (L > 16) { const Both o = across16(v); v = fmaxf(o.a, o.b); }
    if (L > 32) { const Both o = across32(v); v = fmaxf(o.a, o.b); }
    return v;
}

}  // namespace ue
