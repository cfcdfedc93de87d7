// Activations kept in 8 bits: rows to packed rows and back (ue_pack_rows,
// ue_unpack_rows), and the gated activation with its backward pass on packed
// rows (ue_gated, ue_gated_backward).
//
// A block is 32 columns of a row with one power of two, so that rounding is
// the only loss: quotients by it are exact, ties go to even whatever computes
// them, and q 2^e is a bf16 number that a matrix instruction takes as it is.
// Four lanes hold a block, eight elements each; the largest magnitude goes
// round them by two lane moves. The blocks of all rows are one list, so rows of
// any length fill the waves.
//
// Bound: HBM. 32768 rows of 2048, bf16: gated activation, keeping gate and up, 87
// us (541 MB, 6.2 TB/s), its backward pass with the activation again 107 us (675
// MB, 6.3 TB/s), one after the other 194; in short runs with pauses 113 and 111 at
// the median. 4096 rows of 7168 packed in 17-19 us (89 MB), calls for 8192 29 us (178
// MB, 6.1 TB/s) and back to bf16 27, to fp32 87 (294 MB, 3.4 TB/s). A quad of lanes takes one block and no loop: what is in
// flight is other waves'. 13358 rows of 302, fp32, both ways 27 us (element by
// element, as rows that are no multiple of 16 bytes were read once, 68; past the
// caches what is read 35).
#include "ue_train.h"

namespace ue {
namespace {

// Blocks of one launch are numbered below 2^30 (quads of lanes: fewer than
// 2^32 threads; FastDiv takes numbers below 2^31).
constexpr int64_t kLaunchBlocks = int64_t(1) << 29;

template <typename T, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_pack(PackArgs g, FastDiv per_row, uint32_t blocks) {
    const uint32_t b = blockIdx.x * (kBlock / 4) + (threadIdx.x >> 2);
    if (b >= blocks) return;                       // (whole quads)
    const uint32_t m = div_by(b, per_row), c = b - m * per_row.d;
    const int k = c * UE_PACK_BLOCK + (threadIdx.x & 3) * 8;
    float f[8];
    load8<ONCE>(static_cast<const T *>(g.x) + m * g.ldx + k, g.K - k, f);
    uint64_t q;
    const uint32_t s = pack8(f, q);
    *reinterpret_cast<uint64_t *>(g.q + m * g.ldq + k) = q;
    if ((threadIdx.x & 3) == 0) g.scale[m * g.lds + c] = static_cast<uint8_t>(s);
}

template <typename T>
__global__ __launch_bounds__(kBlock) void k_unpack(PackArgs g, FastDiv per_row, uint32_t blocks) {
    const uint32_t b = blockIdx.x * (kBlock / 4) + (threadIdx.x >> 2);
    if (b >= blocks) return;
    const uint32_t m = div_by(b, per_row), c = b - m * per_row.d;
    const int k = c * UE_PACK_BLOCK + (threadIdx.x & 3) * 8;
    const uint64_t q = *reinterpret_cast<const uint64_t *>(g.q_in + m * g.ldq + k);
    float f[8];
    unpack8(q, g.scale_in[m * g.lds + c], f);
    store8<T>(static_cast<T *>(g.out) + m * g.ldx + k, g.K - k, f);
}

template <typename T, bool KEEP, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_gated(GatedArgs g, FastDiv per_row, uint32_t blocks) {
    const uint32_t b = blockIdx.x * (kBlock / 4) + (threadIdx.x >> 2);
    if (b >= blocks) return;
    const uint32_t m = div_by(b, per_row), c = b - m * per_row.d;
    const int k = c * UE_PACK_BLOCK + (threadIdx.x & 3) * 8;
    const T *row = static_cast<const T *>(g.gu) + m * g.ldin + k;
    float gate[8], up[8], h[8];
    load8<ONCE>(row, g.I - k, gate);
    load8<ONCE>(row + g.I, g.I - k, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = silu_of(gate[i]) * up[i];
    store8<T>(static_cast<T *>(g.h) + m * g.ldh + k, g.I - k, h);
    if (KEEP) {
        uint64_t q;
        int8_t *to = g.q + m * g.ldq + k;
        uint8_t *st = g.scale + m * g.lds + c;
        uint32_t s = pack8(gate, q);
        __builtin_nontemporal_store(q, reinterpret_cast<uint64_t *>(to));
        if ((threadIdx.x & 3) == 0) st[0] = static_cast<uint8_t>(s);
        s = pack8(up, q);
        __builtin_nontemporal_store(
            q, reinterpret_cast<uint64_t *>(to + per_row.d * UE_PACK_BLOCK));
        if ((threadIdx.x & 3) == 0) st[per_row.d] = static_cast<uint8_t>(s);
    }
}

template <typename T, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_gated_backward(GatedArgs g, FastDiv per_row,
                                                           uint32_t blocks) {
    const uint32_t b = blockIdx.x * (kBlock / 4) + (threadIdx.x >> 2);
    if (b >= blocks) return;
    const uint32_t m = div_by(b, per_row), c = b - m * per_row.d;
    const int k = c * UE_PACK_BLOCK + (threadIdx.x & 3) * 8;
    const int8_t *from = g.q_in + m * g.ldq + k;
    const uint8_t *st = g.scale_in + m * g.lds + c;
    const uint64_t *pg = reinterpret_cast<const uint64_t *>(from);
    const uint64_t *pu = reinterpret_cast<const uint64_t *>(from + per_row.d * UE_PACK_BLOCK);
    const uint64_t qg = ONCE ? __builtin_nontemporal_load(pg) : *pg;
    const uint64_t qu = ONCE ? __builtin_nontemporal_load(pu) : *pu;
    const uint32_t sg = st[0], su = st[per_row.d];
    float d[8], gate[8], up[8], h[8];
    load8<ONCE>(static_cast<const T *>(g.dh) + m * g.ldin + k, g.I - k, d);
    unpack8(qg, sg, gate);
    unpack8(qu, su, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // s and 1 - s from exp(-|gate|), which never overflows
        const float v = gate[i], e = exp_of(-fabsf(v));
        const float r = __builtin_amdgcn_rcpf(1.0f + e);
        const float s = v >= 0.f ? r : e * r, rest = v >= 0.f ? e * r : r;
        const float silu = v * s;
        h[i] = silu * up[i];
        gate[i] = d[i] * up[i] * (s * __builtin_fmaf(v, rest, 1.0f));
        up[i] = d[i] * silu;
    }
    T *row = static_cast<T *>(g.dgu) + m * g.lddgu + k;
    store8<T>(row, g.I - k, gate);
    store8<T>(row + g.I, g.I - k, up);
    if (g.h) store8<T>(static_cast<T *>(g.h) + m * g.ldh + k, g.I - k, h);
}

// Rows of `per_row` blocks each, in launches of at most kLaunchBlocks blocks:
// f(first row, rows, blocks).
template <class F>
hipError_t in_parts(int M, int per_row, F f) {
    const int64_t rows = kLaunchBlocks / per_row;
    for (int64_t m = 0; m < M; m += rows) {
        const int n = static_cast<int>(M - m < rows ? M - m : rows);
        f(m, static_cast<uint32_t>(n) * per_row);
        const hipError_t he = hipGetLastError();
        if (he != hipSuccess) return he;
    }
    return hipSuccess;
}

dim3 grid_of(uint32_t blocks) { return dim3((blocks + kBlock / 4 - 1) / (kBlock / 4)); }

template <typename P>
P *ahead(P *p, int64_t bytes) {
    typedef typename std::conditional<std::is_const<P>::value, const char, char>::type C;
    return p ? reinterpret_cast<P *>(reinterpret_cast<C *>(p) + bytes) : p;
}
inline const void *ahead(const void *p, int64_t bytes) {
    return p ? static_cast<const char *>(p) + bytes : p;
}
inline void *ahead(void *p, int64_t bytes) {
    return p ? static_cast<char *>(p) + bytes : p;
}

}  // namespace

hipError_t launch_pack(const ue_ctx &, const PackArgs &g, hipStream_t s) {
    const int nb = (g.K + UE_PACK_BLOCK - 1) / UE_PACK_BLOCK;
    return in_parts(g.M, nb, [&](int64_t m, uint32_t blocks) {
        PackArgs p = g;
        p.x = ahead(g.x, m * g.ldx * (g.bf16 ? 2 : 4));
        p.q = g.q + m * g.ldq;
        p.scale = g.scale + m * g.lds;
        const int64_t bytes = static_cast<int64_t>(g.M) * g.K * (g.bf16 ? 2 : 4);
        with_rows(g.bf16, bytes, [&](auto t, auto once) {
            hipLaunchKernelGGL((k_pack<decltype(t), decltype(once)::value>), grid_of(blocks),
                               dim3(kBlock), 0, s, p, fast_div(nb), blocks);
        });
    });
}

hipError_t launch_unpack(const ue_ctx &, const PackArgs &g, hipStream_t s) {
    const int nb = (g.K + UE_PACK_BLOCK - 1) / UE_PACK_BLOCK;
    return in_parts(g.M, nb, [&](int64_t m, uint32_t blocks) {
        PackArgs p = g;
        p.out = ahead(g.out, m * g.ldx * (g.bf16 ? 2 : 4));
        p.q_in = g.q_in + m * g.ldq;
        p.scale_in = g.scale_in + m * g.lds;
        if (g.bf16)
            hipLaunchKernelGGL(k_unpack<uint16_t>, grid_of(blocks), dim3(kBlock), 0, s, p,
                               fast_div(nb), blocks);
        else
            hipLaunchKernelGGL(k_unpack<float>, grid_of(blocks), dim3(kBlock), 0, s, p,
                               fast_div(nb), blocks);
    });
}

hipError_t launch_gated(const ue_ctx &, const GatedArgs &g, hipStream_t s) {
    const int nb = (g.I + UE_PACK_BLOCK - 1) / UE_PACK_BLOCK, es = g.bf16 ? 2 : 4;
    return in_parts(g.M, nb, [&](int64_t m, uint32_t blocks) {
        GatedArgs p = g;
        p.gu = ahead(g.gu, m * g.ldin * es);
        p.h = ahead(g.h, m * g.ldh * es);
        p.q = ahead(g.q, m * g.ldq);
        p.scale = ahead(g.scale, m * g.lds);
        const int64_t bytes = static_cast<int64_t>(g.M) * g.I * 2 * es;
        with_rows(g.bf16, bytes, [&](auto t, auto once) {
            typedef decltype(t) T;
            constexpr bool kOnce = decltype(once)::value;
            if (g.q)
                hipLaunchKernelGGL((k_gated<T, true, kOnce>), grid_of(blocks), dim3(kBlock), 0, s,
                                   p, fast_div(nb), blocks);
            else
                hipLaunchKernelGGL((k_gated<T, false, kOnce>), grid_of(blocks), dim3(kBlock), 0,
                                   s, p, fast_div(nb), blocks);
        });
    });
}

hipError_t launch_gated_backward(const ue_ctx &, const GatedArgs &g, hipStream_t s) {
    const int nb = (g.I + UE_PACK_BLOCK - 1) / UE_PACK_BLOCK, es = g.bf16 ? 2 : 4;
    return in_parts(g.M, nb, [&](int64_t m, uint32_t blocks) {
        GatedArgs p = g;
        p.dh = ahead(g.dh, m * g.ldin * es);
        p.dgu = ahead(g.dgu, m * g.lddgu * es);
        p.h = ahead(g.h, m * g.ldh * es);
        p.q_in = g.q_in + m * g.ldq;
        p.scale_in = g.scale_in + m * g.lds;
        const int64_t bytes = static_cast<int64_t>(g.M) * g.I * (es + 2);
        with_rows(g.bf16, bytes, [&](auto t, auto once) {
            hipLaunchKernelGGL((k_gated_backward<decltype(t), decltype(once)::value>),
                               grid_of(blocks), dim3(kBlock), 0, s, p, fast_div(nb), blocks);
        });
    });
}

}  // namespace ue
