// Rows of activations as 8-bit integers (ue_quantize_rows).
//
// Per row x: top = max |x|, q = rint(x * (127 / top)) (nearest even), scale =
// top / 127, so that q * scale is within half a step of x. A row of zeros gets
// q = 0 and scale 0. A row that holds an infinity or a NaN gets q = 0 and a
// scale of NaN: every product of that row is then NaN, and no other row's.
//
// Many rows of up to kWaveRow elements take one wave each, longer or few ones a
// workgroup (a workgroup per row of 1024 left half its lanes without work:
// 44 us for 32768 of them, fp32, against 26 by waves; 333 rows of 1900, bf16
// and unaligned, take 4.2 by workgroups and 6.3 by waves). Rows of up to kVec
// elements per lane stay in registers between the maximum and the rounding;
// longer rows are read again.
//
// Bound: HBM. 8192 rows of 7168, bf16: 32 us for 176 MB (5.5 TB/s).
#include "ue_gate.h"

namespace ue {
namespace {

constexpr int kVec = 32;      // elements a thread keeps, in pieces of kPiece
constexpr int kPiece = 8;

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<uint16_t>(uint16_t v) {
    return bf16_to_f32(v);
}

// Elements [k, k + kPiece) of a row as floats, 0 past the end.
template <typename T>
__device__ __forceinline__ void load_piece(const T *x, int k, int K, bool vec,
                                           float (&f)[kPiece]) {
    if (vec && k + kPiece <= K) {
        struct alignas(16) Pack { T v[kPiece]; };
        const Pack p = *reinterpret_cast<const Pack *>(x + k);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) f[i] = as_float<T>(p.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            f[i] = k + i < K ? as_float<T>(x[k + i]) : 0.f;
    }
}

constexpr int kWaveRow = 64 * kVec;
constexpr int kManyRows = 2048;

// LANES: of a row, a wave's or a workgroup's.
template <typename T, int LANES>
__global__ __launch_bounds__(kBlock) void k_quantize(QuantArgs g) {
    __shared__ uint32_t wtop[kWaves];
    const int tid = threadIdx.x % LANES;
    const int64_t m = LANES == kBlock ? blockIdx.x
                                      : static_cast<int64_t>(blockIdx.x) * kWaves +
                                            (threadIdx.x >> 6);
    if (m >= g.M) return;               // (whole waves; no barrier below then)
    const T *x = static_cast<const T *>(g.x) + m * g.ldx;
    float f[kVec / kPiece][kPiece];
    // magnitudes order like their bits; infinities and NaN come last
    uint32_t top = 0;
    const int step = LANES * kPiece;
#pragma unroll
    for (int c = 0; c < kVec / kPiece; ++c)
        load_piece<T>(x, c * step + tid * kPiece, g.K, g.vec, f[c]);
#pragma unroll
    for (int c = 0; c < kVec / kPiece; ++c)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const uint32_t b = __float_as_uint(f[c][i]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
    for (int k = LANES * kVec + tid * kPiece; k < g.K; k += step) {
        float e[kPiece];
        load_piece<T>(x, k, g.K, g.vec, e);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const uint32_t b = __float_as_uint(e[i]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
    }
    top = wave_max_u32(top);
    if constexpr (LANES == kBlock) {
        if (lane_id() == 0) wtop[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = wtop[i] > top ? wtop[i] : top;
    }
    const bool finite = top < 0x7F800000u;
    const float t = __uint_as_float(top);
    // (127 / top overflows for a row of the smallest numbers: such a row
    // counts as zeros)
    float inv = finite && top ? 127.0f / t : 0.f;
    if (inv > __FLT_MAX__) inv = 0.f;
    if (tid == 0)
        g.scale[m] = finite ? (inv > 0.f ? t / 127.0f : 0.f)
                            : __builtin_nanf("");
    int8_t *q = g.q + m * g.ldq;
    auto store = [&](int k, const float (&e)[kPiece]) {
        // pads the row with zeros up to a multiple of 16
        if (k >= g.Kpad) return;
        union { int8_t b[kPiece]; uint64_t w; } u;
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            u.b[i] = static_cast<int8_t>(
                finite ? static_cast<int>(rintf(e[i] * inv)) : 0);
        *reinterpret_cast<uint64_t *>(q + k) = u.w;
    };
#pragma unroll
    for (int c = 0; c < kVec / kPiece; ++c)
        store(c * step + tid * kPiece, f[c]);
    for (int k = LANES * kVec + tid * kPiece; k < g.Kpad; k += step) {
        float e[kPiece];
        load_piece<T>(x, k, g.K, g.vec, e);
        store(k, e);
    }
}

template <typename T>
hipError_t quantize_any(const QuantArgs &g, hipStream_t s) {
    if (g.K <= kWaveRow && g.M >= kManyRows)
        hipLaunchKernelGGL((k_quantize<T, 64>), dim3((static_cast<int64_t>(g.M) + kWaves - 1) / kWaves),
                           dim3(kBlock), 0, s, g);
    else
        hipLaunchKernelGGL((k_quantize<T, kBlock>), dim3(g.M), dim3(kBlock), 0, s, g);
    return hipGetLastError();
}

}  // namespace

// In launches of at most 2^23 rows: a launch has fewer than 2^32 threads (of one
// with more the runtime reports success and runs the rest modulo 2^32).
hipError_t launch_quantize(const QuantArgs &g, hipStream_t s) {
    constexpr int kRows = 1 << 23;
    for (int64_t m = 0; m < g.M; m += kRows) {
        QuantArgs part = g;
        part.M = static_cast<int>(g.M - m < kRows ? g.M - m : kRows);
        part.x = static_cast<const char *>(g.x) + m * g.ldx * (g.bf16 ? 2 : 4);
        part.q = g.q + m * g.ldq;
        part.scale = g.scale + m;
        const hipError_t he = g.bf16 ? quantize_any<uint16_t>(part, s)
                                     : quantize_any<float>(part, s);
        if (he != hipSuccess) return he;
    }
    return hipSuccess;
}

}  // namespace ue
