// Which kernel an int8 product takes, and how many workgroups its launch has.
// Host code of its own, without HIP, so that a test can ask the same rule.
#pragma once

#include <cstdint>

namespace ue {

// A launch has fewer than 2^32 threads along an axis: of one with more, the
// runtime reports success and runs what is left modulo 2^32.
constexpr int64_t kLaunchThreads = 0xFFFFFFFFll;

// Which kernel, by what each measured on an MI355X (us; rows x K x channels,
// G: groups, each with a matrix of its own):
//                        256x256  128x256  128x128   64x64   32x64    rows
//   8192x7168x4096           192      220      231     370     540
//   1000x2048x2048            28       18     12.8    10.0    14.7
//   333x1900x1002             38       23     14.4     7.8     7.0
//   128x7168x4096             71       43     44.0    17.5    15.9
//   32x7168x4096              62       39     26.6    14.7    14.5
//   16x7168x4096              60       38     25.6    14.7    14.4     9.5
//   1x7168x4096               60       38     25.1    14.4    14.1     6.6
//   G=64, 512 rows each:
//     32768x4096x2048        306      326      355
//     32768x1024x4096        233      285      302
//   G=72, 150 to 800 rows:
//     32768x4096x2048        445      392      437
//     32768x1024x4096        288      300      317
//   G=64: 4096x1024x4096      79               69.7    80.7     112
//   G=64: 2048x4096x2048     142                138     119     114
// Larger tiles read each operand less often and cost less energy (with random
// data the power limit, not the issue rate, sets the clock); smaller ones give
// the launch enough workgroups. So: the largest tile that groups of the mean
// length at least half fill and that makes three workgroups for every four
// CUs; up to 16 rows go to the row kernel. Groups with long rows, whose
// matrices come from HBM, take the tile with three stages: its loads have two
// stages' time to arrive, and its lesser height fits uneven groups better (392
// against 445 us above; with even groups, which the host cannot tell since the
// offsets are on the device, it loses 326 to 306). Where between K = 1024 and
// 4096 the two cross was not measured. From 17 to some hundred rows the times
// are latency's (14.6 us for 17 rows, 15.6 for 128; the matrix's bytes take 6):
// 64 to 128 workgroups, each walking all of K.
enum I8Kernel {
    kI8Rows,        // up to 16 rows, the matrix streamed past them
    kI8Tall,        // 256 rows by 256 channels, two stages in LDS
    kI8Deep,        // 128 by 256, three stages
    kI8Mid,         // 128 by 128, two stages
    kI8Small,       // 64 by 64, four stages
    kI8Least,       // 32 by 64, six stages
    kI8Wide         // as kI8Small, rows of activations past 4 GiB
};

struct I8Tile {
    const char *name;
    int bm, bn, threads;    // rows and matrix rows of a workgroup
};

constexpr I8Tile i8_tile(I8Kernel k) {
    constexpr I8Tile t[] = {{"rows", 16, 16, 512},      {"256x256", 256, 256, 512},
                            {"128x256", 128, 256, 512}, {"128x128", 128, 128, 512},
                            {"64x64", 64, 64, 256},     {"32x64", 32, 64, 256},
                            {"64x64 wide", 64, 64, 256}};
    return t[k];
}

struct I8Size {
    int M;
    int64_t N;              // channels out
    int K, G;               // G: groups, 1 without offsets
    bool gated, grouped;    // grouped: offsets are given
    bool wide;              // offsets of indexed rows need 64 bits
    int num_cu;
};

constexpr int kFewRows = 16;

inline I8Kernel i8_kernel(const I8Size &z) {
    const int64_t channels = z.gated ? 2 * z.N : z.N;
    if (z.wide) return kI8Wide;
    if (z.M <= kFewRows && z.G <= 65535 &&
        (z.N + 15) / 16 * i8_tile(kI8Rows).threads <= kLaunchThreads)
        return kI8Rows;
    auto fits = [&](I8Kernel k) {
        const I8Tile t = i8_tile(k);
        const int64_t tiles = ((static_cast<int64_t>(z.M) + t.bm - 1) / t.bm +
                               (z.grouped ? z.G / 2 : 0)) *
                              ((channels + t.bn - 1) / t.bn);
        return z.M / z.G >= t.bm / 2 && tiles >= z.num_cu * 3 / 4;
    };
    if (fits(kI8Tall)) return z.grouped && z.K >= 2048 ? kI8Deep : kI8Tall;
    if (fits(kI8Mid)) return kI8Mid;
    return fits(kI8Small) ? kI8Small : kI8Least;
}

// Workgroups along the grid's first axis (the row kernel's groups are the
// second).
inline int64_t i8_workgroups(I8Kernel k, const I8Size &z) {
    const I8Tile t = i8_tile(k);
    const int out = z.gated && k != kI8Rows ? t.bn / 2 : t.bn;
    const int64_t columns = (z.N + out - 1) / out;
    if (k == kI8Rows) return columns;
    // each group's last tile may be partial
    return columns * ((static_cast<int64_t>(z.M) + t.bm - 1) / t.bm + (z.grouped ? z.G : 0));
}

}  // namespace ue
