// Host-side choices of the int8 layer: which kernel, which tile and which split a size takes.
// Shared by the launchers, the workspace-size queries and the tests.
#pragma once

#include <algorithm>
#include <cstdint>

namespace qlora {

// ---- forward, up to kInt8GemvMaxM tokens: one launch
constexpr int kInt8GemvMaxM = 16;
inline bool int8_gemv_supported(int64_t M, int64_t N, int64_t K, int r) {
    // (buffer offsets of B and A within 31 bits)
    return M <= kInt8GemvMaxM && (int64_t)r * N * 2 < (int64_t(1) << 31) && (int64_t)r * K * 2 < (int64_t(1) << 31);
}

inline bool int8_gemv_quantizes(int64_t M, int64_t K) { return M * (K + 16) <= (int64_t(72) << 10); }

// ---- preparation of x (and u of few tokens)
// Tokens per workgroup: with few of them a CU's own rate bounds a workgroup, so it takes
// fewer tokens (of the MFMA's 16 columns the others multiply zeros) while that fills the chip.
// The forward of 333 x 11008 -> 4096, r = 8: 50.1 us with 16 tokens each, 39.6 us with 2;
// 128 x 4096 -> 4096, r = 16: 21.1 and 16.7 us.
inline int int8_rows_per_wg(int64_t M) {
    int per = 16;
    while (per > 2 && M <= 256 * (per / 2)) per /= 2;
    return per;
}

// The forward's preparation: 32 tokens halve what each workgroup reads of A, but only where there
// are tokens for every CU (and registers for them).
inline int int8_prep_rows(int64_t M, int r) { return r <= 64 && M > 4096 ? 32 : int8_rows_per_wg(M); }

// Every workgroup of the backward's u reads all of B, so this pays for few tokens, narrow layers and small ranks.
// The whole dx call, us, here and with split sums (tokens x N, r): 300 x 4096, 16: 38.1, 46.6;
// 512 x 4096, 64: 55.2, 64.4; 100 x 11008, 64: 88.3, 106.1; 512 x 11008, 16: 77.6, 80.2; but
// 777 x 11000, 24: 108.6, 106.6; 512 x 11008, 64: 111.2, 93.3; 64 x 28672, 64: 186.4, 159.6.
inline bool int8_u_supported(int64_t M, int64_t N, int r) {
    return N % 8 == 0 && N <= 16384 && M <= 1024 && M * r * N <= 150000000;
}

// ---- forward, more tokens
enum Int8FwdTile { kFwd256x256, kFwd256x192, kFwd128x128, kFwd64x64 };
struct Int8Choice {
    int tile, splits;
};

inline int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

// The tile, and the split of the reduction, with the least estimated time in microseconds.
// A round of n tiles on the 256 CUs takes a start and end plus, per 64 k, the larger of a
// tile's MFMA time and its share of what the chip sustains.  The constants are fitted to such
// measurements; with every tile forced in turn (captured calls, r = 0, codes of x included, us; K = 4096
// unless given):
//   M x N                   256x256  256x192  128x128  split 2  split 4   64x64
//   8192 x 28672, K = 8192   1486.9   1602.0   2142.6
//   4096 x 4096                76.5     88.5     81.0                     134.1
//   2048 x 11008              100.9     89.4    105.8                     174.8
//   1024 x 4096                46.6     40.9     24.9     30.1             39.7
//   512 x 4096                 44.6     39.1     20.9     20.4     25.2    23.2
//   333 x 4096, K = 11008      97.4     85.6     40.5     31.1     35.9    52.9
//   100 x 11008                41.4     35.3     18.4     17.8     23.2    19.8
//   128 x 4096                 41.0     34.4     16.9     16.3     16.3    12.1
//   33 x 4096                  40.4     33.9     16.0     15.4     15.4    10.1
inline Int8Choice int8_fwd_choice(int64_t M, int64_t N, int64_t K, bool may_split) {
    const double steps = (double)K / 64;
    auto rounds = [&](int64_t n, double ends, double tile_us, double chip_us) {
        const double last = (double)(n % 256);
        return (double)(n / 256) * (ends + steps * chip_us) +
               (last > 0 ? ends + 4.0 + steps * std::max(tile_us, chip_us * last / 256) : 0.0);
    };
    Int8Choice best{kFwd256x256, 1};
    double us = rounds(tiles_of(M, N, 256, 256), 9.5, 0.44, 0.80);
    auto offer = [&](double t, int tile, int splits) {
        if (t < us) {
            us = t;
            best = Int8Choice{tile, splits};
        }
    };
    offer(rounds(tiles_of(M, N, 256, 192), 8.0, 0.34, 0.62), kFwd256x192, 1);
    const int64_t n128 = tiles_of(M, N, 128, 128), n64 = tiles_of(M, N, 64, 64);
    auto small = [&](int64_t n, double s) {   // 128 x 128, s steps each
        const double last = (double)(n % 256);
        return (double)(n / 256) * (2.5 + s * 0.28) + (last > 0 ? 4.0 + s * (0.12 + 0.16 * last / 256) : 0.0);
    };
    offer(small(n128, steps), kFwd128x128, 1);
    // a split adds a partial tile of 64 KB, written and read, and the wait for it
    if (may_split && K >= 1024)
        for (int s = 2; s <= 4 && n128 * s <= 256; ++s) offer(small(n128 * s, steps / s) + 3.0 + s, kFwd128x128, s);
    offer((double)((n64 + 511) / 512) * 3.0 + steps * (0.04 + 0.0005 * (double)n64), kFwd64x64, 1);
    return best;
}

// ---- input gradient
constexpr int kDxStep = 64;   // rows n of a step
enum Int8DxTile { kDx256x256, kDx128x256, kDx128x128, kDx64x128 };

// Direct loads of dy: whole 16-byte chunks, a panel's offsets within a buffer's 31 bits.
inline bool direct_dy(int64_t N) { return N % 8 == 0 && 512 * N < (int64_t(1) << 31); }

// The tile (tokens x columns), and the split of the reduction, with the least estimated time
// in microseconds: a round of n tiles on the 256 CUs takes a start and end plus, per 64 n,
// the larger of a lone tile's time and its share of what the chip sustains.  With every tile
// forced in turn (captured calls, r = 0, us; tokens x N x K):
//                        256x256  128x256  split 2  split 4  128x128  64x128
//   4096 x 11008 x 4096    276.3    324.8    352.5    401.8    402.4   453.6
//   2048 x 4096 x 4096      84.6     65.5     75.6     93.4     76.9    88.0
//   777 x 11000 x 4096     230.7    138.0     89.5     98.9     94.5   107.7
//   300 x 4096 x 4096       76.9     51.2     35.8     29.1     34.0    28.9
inline Int8Choice int8_dx_choice(int64_t M, int64_t N, int64_t K, bool may_split) {
    const double steps = (double)((N + kDxStep - 1) / kDxStep);
    auto rounds = [&](int64_t n, double s, double ends, double tile_us, double chip_us) {
        const double last = (double)(n % 256);
        return (double)(n / 256) * (ends + s * chip_us) +
               (last > 0 ? ends + s * std::max(tile_us, chip_us * last / 256) : 0.0);
    };
    Int8Choice best{kDx128x128, 1};
    double us = rounds(tiles_of(M, K, 128, 128), steps, 4.0, 0.47, 0.60);
    auto offer = [&](double t, int tile, int splits) {
        if (t < us) {
            us = t;
            best = Int8Choice{tile, splits};
        }
    };
    offer(rounds(tiles_of(M, K, 64, 128), steps, 3.0, 0.39, 0.39), kDx64x128, 1);
    if (!direct_dy(N)) return best;
    offer(rounds(tiles_of(M, K, 256, 256), steps, 9.0, 1.15, 1.72), kDx256x256, 1);
    const int64_t n = tiles_of(M, K, 128, 256);
    offer(rounds(n, steps, 4.0, 0.74, 1.03), kDx128x256, 1);
    // a split adds a partial tile of 128 KB, written and read, and the wait for it
    if (may_split)
        for (int s = 2; s <= 8 && n * s <= 256 && steps >= 4 * s; ++s)
            offer(rounds(n * s, steps / s, 4.0, 0.74, 1.03) + 4.0 + s, kDx128x256, s);
    return best;
}

}  // namespace qlora
