// Host-side choices of the 8-bit float layer: which kernel, which tile and which split a size
// takes.  Shared by the launchers, the workspace-size queries and the tests.
#pragma once

#include <algorithm>
#include <cstdint>

#include "lora_plan.h"

namespace qlora {

constexpr int kFp8Block = 128;
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
inline int64_t pad4(int64_t n) { return (n + 3) & ~int64_t(3); }

// ---- forward, up to kFp8GemvMaxM tokens: one launch
constexpr int kFp8GemvMaxM = 16;
// (LDS holds the scales of 16 tokens: K / 8 bytes)
inline bool fp8_gemv_supported(int64_t M, int64_t K) { return M <= kFp8GemvMaxM && K <= (int64_t(1) << 18); }
// (the codes of x beside the rest in LDS, rows of whole runs of 512 and 16 bytes)
inline bool fp8_gemv_quantizes(int64_t M, int64_t K) { return M * ((K + 511) / 512 * 512 + 16) <= (int64_t(72) << 10); }

// ---- products
enum Fp8Tile { kFp8T256x256, kFp8T128x128, kFp8T64x64 };
struct Fp8Choice {
    int tile, splits;
};

// Tokens M x outputs O, reduction C.  The tile, and the split of the reduction, with the least
// estimated time in microseconds: a round of n tiles on the 256 CUs takes a start and end plus,
// per block of 128, the larger of a lone tile's time and its share of what the chip sustains.
// Fitted to captured calls with every choice forced in turn (r = 0, the operand's codes included, us):
//   M x O, C                256x256  128x128  split 2  split 4  64x64
//   8192 x 28672, 8192       1455.4   2119.8
//   4096 x 4096, 4096          64.8     79.5                    120.7
//   2048 x 11008, 4096        102.0    105.7                    160.1
//   1024 x 4096, 4096          49.4     25.1                     34.2
//   512 x 4096, 4096           47.7     21.3     21.1            20.2
//   333 x 4096, 11008         114.1     41.0     32.2            41.9
//   128 x 4096, 4096           43.8     18.1     17.3     16.9   14.2
//   100 x 4096, 11008 (dx)    103.4     41.6     28.3     24.2   32.4
inline Fp8Choice fp8_choice(int64_t M, int64_t O, int64_t C, bool may_split) {
    const double steps = (double)fp8_blocks(C);
    auto tiles = [&](int b) { return ((M + b - 1) / b) * ((O + b - 1) / b); };
    auto rounds = [&](int64_t n, double s, double ends, double more, double tile_us, double chip_us) {
        const double last = (double)(n % 256);
        return ends - more + (double)(n / 256) * (more + s * chip_us) +
               (last > 0 ? more + s * std::max(tile_us, chip_us * last / 256) : 0.0);
    };
    Fp8Choice best{kFp8T256x256, 1};
    double us = rounds(tiles(256), steps, 8.0, 8.0, 1.0, 1.45);
    auto offer = [&](double t, int tile, int splits) {
        if (t < us) {
            us = t;
            best = Fp8Choice{tile, splits};
        }
    };
    offer(rounds(tiles(128), steps, 4.0, 2.5, 0.33, 0.47), kFp8T128x128, 1);
    // a split adds a partial tile of 64 KB, written and read, and the wait for it
    if (may_split)
        for (int s = 2; s <= 8 && tiles(128) * s <= 256 && steps >= 4 * s; ++s)
            offer(rounds(tiles(128) * s, steps / s, 4.0, 2.5, 0.33, 0.47) + 2.5 + 1.1 * s, kFp8T128x128, s);
    const int64_t n64 = tiles(64);
    offer((double)((n64 + 511) / 512) * 3.0 + steps * (0.165 + 0.00052 * (double)n64), kFp8T64x64, 1);
    return best;
}

}  // namespace qlora
