// Host-side work split of the gradients with dropout (lora_grads_dropout.hip).
#pragma once

#include "lora_plan.h"

namespace qlora {

constexpr int kGradCols = 128;                                   // columns of X per workgroup
constexpr int64_t kGradMaxWidth = int64_t(1) << 22;              // of X: a wave's rows lie within 31-bit offsets
inline int ranks_per_lane(int r) { return r <= 32 ? 1 : r <= 64 ? 2 : 4; }
inline int64_t grad_tiles(int64_t D) { return (D + kGradCols - 1) / kGradCols; }

// Splits of M rows for a launch of all_tiles output tiles.  A split costs a partial tile, written
// and read again (32 KB at r = 64 against 256 bytes a row of X), and lies in a workspace of
// tn_ws_bytes, whose partial tiles are of whole 32 ranks.  Enough for 512 workgroups, two a CU, of
// 128 rows or more, and 2048 rows at most.  Measured, us: one layer of 4096 tokens, K = 4096, N = 11008,
// r = 64: 31.7 (4 splits), 35.9 (2), 40.2 (11); 500 tokens at r = 16: 11.4 (3 splits), 12.5 (1);
// seven layers of a 7B-size block, 4096 tokens, r = 64: 151 (2 splits), 156 (1), 161 (4).
inline SplitPlan plan_grad_dropout(int64_t M, int64_t D, int r, int64_t all_tiles) {
    // a wave's quarter of a chunk, addressed with 31 bits
    const int64_t most = ((int64_t(1) << 31) - 1) / (2 * std::max<int64_t>(D, 128)) / 16 * 64;
    const int64_t fit = (int64_t)(plan_tn(M, D, r).splits - 1) * ((r + 31) / 32) / ranks_per_lane(r) + 1;
    const int64_t want = std::max(std::min<int64_t>(512 / all_tiles, M / 128), (M + 2047) / 2048);
    const int64_t s = std::max<int64_t>({1, (M + most - 1) / most, std::min(want, fit)});
    const int64_t chunk = ((M + s - 1) / s + 63) / 64 * 64;
    return SplitPlan{(int)((M + chunk - 1) / chunk), (int)chunk};
}

}  // namespace qlora
