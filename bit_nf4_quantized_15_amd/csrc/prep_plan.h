// Host-side work split of the products of lora_prep.h; shared by the launchers and by the
// workspace-size queries.
#pragma once

#include "lora_plan.h"

namespace qlora {

// 128 tokens a workgroup, and splits of C, in whole blocks of 128, for about `wgs` workgroups over
// all `items` of a launch.
inline SplitPlan plan_stream(int64_t M, int64_t C, int items, int64_t most) {
    const int64_t tiles = (M + 127) / 128, blocks = (C + 127) / 128, wgs = 512;
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>(std::min(blocks, most), wgs / (tiles * items)));
    const int64_t chunk = (blocks + s - 1) / s * 128;
    return SplitPlan{(int)((C + chunk - 1) / chunk), (int)chunk};
}
// fp32 sums of every split [split][M][r rounded up to 4]
inline size_t stream_ws_bytes(int64_t M, int64_t C, int r) {
    const int splits = plan_stream(M, C, 1, C).splits;
    return splits > 1 ? align256((size_t)splits * M * ((r + 3) & ~3) * 4) : 0;
}
// In a workspace of nt_ws_bytes: the sums of all splits but one lie there, of whole tiles.
inline SplitPlan plan_down(int64_t M, int64_t C, int r, int items) {
    return plan_stream(M, C, items, plan_nt(M, C, r).splits - 1);
}

}  // namespace qlora
