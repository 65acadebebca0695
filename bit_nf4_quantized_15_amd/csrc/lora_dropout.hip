// The LoRA branch's product with dropout (dropout.h), t = s drop(x) A of several layers in one launch
// (lora_prep.h), and the generator's arguments.
#include <cmath>

#include "lora_prep.h"

namespace qlora {

bool drop_args(const qlora_dropout* d, DropArgs* out) {
    *out = DropArgs{0u, 0u, 0u, 0u, 0u, 1.0f};
    if (!d) return true;
    if (!(d->p >= 0.0 && d->p < 1.0)) return false;
    const double thr = std::nearbyint(d->p * 65536.0);
    if (thr > 65535.0) return false;
    out->k0 = (uint32_t)d->seed;
    out->k1 = (uint32_t)(d->seed >> 32);
    out->o0 = (uint32_t)d->offset;
    out->o1 = (uint32_t)(d->offset >> 32);
    out->thr = (uint32_t)thr;
    out->inv = (float)(65536.0 / (65536.0 - thr));
    return true;
}

namespace {

// (two workgroups on a CU where the ranks' registers allow)
template <int TQ, bool VEC, int DT>
__global__ __launch_bounds__(256, TQ <= 2 ? 2 : 1) void down_stream_kernel(const StreamArgs a) {
    stream_body<TQ, VEC, true, true, false, DT>(a);
}

// n <= kStreamItems products
qlora_status down_stream(const NtDesc* d, const DropArgs* drop, int n, int r, int dt, hipStream_t s) {
    StreamArgs a{};
    bool vec = r % 8 == 0;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        a.item[i] = stream_item(d[i].X, d[i].Y, d[i].out, d[i].ws, drop[i], d[i].scale, d[i].M, d[i].C,
                                plan_down(d[i].M, d[i].C, r, n));
        // vector path: 16-byte rows, and one workgroup's rows under 1 GiB of buffer offsets
        vec = vec && d[i].C % 8 == 0 && (int64_t)d[i].C * 128 * 2 < (int64_t(1) << 30);
        a.first[i] = (int)total;
        total += (int64_t)a.item[i].tiles * a.item[i].splits;
        if (total * 256 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    }
    a.first[n] = (int)total;
    a.n = n;
    a.r = r;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_S(TQ)                                                                                                    \
    if (vec) hipLaunchKernelGGL((down_stream_kernel<TQ, true, DT>), dim3((unsigned)total), dim3(256), 0, s, a);    \
    else hipLaunchKernelGGL((down_stream_kernel<TQ, false, DT>), dim3((unsigned)total), dim3(256), 0, s, a);
        switch ((r + 31) / 32) {
            case 1: QL_S(1) break;
            case 2: QL_S(2) break;
            case 3: QL_S(3) break;
            default: QL_S(4) break;
        }
#undef QL_S
    });
    const qlora_status st = launch_status();
    return st == QLORA_OK ? launch_reduce(a, dt, s) : st;
}

}  // namespace

qlora_status launch_nt_batch_dropout(const NtDesc* d, const DropArgs* drop, int count, int r, int dt, hipStream_t s) {
    qlora_status st = QLORA_OK;
    for (int i = 0; i < count && st == QLORA_OK; i += kStreamItems)
        st = down_stream(d + i, drop + i, std::min(kStreamItems, count - i), r, dt, s);
    return st;
}

}  // namespace qlora
