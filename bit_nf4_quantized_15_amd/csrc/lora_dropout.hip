// The LoRA products of a training step with dropout (dropout.h): t = s drop(x) A and dA =
// drop(x)^T u beside dB = t^T dy, for several layers in one launch each.  The bodies are those of
// lora_body.h; a lane holds 8 consecutive columns of a row of x, the unit of the generator, and
// masks them in registers between the load and the MFMA operand (t) or the LDS tile (dA).
#include <cmath>

#include "lora_body.h"

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

struct NtDropBatch {
    NtBatch b;
    DropArgs drop[kNtBatch];
};

template <int TQ, bool VEC, int NST, int DT>
__global__ __launch_bounds__(256) void ntb_dropout_kernel(const NtDropBatch bt) {
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.b.n && b >= bt.b.first[i + 1]) ++i;
    const NtProb& p = bt.b.p[i];
    const int c = b - bt.b.first[i];
    const NtMore more{bt.drop[i], nullptr, nullptr, 0, 0};
    nt_body<TQ, VEC, true, NST, DT, true>(p.X, p.Y, p.tags, p.part, p.out, p.scale, p.M, p.C, bt.b.r, p.chunk,
                                          c % p.tiles, c / p.tiles, p.tiles, p.splits, more);
}

template <int TQ, bool VEC, int NST, int DT>
__global__ __launch_bounds__(256, TQ <= 2 && VEC ? 2 : 1) void tnb_dropout_kernel(const TnBatch bt) {
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.n && b >= bt.first[i + 1]) ++i;
    const int c = b - bt.first[i];
    tn_body<TQ, VEC, NST, DT, true>(bt.p[i], c % bt.p[i].tiles, c / bt.p[i].tiles);
}

struct TnDropLaunch {
    const TnBatch& b;
    unsigned n;
    hipStream_t s;
    template <int TQ, bool V, int NST, int DT>
    void operator()() const {
        hipLaunchKernelGGL((tnb_dropout_kernel<TQ, V, NST, DT>), dim3(n), dim3(256), 0, s, b);
    }
};

}  // namespace

qlora_status launch_nt_batch_dropout(const NtDesc* d, const DropArgs* drop, int count, int r, int dt, hipStream_t s) {
    const int tq = (r + 31) / 32;
    for (int i0 = 0; i0 < count; i0 += kNtBatch) {
        NtDropBatch db{};
        bool vec = false;
        int chunk = 64;
        unsigned total = 0;
        const qlora_status st = nt_batch(d + i0, std::min(kNtBatch, count - i0), true, r, db.b, vec, chunk, total);
        if (st != QLORA_OK) return st;
        for (int i = 0; i < db.b.n; ++i) {
            db.drop[i] = drop[i0 + i];
            db.b.p[i].scale *= drop[i0 + i].inv;
        }
        const int nst = steps_template(chunk);
#define QL_D(TQ, V, NST) \
    hipLaunchKernelGGL((ntb_dropout_kernel<TQ, V, NST, DT>), dim3(total), dim3(256), 0, s, db);
#define QL_D1(TQ, V)                       \
    if (nst == 2) { QL_D(TQ, V, 2) }       \
    else if (nst == 4) { QL_D(TQ, V, 4) }  \
    else { QL_D(TQ, V, (TQ == 4 ? 4 : 8)) }
#define QL_D2(TQ) \
    if (vec) { QL_D1(TQ, true) } else { QL_D1(TQ, false) }
        with_dt(dt, [&](auto dtc) {
            constexpr int DT = decltype(dtc)::value;
            switch (tq) {
                case 1: QL_D2(1) break;
                case 2: QL_D2(2) break;
                case 3: QL_D2(3) break;
                default: QL_D2(4) break;
            }
        });
#undef QL_D2
#undef QL_D1
#undef QL_D
        const qlora_status ls = launch_status();
        if (ls != QLORA_OK) return ls;
    }
    return QLORA_OK;
}

qlora_status launch_tn_batch_dropout(const TnDesc* d, const DropArgs* drop, int count, int r, int dt, hipStream_t s) {
    for (int i0 = 0; i0 < count; i0 += kTnBatch) {
        TnBatch b{};
        bool vec = false;
        int chunk = 64;
        unsigned total = 0;
        const qlora_status st = tn_batch(d + i0, std::min(kTnBatch, count - i0), r, b, vec, chunk, total);
        if (st != QLORA_OK) return st;
        for (int i = 0; i < b.n; ++i) b.p[i].drop = drop[i0 + i];
        const TnDropLaunch go{b, total, s};
        tn_dispatch(r, vec, chunk, dt, go);
        const qlora_status ls = launch_status();
        if (ls != QLORA_OK) return ls;
    }
    return QLORA_OK;
}

}  // namespace qlora
