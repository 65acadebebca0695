// Input gradient of the int8 layer on MFMA (v_mfma_f32_32x32x16_{bf16,f16}), gfx950:
//
//   dx[m,k] = RNE_16( sum_n dy[m,n] W_16[n,k] + sum_j u[m,j] A[k,j] ),
//   W_16[n,k] = RNE_16( fl32( sw[n] wq[n,k] ) )
//
// ("bitsandbytes deep dive", section 4: vector-wise int8; 12.4: frozen base, no dW.)  The
// reduction runs down the stored rows n, 64 per step: dy (whole 128-byte lines) and the int8
// weight (64 rows of its codes) are copied HBM -> LDS by direct loads.  An MFMA operand is 8
// consecutive n of one column k: gfx950's transposed byte read (ds_read_b64_tr_b8) hands a
// lane exactly those 8 codes, which it scales (a scale per n, the same for all columns) and
// rounds in registers: 20 VALU instructions per operand.  Each wave owns its columns over all
// rows of the tile, so no weight is expanded twice and the weight's LDS traffic is its one
// byte per element.
//
// While the MFMAs of 16 n run, dy and codes of the 16 n two further on are read and the codes
// read before are expanded for the next 16.  Bound by the MFMAs and the power they draw (the
// expansion's VALU work runs beside them).  4096 x 11008 x 4096, r = 64, traced: 278 us for a given
// u, 1.33 PFLOP/s; 309 us behind the kernel that makes u, 1.19 PFLOP/s.
#include "int8_gemm_dx.h"

namespace qlora {
namespace {

template <int MT, int NT, int RING, bool SPLIT, bool DYV, bool AV, int DT>
__global__ __launch_bounds__(kThreads, 1) void int8_gemm_dx_kernel(
    const uint16_t* __restrict__ dy, const int8_t* __restrict__ wq, const float* __restrict__ sw,
    const uint16_t* __restrict__ u, const uint16_t* __restrict__ A, uint16_t* __restrict__ dx, int M, int N, int K,
    int r, int tm, int tn, int gm, Split sp) {
    int8_gemm_dx_body<MT, NT, RING, SPLIT, DYV, AV, DT, false>(dy, wq, sw, u, A, dx, M, N, K, r, tm, tn, gm, sp,
                                                               DropArgs{});
}

template <int MT, int NT, int RING, bool SPLIT>
qlora_status run(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u, const uint16_t* A,
                 uint16_t* dx, int M, int N, int K, int r, int dt, bool dyv, int splits, void* ws, hipStream_t s) {
    constexpr int kBM = 32 * MT, kBN = 32 * NT * kWaves;
    const int tm = (int)(((int64_t)M + kBM - 1) / kBM), tn = (int)(((int64_t)K + kBN - 1) / kBN), gm = 4;
    const int64_t tiles = (int64_t)tm * tn;
    Split sp{};
    if (SPLIT) {
        const int steps = (int)(((int64_t)N + kStep - 1) / kStep);
        sp.per = (steps + splits - 1) / splits;
        sp.splits = (steps + sp.per - 1) / sp.per;
        sp.tags = static_cast<uint64_t*>(ws);
        sp.part = static_cast<uint8_t*>(ws) + align256((size_t)(tiles * splits) * 8);
    }
    const int64_t total = tiles * (SPLIT ? sp.splits : 1);
    if (total * kThreads >= (int64_t(1) << 32) || (int64_t)gm * tn >= (int64_t(1) << 31))
        return QLORA_ERR_UNSUPPORTED_SHAPE;
    const bool av = r % 8 == 0;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_DX(V, W)                                                                                            \
    hipLaunchKernelGGL((int8_gemm_dx_kernel<MT, NT, RING, SPLIT, V, W, DT>), dim3((unsigned)total), dim3(kThreads), 0, s, dy, \
                       wq, sw, u, A, dx, M, N, K, r, tm, tn, gm, sp)
        if constexpr (NT == 2) {   // (chosen for direct loads only)
            if (av) QL_DX(true, true); else QL_DX(true, false);
        } else if (dyv) {
            if (av) QL_DX(true, true); else QL_DX(true, false);
        } else {
            if (av) QL_DX(false, true); else QL_DX(false, false);
        }
#undef QL_DX
    });
    return launch_status();
}

}  // namespace

size_t int8_gemm_dx_workspace(int64_t M, int64_t N, int64_t K) {
    const Int8Choice c = int8_dx_choice(M, N, K, true);
    if (c.splits == 1) return 0;
    const int64_t tiles = tiles_of(M, K, 128, 256);
    return align256((size_t)(tiles * c.splits) * 8) + (size_t)(tiles * (c.splits - 1)) * 128 * 256 * 4;
}

qlora_status launch_int8_gemm_bwd_dx(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                     const uint16_t* A, uint16_t* dx, int M, int N, int K, int r, int dt, void* ws,
                                     hipStream_t s) {
    const bool dyv = direct_dy(N);
    const Int8Choice c = int8_dx_choice(M, N, K, ws != nullptr);
    switch (c.tile) {
        case kDx256x256: return run<8, 2, 2, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        case kDx128x256:
            return c.splits > 1 ? run<4, 2, 4, true>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, c.splits, ws, s)
                                : run<4, 2, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        case kDx128x128: return run<4, 1, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        default: return run<2, 1, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
    }
}

}  // namespace qlora
