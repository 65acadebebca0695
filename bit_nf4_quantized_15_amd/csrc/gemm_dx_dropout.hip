// Backward dx of the NF4 / FP4 layer with dropout on the LoRA branch:
//   dx[m,k] = sum_n dy[m,n] w_hat[n,k] + drop( sum_j u[m,j] A[k,j] )
// (gemm_dx.h's kernel; dropout.h).  The r steps of u A^T come first and drop() is applied to
// their fp32 sums, onto which the base's steps are then added: no accumulators more, and one
// rounding.  A 256 x 256 tile takes 8192 generator calls, 32 to a wave's SIMD.  u and dx in a graph, us, without
// dropout and with: 2048 x 4096 -> 4096, r = 64: 114, 121 (128 tiles on 256 CUs); 4096 x 11008 -> 4096: 348, 353.
#include "gemm_dx.h"

namespace qlora {
qlora_status launch_gemm_bwd_dx_dropout(const uint16_t* dy, const uint8_t* codes, const uint8_t* q8, const float* a2,
                                        int cb, int dt, const uint16_t* u, const uint16_t* A, const DropArgs& drop,
                                        uint16_t* dx, int M, int N, int K, int r, hipStream_t s) {
    const int tm = (M + kTM - 1) / kTM, tk = (K + kTN - 1) / kTN;
    // Direct loads only when every step is 64 whole columns: a tile load puts the
    // column offset in soffset, which the buffer range check does not cover, so a
    // partial last step would read past row ends (the next row's head, or past the
    // end of dy for the panel's last row).  Other widths take the register path,
    // which zeroes every element past N.
    const bool vec = (N % kTK == 0) && ((reinterpret_cast<uintptr_t>(dy) & 15u) == 0) &&
                     ((int64_t)kTM * N * 2 < (int64_t(1) << 32));
    // q8 == NULL: no double quantization, a2 holds one fp32 absmax per block
    with_cb_dt(cb, dt, [&](auto cbc, auto dtc) {
        constexpr int CB = decltype(cbc)::value, DT = decltype(dtc)::value;
#define QL_BWD(V, DQ)                                                                                           \
    hipLaunchKernelGGL((nf4_gemm_bwd_dx_kernel<V, DQ, CB, DT, DropArgs>), dim3(tm * tk), dim3(kT8), 0, s, dy, codes, q8, a2, u, \
                       A, dx, M, N, K, r, tm, tk, drop)
        if (q8) {
            if (vec) QL_BWD(true, true); else QL_BWD(false, true);
        } else {
            if (vec) QL_BWD(true, false); else QL_BWD(false, false);
        }
#undef QL_BWD
    });
    return launch_status();
}

}  // namespace qlora
