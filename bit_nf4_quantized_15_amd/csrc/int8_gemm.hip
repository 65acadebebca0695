// int8 matrix products of the layer on MFMA (gfx950).
//
// Forward  y[m,n]  = sx[m] sw[n] sum_k xq[m,k] wq[n,k] + sum_j t[m,j] B[j,n]
// Backward dx[m,k] = sum_n dy[m,n] W_16[n,k] + sum_j u[m,j] A[k,j],  W_16 = RNE_16(sw wq)
// ("bitsandbytes deep dive", section 4: vector-wise int8.)
#include "int8.h"

namespace qlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int DT>
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// 8 values at column j0.. of row `row` of a row-major [.., ld] matrix, zero outside
__device__ __forceinline__ u32x4_t row8(const uint16_t* __restrict__ p, int64_t ld, int row, bool ok, int j0, int jmax) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = j0 + 2 * i, b = a + 1;
        const uint32_t lo = ok && a < jmax ? p[row * ld + a] : 0u;
        const uint32_t hi = ok && b < jmax ? p[row * ld + b] : 0u;
        w[i] = lo | (hi << 16);
    }
    return u32x4_t{w[0], w[1], w[2], w[3]};
}
// 8 values of rows j0.. of column `col`
__device__ __forceinline__ u32x4_t col8(const uint16_t* __restrict__ p, int64_t ld, int col, bool ok, int j0, int jmax) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = j0 + 2 * i, b = a + 1;
        const uint32_t lo = ok && a < jmax ? p[a * ld + col] : 0u;
        const uint32_t hi = ok && b < jmax ? p[b * ld + col] : 0u;
        w[i] = lo | (hi << 16);
    }
    return u32x4_t{w[0], w[1], w[2], w[3]};
}

template <int DT>
__global__ __launch_bounds__(64) void int8_dx_simple_kernel(const uint16_t* __restrict__ dy,
                                                            const int8_t* __restrict__ wq,
                                                            const float* __restrict__ sw,
                                                            const uint16_t* __restrict__ u,
                                                            const uint16_t* __restrict__ A, uint16_t* __restrict__ dx,
                                                            int M, int N, int K, int r, int tk) {
    const int lane = threadIdx.x, h = lane >> 5, l32 = lane & 31;
    const int m0 = (int)(blockIdx.x / tk) * 32, k0 = (int)(blockIdx.x % tk) * 32;
    f32x16_t f;
#pragma unroll
    for (int v = 0; v < 16; ++v) f[v] = 0.0f;
    for (int n = 0; n < N; n += 16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int nn = n + 8 * h + 2 * i + p;
                e[p] = nn < N ? sw[nn] * (float)wq[(int64_t)nn * K + k0 + l32] : 0.0f;
            }
            w[i] = pack2<DT>(e[0], e[1]);
        }
        f = mfma32<DT>(row8(dy, N, m0 + l32, m0 + l32 < M, n + 8 * h, N), u32x4_t{w[0], w[1], w[2], w[3]}, f);
    }
    for (int j = 0; j < r; j += 16)
        f = mfma32<DT>(row8(u, r, m0 + l32, m0 + l32 < M, j + 8 * h, r), row8(A, r, k0 + l32, true, j + 8 * h, r), f);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int m = m0 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < M) dx[(int64_t)m * K + k0 + l32] = (uint16_t)(pack2<DT>(f[v], 0.0f) & 0xFFFFu);
    }
}

}  // namespace

qlora_status launch_int8_gemm_bwd_dx(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                     const uint16_t* A, uint16_t* dx, int M, int N, int K, int r, int dt,
                                     hipStream_t s) {
    const int64_t tm = ((int64_t)M + 31) / 32, tk = K / 32;
    if (tm * tk >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        hipLaunchKernelGGL(int8_dx_simple_kernel<DT>, dim3((unsigned)(tm * tk)), dim3(64), 0, s, dy, wq, sw, u, A, dx,
                           M, N, K, r, (int)tk);
    });
    return launch_status();
}

}  // namespace qlora
