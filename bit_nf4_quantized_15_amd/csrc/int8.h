// Launchers and device helpers of the int8 layer (int8 codes with one fp32 scale per
// row; declared in qlora.h, section "int8").
#pragma once

#include "common.h"
#include "int8_plan.h"

namespace qlora {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// int32 sums of K products of codes stay below 2^31: 128 * 128 * (2^17 - 64) < 2^31.
constexpr int64_t kInt8MaxK = int64_t(1) << 17;
// Rows (tokens, outputs) of a product: kernels count tiles and chunks in 32 bits up to 8208 rows
// past the last (the decode kernel asks for the row tile after its own, 512 tiles of 16 on).
constexpr int64_t kInt8MaxRows = (int64_t(1) << 31) - 16384;
// The input gradient's tiles have up to 256 rows of K 16-bit values within 31-bit offsets.
constexpr int64_t kInt8DxMaxK = int64_t(1) << 22;
// It reads the weight's scales, 4 bytes each, at 31-bit offsets too.
constexpr int64_t kInt8DxMaxN = int64_t(1) << 29;

// The 16-bit values of the four codes of a dword, two per result word:
// RNE_16(fl32(scale * code)).  The compiler converts each signed byte in place
// (v_cvt_f32_i32 with a byte selector), so a value costs 2.5 VALU instructions.
template <int DT>
__device__ __forceinline__ u32x2_t int8_values4(uint32_t b, float scale) {
    const float f0 = (float)(int32_t)(int8_t)b * scale;
    const float f1 = (float)(int32_t)(int8_t)(b >> 8) * scale;
    const float f2 = (float)(int32_t)(int8_t)(b >> 16) * scale;
    const float f3 = (float)((int32_t)b >> 24) * scale;
    return u32x2_t{pack2<DT>(f0, f1), pack2<DT>(f2, f3)};
}

// ---- codes of a row.
// With a = max|x| of the row, the code is the integer nearest to 127 x / a in exact
// arithmetic, ties toward zero.  One fma decides it: fma(x, inv, 1.5 * 2^23) with
// inv = fl(127/a) (1 - 2^-21), whose low byte is the rounded integer in two's
// complement.  inv is below 127/a by a relative 2^-21 +- 2^-23.  A real quotient that is
// no tie lies at least 1/(254 * 2047) > 2^-19 (fp16; bf16 1/(254 * 255) > 2^-16) of itself
// away from any half-integer, because 254 x and (2j + 1) a differ by a whole unit of
// x's mantissa; so the small cut moves no such quotient across a half, and it moves every
// tie to just below its half: toward zero.
template <int DT>
constexpr uint32_t kInfBits = DT == kDtF16 ? 0x7C00u : 0x7F80u;

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// The larger magnitude bits of two packed pairs (as integers: NaN above infinity above finite).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) {
    const u16x2_t a = __builtin_bit_cast(u16x2_t, m), b = __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

// What a row's codes need: one multiplier (and a power of two for rows of tiny values,
// whose reciprocal would overflow).
struct RowScale {
    float inv, pre, scale;
    bool bad;
};
template <int DT>
__device__ __forceinline__ RowScale row_scale(uint32_t abits) {
    RowScale r;
    r.bad = abits >= kInfBits<DT>;
    const float a = h16_to_f32<DT>(abits);
    r.scale = r.bad ? __builtin_nanf("") : a / 127.0f;
    r.pre = DT == kDtBf16 && a < 0x1p-100f ? 0x1p100f : 1.0f;   // exact: bf16 values are multiples of 2^-133
    r.inv = abits == 0u || r.bad ? 0.0f : 127.0f / (a * r.pre) * (1.0f - 0x1p-21f);
    return r;
}

// Codes of the 8 values of v; zero rows and rows that are not finite give 0 (inv = 0, and
// for the latter the value is replaced before the fma).
template <int DT>
__device__ __forceinline__ u32x2_t codes8(u32x4_t v, const RowScale& r) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = r.bad ? 0u : v[i];
        float lo = h16_to_f32<DT>(w & 0xFFFFu), hi = h16_to_f32<DT>(w >> 16);
        if (DT == kDtBf16) {
            lo *= r.pre;
            hi *= r.pre;
        }
        b[2 * i] = __float_as_uint(__builtin_fmaf(lo, r.inv, 12582912.0f));
        b[2 * i + 1] = __float_as_uint(__builtin_fmaf(hi, r.inv, 12582912.0f));
    }
    u32x2_t o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t p01 = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u);
        const uint32_t p23 = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000C0Cu);
        o[i] = p01 | p23;
    }
    return o;
}

// ---- sum sx sw in fp32: (sum sx) sw, in this order.
// Scales of bf16 rows reach from 2^-149 to 2^121, so the product of two may be subnormal, zero
// or infinite where the sum's is not.  A sum is zero or from 1 to 2^31 in size: sum sx does not
// fall below sx (and is exact while subnormal), but passes 2^128 where sx does not.  A token
// with such a scale takes 2^-32 of it, and the product 2^32 at the end.
constexpr float kLoudScale = 0x1p90f, kLoudDown = 0x1p-32f, kLoudUp = 0x1p32f;
__device__ __forceinline__ bool loud_scale(float sx) { return __builtin_fabsf(sx) > kLoudScale; }

qlora_status launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes, float* scale, int dt,
                                  hipStream_t s);
// launch_int8_quantize and t = RNE_16(s x A) [M, r] (1 <= r <= 128) in one launch
qlora_status launch_int8_prep(const uint16_t* x, const uint16_t* A, float s, int M, int K, int r, int8_t* codes,
                              float* scale, uint16_t* t, int dt, hipStream_t st);
// u = RNE_16(s dy B^T) [M, r] without split sums, where int8_u_supported
qlora_status launch_int8_u(const uint16_t* dy, const uint16_t* B, float s, int M, int N, int r, uint16_t* u, int dt,
                           hipStream_t st);
qlora_status launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t rows, int64_t cols, int dt,
                                    uint16_t* out, hipStream_t s);
// y = RNE_16(sx sw (xq wq^T) + t B); r == 0: no t B.  ws (nullable): int8_gemm_fwd_workspace
// bytes that need no clearing, with which small products split their reduction.
size_t int8_gemm_fwd_workspace(int64_t M, int64_t N, int64_t K);
qlora_status launch_int8_gemm_fwd(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                  const uint16_t* t, const uint16_t* B, uint16_t* y, int M, int N, int K, int r, int dt,
                                  void* ws, hipStream_t s);
// The forward for up to kInt8GemvMaxM tokens in one launch.  x 16-bit, quantized by the kernel
// (xq null; int8_gemv_quantizes says for which sizes), or its codes xq, sx; t given, or made
// from x (then not null) and A in the launch, with int8_gemv_workspace(r) bytes of workspace
// that need no clearing, and stored to t_out (nullable).
size_t int8_gemv_workspace(int r);
qlora_status launch_int8_gemv(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                              const uint16_t* t, const uint16_t* A, const uint16_t* B, float scale, uint16_t* y,
                              uint16_t* t_out, void* ws, int M, int N, int K, int r, int dt, hipStream_t s);
// dx = RNE_16(dy W_16 + u A^T); r == 0: no u A^T.  ws (nullable): int8_gemm_dx_workspace bytes
// that need no clearing, with which small products split their reduction.
size_t int8_gemm_dx_workspace(int64_t M, int64_t N, int64_t K);
qlora_status launch_int8_gemm_bwd_dx(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                     const uint16_t* A, uint16_t* dx, int M, int N, int K, int r, int dt, void* ws,
                                     hipStream_t s);

// LoRA gradients from 8-bit checkpoints: up to kInt8GradLayers layers (two contractions each)
// in one launch.  A contraction out[d, j] = sum_m X[m, d] S[m, j] takes codes with a scale per
// row (out [D, r]) or, scale null, 16-bit values (out [r, D]).  all_tiles is the number of
// 128-column tiles of the whole launch; the workspace of ws bytes needs no clearing.
constexpr int kInt8GradLayers = 8;
constexpr int kInt8GradChunk = 4096;   // rows per workgroup at most (their scales sit in LDS)
struct Int8GradPlan {
    int64_t tiles, splits, chunk;
    size_t ws_tags, ws;
};
Int8GradPlan plan_int8_grad(int64_t M, int64_t D, int r, int64_t all_tiles);
struct Int8GradDesc {
    const void* X;
    const float* scale;
    const uint16_t* S;
    float* out;
    void* ws;
    int M, D;
    Int8GradPlan plan;
};
qlora_status launch_int8_grads(const Int8GradDesc* d, int count, int r, int dt, hipStream_t s);

}  // namespace qlora
