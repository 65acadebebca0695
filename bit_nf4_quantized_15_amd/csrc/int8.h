// Launchers and device helpers of the int8 layer (int8 codes with one fp32 scale per
// row; declared in qlora.h, section "int8").
#pragma once

#include "common.h"

namespace qlora {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// int32 sums of K products of codes stay below 2^31: 128 * 128 * (2^17 - 64) < 2^31.
constexpr int64_t kInt8MaxK = int64_t(1) << 17;

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

qlora_status launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes, float* scale, int dt,
                                  hipStream_t s);
qlora_status launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t rows, int64_t cols, int dt,
                                    uint16_t* out, hipStream_t s);
// y = RNE_16(sx sw (xq wq^T) + t B); r == 0: no t B
qlora_status launch_int8_gemm_fwd(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                  const uint16_t* t, const uint16_t* B, uint16_t* y, int M, int N, int K, int r, int dt,
                                  hipStream_t s);
// dx = RNE_16(dy W_16 + u A^T); r == 0: no u A^T
qlora_status launch_int8_gemm_bwd_dx(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                     const uint16_t* A, uint16_t* dx, int M, int N, int K, int r, int dt,
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
