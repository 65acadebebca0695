// Launchers and device helpers of the 8-bit float layer (e4m3 codes with a power-of-two scale
// for each block; declared in qlora.h, section "fp8").
#pragma once

#include "common.h"
#include "dropout.h"
#include "fp8_codes.h"
#include "fp8_plan.h"

namespace qlora {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x8_t __attribute__((ext_vector_type(8)));

// ---- quantization
// Rows: blocks of 1 x 128 of x [rows, cols] into codes with ld codes a row (ld >= cols; the ones
// past cols become 0) and scale bytes [ceil(cols / 128)][rs]; bytes of rows past the last: 0.
qlora_status launch_fp8_quantize_rows(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, int64_t ld,
                                      uint8_t* scale, int64_t rs, int dt, hipStream_t s);
// Weights: blocks of 128 x 128 of W [rows, cols]; scale bytes [ceil(rows / 128)][rs], bytes past
// the last block of a row of blocks: 0.
qlora_status launch_fp8_quantize_blocks(const uint16_t* W, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scale,
                                        int64_t rs, int dt, hipStream_t s);
qlora_status launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t cols, int64_t rs,
                                   bool by_rows, int dt, uint16_t* out, hipStream_t s);

// ---- preparation: the codes and scales of X [M, C] (as launch_fp8_quantize_rows) and out [M, r] =
// RNE_16(scale drop(X) Y) in one pass over X; Y [C, r] with y_natural, [r, C] otherwise (then
// nothing is dropped).  ws: fp8_prep_ws bytes that need no clearing.
size_t fp8_prep_ws(int64_t M, int64_t C, int r);
qlora_status launch_fp8_prep(const uint16_t* X, const uint16_t* Y, bool y_natural, const DropArgs& drop, float scale,
                             int M, int C, int r, uint8_t* codes, int64_t ld, uint8_t* sx, int64_t rs, uint16_t* out,
                             void* ws, int dt, hipStream_t s);

// ---- products.  Activations: codes with ld a row, scale bytes [block][rs].  Weight [N, K]: codes,
// scale bytes [ceil(N / 128)][wrs].
struct Fp8Gemm {
    const uint8_t* x;        // codes [M, ld]: of x (forward), of dy (input gradient)
    const uint8_t* sx;
    const uint8_t* w;
    const uint8_t* sw;
    const uint16_t* t;       // [M, r]: t, or u
    const uint16_t* L;       // B [r, N], or A [K, r]
    uint16_t* out;           // y [M, N], or dx [M, K]
    int M, N, K, r;
    int ld;                  // a multiple of 16
    int64_t rs, wrs;
    DropArgs drop;           // of t L (input gradient)
};
// ws (nullable): fp8_gemm_workspace bytes that need no clearing, with which small products
// split their reduction.
size_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K, bool dx);
qlora_status launch_fp8_gemm(const Fp8Gemm& g, bool dx, int dt, void* ws, hipStream_t s);

// The forward for up to kFp8GemvMaxM tokens in one launch (fp8_gemv_supported).  x 16-bit, quantized
// by the kernel (g.x null; fp8_gemv_quantizes says for which sizes), or its codes; t given (g.t),
// or made from x (then not null) and A in the launch, t = RNE_16(scale x A), with
// fp8_gemv_workspace(r) bytes of workspace that need no clearing, and stored to t_out (nullable).
size_t fp8_gemv_workspace(int r);
qlora_status launch_fp8_gemv(const Fp8Gemm& g, const uint16_t* x, const uint16_t* A, float scale, uint16_t* t_out,
                             void* ws, int dt, hipStream_t s);

}  // namespace qlora
