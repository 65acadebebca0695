// 8-bit float codes with a power-of-two scale for each block ("bitsandbytes deep dive",
// sections 5.1 and 8.2: blockwise scales, a low-bit storage format), and back.
//
//   e = least byte with max|x| <= 448 * 2^(e - 127),   code = RNE_e4m3(x / 2^(e - 127))
//
// Memory bound: x is read once and held in registers between the maximum and the codes.
//  - rows (blocks of 1 x 128): 16 lanes take a block, 16 bytes each; a workgroup takes 16 rows x
//    512 columns, so that the scale bytes of neighbouring rows, which lie side by side, are
//    written together and four blocks' loads are in flight.
//  - weights (128 x 128): a workgroup takes a block, 8 loads of 16 bytes in flight per lane.
// Traced, bf16 28672 x 8192: 147 us (4.8 TB/s read and written), and back 118 us (6.0 TB/s, of codes partly
// in the caches); 77 x 4096 rows: 3.3 and 2.7 us, a launch and one load's latency.
#include "fp8.h"

namespace qlora {
namespace {

// 8 values of a row at column c of `cols`, zero past them.
template <bool VEC>
__device__ __forceinline__ u32x4_t load8(const uint16_t* __restrict__ row, int64_t c, int64_t cols, bool on) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (VEC) {
        if (on && c < cols) v = *reinterpret_cast<const u32x4_t*>(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (on && c + e < cols) v[e >> 1] |= (uint32_t)row[c + e] << (16 * (e & 1));
    }
    return v;
}

constexpr int kRowsWg = 16, kBlocksWg = 4;

// VEC: cols % 8 == 0.  Codes are written up to ld (a multiple of 8), scale bytes up to rs.
template <bool VEC, int DT>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols,
                                                       uint8_t* __restrict__ codes, int64_t ld,
                                                       uint8_t* __restrict__ scale, int64_t rs, int64_t wgs_x) {
    const int64_t by = blockIdx.x / wgs_x, bx = blockIdx.x - by * wgs_x;
    const int64_t row = by * kRowsWg + (threadIdx.x >> 4), c0 = bx * kBlocksWg * kFp8Block + 8 * (threadIdx.x & 15);
    const bool on = row < rows;
    const uint16_t* xr = x + row * cols;
    u32x4_t v[kBlocksWg];
#pragma unroll
    for (int b = 0; b < kBlocksWg; ++b) v[b] = load8<VEC>(xr, c0 + b * kFp8Block, cols, on);
#pragma unroll
    for (int b = 0; b < kBlocksWg; ++b) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_mag2(m, v[b][i]);
        const uint32_t byte = fp8_scale_byte<DT>(max_row16(m));
        const int64_t c = c0 + b * kFp8Block;
        if (on && c < ld) *reinterpret_cast<u32x2_t*>(codes + row * ld + c) = fp8_codes8<DT>(v[b], byte);
        const int64_t block = bx * kBlocksWg + b;
        if ((threadIdx.x & 15) == 0 && block * kFp8Block < cols && row < rs)
            scale[block * rs + row] = on ? (uint8_t)byte : 0;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_blocks_kernel(const uint16_t* __restrict__ W, int64_t rows, int64_t cols,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scale,
                                                         int64_t rs, int64_t nbx) {
    __shared__ uint32_t am[4];
    const int64_t by = blockIdx.x / nbx, bx = blockIdx.x - by * nbx;
    const int64_t r0 = by * kFp8Block + (threadIdx.x >> 4), c = bx * kFp8Block + 8 * (threadIdx.x & 15);
    u32x4_t v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = load8<true>(W + (r0 + 16 * p) * cols, c, cols, r0 + 16 * p < rows);
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_mag2(m, v[p][i]);
    m = max_row16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 63) == 0) am[threadIdx.x >> 6] = m;
    __syncthreads();
    const uint32_t byte = fp8_scale_byte<DT>(max(max(am[0], am[1]), max(am[2], am[3])));
#pragma unroll
    for (int p = 0; p < 8; ++p)
        if (r0 + 16 * p < rows && c < cols)
            *reinterpret_cast<u32x2_t*>(codes + (r0 + 16 * p) * cols + c) = fp8_codes8<DT>(v[p], byte);
    if (threadIdx.x == 0) scale[by * rs + bx] = (uint8_t)byte;
    if (bx == nbx - 1 && bx + 1 + threadIdx.x < rs) scale[by * rs + bx + 1 + threadIdx.x] = 0;
}

// 16 codes a thread (cols % 64 == 0: within a block).
template <bool ROWS, int DT>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scale, int64_t count,
                                                             int64_t cols, int64_t rs, uint16_t* __restrict__ out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
    if (i >= count) return;
    const int64_t row = i / cols, b = (i - row * cols) >> 7;
    const uint32_t byte = ROWS ? scale[b * rs + row] : scale[(row >> 7) * rs + b];
    const float s = byte == kFp8Nan ? __builtin_nanf("") : fp8_scale_value(byte);
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(codes + i);
    u32x4_t o[2];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const f32x2_t lo = __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_pk_f32_fp8((int)q[w], false));
        const f32x2_t hi = __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_pk_f32_fp8((int)q[w], true));
        o[w >> 1][2 * (w & 1)] = pack2<DT>(lo[0] * s, lo[1] * s);
        o[w >> 1][2 * (w & 1) + 1] = pack2<DT>(hi[0] * s, hi[1] * s);
    }
    *reinterpret_cast<u32x4_t*>(out + i) = o[0];
    *reinterpret_cast<u32x4_t*>(out + i + 8) = o[1];
}

}  // namespace

qlora_status launch_fp8_quantize_rows(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, int64_t ld,
                                      uint8_t* scale, int64_t rs, int dt, hipStream_t s) {
    const int64_t wgs_x = (fp8_blocks(cols) + kBlocksWg - 1) / kBlocksWg, wgs = wgs_x * ((rows + kRowsWg - 1) / kRowsWg);
    if (wgs * 256 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    const bool vec = cols % 8 == 0;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        if (vec)
            hipLaunchKernelGGL((fp8_rows_kernel<true, DT>), dim3((unsigned)wgs), dim3(256), 0, s, x, rows, cols, codes, ld,
                               scale, rs, wgs_x);
        else
            hipLaunchKernelGGL((fp8_rows_kernel<false, DT>), dim3((unsigned)wgs), dim3(256), 0, s, x, rows, cols, codes,
                               ld, scale, rs, wgs_x);
    });
    return launch_status();
}

qlora_status launch_fp8_quantize_blocks(const uint16_t* W, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scale,
                                        int64_t rs, int dt, hipStream_t s) {
    const int64_t nbx = fp8_blocks(cols), wgs = nbx * fp8_blocks(rows);
    if (wgs * 256 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        hipLaunchKernelGGL((fp8_blocks_kernel<DT>), dim3((unsigned)wgs), dim3(256), 0, s, W, rows, cols, codes, scale, rs,
                           nbx);
    });
    return launch_status();
}

qlora_status launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t cols, int64_t rs,
                                   bool by_rows, int dt, uint16_t* out, hipStream_t s) {
    const int64_t count = rows * cols, wgs = (count / 16 + 255) / 256;
    if (wgs * 256 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        if (by_rows)
            hipLaunchKernelGGL((fp8_dequantize_kernel<true, DT>), dim3((unsigned)wgs), dim3(256), 0, s, codes, scale, count,
                               cols, rs, out);
        else
            hipLaunchKernelGGL((fp8_dequantize_kernel<false, DT>), dim3((unsigned)wgs), dim3(256), 0, s, codes, scale,
                               count, cols, rs, out);
    });
    return launch_status();
}

}  // namespace qlora
