// int8 codes with one fp32 scale per row, and the 16-bit values back from them
// ("bitsandbytes deep dive", section 4: absmax int8, one scale per row).
// The rounding of a code is decided as int8.h shows.
#include "int8.h"

namespace qlora {
namespace {

constexpr int kQT = 256;   // lanes per workgroup

// A row's largest magnitude bits over the W waves that share it.
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
    uint32_t a = max(m & 0xFFFFu, m >> 16);
#pragma unroll
    for (int d = 32; d; d >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, d));
    if (W > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) a = max(a, red[w]);
    }
    return a;
}

// Rows of up to 512 W C values: W waves hold a row in registers, C 16-byte chunks per lane,
// so x is read once (HBM bound: one pass in, half of it out).  8192 x 28672, traced: 133 us where
// x is another each time, 5.3 TB/s (147 where it is the same; a kernel that read the row twice
// took 182); 77 x 4096: 3.1 us, a launch and one row's latency.
template <int W, int C, int DT>
__global__ __launch_bounds__(kQT) void int8_quantize_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                            int8_t* __restrict__ codes, float* __restrict__ scale) {
    constexpr int kPer = kQT / 64 / W;   // rows per workgroup
    __shared__ uint32_t red[2][kQT / 64];
    const int lane = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W), nch = cols >> 3;
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * kPer; base < rows; base += (int64_t)gridDim.x * kPer, turn ^= 1) {
        const int64_t row = base + sub;
        const bool on = row < rows;
        const u32x4_t* xr = reinterpret_cast<const u32x4_t*>(x + (on ? row : rows - 1) * cols);
        u32x4_t v[C];
#pragma unroll
        for (int e = 0; e < C; ++e) v[e] = xr[min(lane + 64 * W * e, nch - 1)];   // (the last chunk again)
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < C; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_abs2(m, v[e][i]);
        // two buffers: a wave may be a row ahead of one that still reads
        const RowScale r = row_scale<DT>(row_max<W>(m, red[turn]));
        if (!on) continue;
        if (lane == 0) scale[row] = r.scale;
        u32x2_t* cr = reinterpret_cast<u32x2_t*>(codes + row * cols);
#pragma unroll
        for (int e = 0; e < C; ++e) {
            const int c = lane + 64 * W * e;
            if (c < nch) cr[c] = codes8<DT>(v[e], r);
        }
    }
}

// Longer rows: one workgroup per row, two passes over it.
template <int DT>
__global__ __launch_bounds__(kQT) void int8_quantize_long_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                                 int8_t* __restrict__ codes, float* __restrict__ scale) {
    __shared__ uint32_t red[2][kQT / 64];
    const int tid = threadIdx.x, nch = cols >> 3;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        const u32x4_t* xr = reinterpret_cast<const u32x4_t*>(x + row * cols);
        u32x2_t* cr = reinterpret_cast<u32x2_t*>(codes + row * cols);
        uint32_t m = 0;
        for (int c = tid; c < nch; c += kQT) {
            const u32x4_t v = xr[c];
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_abs2(m, v[i]);
        }
        const RowScale r = row_scale<DT>(row_max<kQT / 64>(m, red[turn]));
        if (tid == 0) scale[row] = r.scale;
        for (int c = tid; c < nch; c += kQT) cr[c] = codes8<DT>(xr[c], r);
    }
}

// HBM bound (8192 x 28672, traced: 139 us, 5.1 TB/s).  16 codes per lane; `base` counts 16-code chunks of the whole tensor.
constexpr int kDqPer = 1024;  // chunks per workgroup
template <int DT>
__global__ __launch_bounds__(256) void int8_dequantize_kernel(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scale, int64_t rows, int cols,
                                                              uint16_t* __restrict__ out) {
    const uint32_t cpr = (uint32_t)cols >> 4;
    const int64_t base = (int64_t)blockIdx.x * kDqPer;
    const int64_t row0 = base / cpr;
    const uint32_t rem = (uint32_t)(base - row0 * cpr);
#pragma unroll
    for (int e = 0; e < kDqPer / 256; ++e) {
        const uint32_t i = rem + (uint32_t)(threadIdx.x + 256 * e);
        const int64_t row = row0 + i / cpr;
        if (row >= rows) continue;
        const int64_t chunk = base + threadIdx.x + 256 * e;
        const u32x4_t c = reinterpret_cast<const u32x4_t*>(codes)[chunk];
        const float s = scale[row];
        u32x4_t o[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u32x2_t v = int8_values4<DT>(c[j], s);
            o[j >> 1][2 * (j & 1)] = v[0];
            o[j >> 1][2 * (j & 1) + 1] = v[1];
        }
        u32x4_t* dst = reinterpret_cast<u32x4_t*>(out) + 2 * chunk;
        dst[0] = o[0];
        dst[1] = o[1];
    }
}

}  // namespace

qlora_status launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes, float* scale, int dt,
                                  hipStream_t s) {
    const int nch = (int)(cols >> 3);
    const unsigned grid4 = (unsigned)std::min<int64_t>((rows + 3) / 4, 1 << 20);   // four rows per workgroup
    const unsigned grid1 = (unsigned)std::min<int64_t>(rows, 1 << 20);
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_Q(W, C) \
    hipLaunchKernelGGL((int8_quantize_kernel<W, C, DT>), dim3(W == 1 ? grid4 : grid1), dim3(kQT), 0, s, x, rows, \
                       (int)cols, codes, scale)
        if (nch <= 64) QL_Q(1, 1);
        else if (nch <= 256) QL_Q(1, 4);
        else if (nch <= 512) QL_Q(4, 2);
        else if (nch <= 1024) QL_Q(4, 4);
        else if (nch <= 2048) QL_Q(4, 8);
        else if (nch <= 4096) QL_Q(4, 16);
        else
            hipLaunchKernelGGL(int8_quantize_long_kernel<DT>, dim3(grid1), dim3(kQT), 0, s, x, rows, (int)cols, codes,
                               scale);
#undef QL_Q
    });
    return launch_status();
}

qlora_status launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t rows, int64_t cols, int dt,
                                    uint16_t* out, hipStream_t s) {
    const int64_t wgs = (rows * (cols >> 4) + kDqPer - 1) / kDqPer;
    if (wgs >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        hipLaunchKernelGGL(int8_dequantize_kernel<DT>, dim3((unsigned)wgs), dim3(256), 0, s, codes, scale, rows,
                           (int)cols, out);
    });
    return launch_status();
}

}  // namespace qlora
