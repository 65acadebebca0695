// What the int8 forward needs of x, in one launch: its codes and scales, and the LoRA
// branch's t = RNE_16(s x A) ("bitsandbytes deep dive", section 4: absmax int8 per row;
// 12.2: the LoRA side path).
//
// A workgroup of 8 waves takes 2 to 32 tokens over all of K, so t needs no split sums and a
// row's maximum no second launch; its waves deal the 64-wide steps of K round robin.  Pass 1
// reads x as MFMA operands (a lane: 16 values of one token), keeps the maxima, and multiplies
// with A, of which each wave copies its 64 rows (one contiguous run) through LDS of its own
// and reads them down their columns.  Pass 2 reads the rows again (L2) and writes codes.
// Bound by A from L2 (2 K r bytes per workgroup) and, above some thousand tokens, by x; traced:
// 2048 x 4096, r = 64: 15 us; 8192 x 8192, r = 64: 74 us, 2.7 TB/s of x and codes.
//
// t is rounded to 16 bits, also where the caller keeps none: the products t B and t^T dy take
// it as a 16-bit MFMA operand, and y is the same whether t is kept or not.  An fp32 t would
// take a second operand for its low bits.
#include "int8.h"

namespace qlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
constexpr uint32_t kNone = 0x80000000u;   // past every buffer here: reads zero

template <int DT>
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

constexpr int kWaves = 8, kThreads = 512;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* as_lds(const void* p) {
    return (__attribute__((address_space(3))) T*)(p);
}

// LDS of a kernel: each wave's 64 rows of A (rows of 16 TQ + 16 halves: the four rows of a
// transposed read lie on different banks), or afterwards the waves' sums.
template <int TQ, int NR>
constexpr int prep_lds() {
    constexpr int a = kWaves * 64 * (16 * TQ + 16) * 2, s = kWaves * TQ * NR * 64 * 16;
    return a > s ? a : s;
}

// TQ: groups of 16 ranks (1, 2, 4, 8); NR: groups of 16 tokens; VEC: r % 8 == 0.
template <int TQ, int NR, bool VEC, int DT>
__global__ __launch_bounds__(kThreads, 2) void int8_prep_kernel(const uint16_t* __restrict__ x,
                                                                const uint16_t* __restrict__ A, float s, int M, int K,
                                                                int r, int per, int8_t* __restrict__ codes,
                                                                float* __restrict__ scale, uint16_t* __restrict__ t) {
    constexpr int kLd = 16 * TQ + 16, kAL = 2 * TQ;        // halves of a staged row of A; 16-byte loads per lane
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t am[kWaves][16 * NR];
    __shared__ RowScale rs[16 * NR];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * per;
    const int rows = (int)min((int64_t)per, M - m0), KS = K >> 6;
    const rsrc_t xrs = buf_rsrc(x + m0 * K, (uint64_t)rows * K * 2);
    const rsrc_t ars = buf_rsrc(A, (uint64_t)K * r * 2);
    const uint32_t xoff = (uint32_t)i * (uint32_t)K * 2u + 32u * g;
    uint16_t* const slice = reinterpret_cast<uint16_t*>(lds) + wave * 64 * kLd;
    uint32_t put[VEC ? kAL : 1];                            // where a lane's 8 ranks go in LDS
    if (VEC)
#pragma unroll
        for (int e = 0; e < kAL; ++e) {
            const int c = lane + 64 * e, per = r >> 3;
            put[VEC ? e : 0] = (uint32_t)((c / per) * kLd + 8 * (c % per));
        }

    struct Step {
        u32x4_t x[NR][2], a[kAL];
    };
    auto load = [&](Step& q, int st) __attribute__((always_inline)) {
        const bool on = st < KS;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)   // (rows past the last lie past the buffer)
                q.x[n][c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                    xrs, on ? xoff + (uint32_t)(16 * n) * (uint32_t)K * 2u + 128u * (uint32_t)st + 16u * c : kNone, 0, 0));
        // rows 64 st .. of A: 128 r consecutive bytes
#pragma unroll
        for (int e = 0; e < kAL; ++e)
            q.a[e] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                ars, (on & (lane + 64 * e < 8 * r)) ? (uint32_t)st * 128u * (uint32_t)r + 16u * (uint32_t)(lane + 64 * e) : kNone,
                0, 0));
    };
    auto stage = [&](const Step& q) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < kAL; ++e) {
            if (VEC) {
                if (8 * e < r) *reinterpret_cast<u32x4_t*>(slice + put[VEC ? e : 0]) = q.a[e];
            } else if (lane + 64 * e < 8 * r) {
                int row = 8 * (lane + 64 * e) / r, col = 8 * (lane + 64 * e) - row * r;
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    slice[row * kLd + col] = (uint16_t)(q.a[e][h >> 1] >> (16 * (h & 1)));
                    if (++col == r) {
                        col = 0;
                        ++row;
                    }
                }
            }
        }
    };
    f32x4_t acc[TQ][NR];
    uint32_t top[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        top[n] = 0;
#pragma unroll
        for (int c = 0; c < TQ; ++c) acc[c][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto use = [&](const Step& q) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int w = 0; w < 4; ++w) top[n] = max_abs2(top[n], q.x[n][c][w]);
        // lane (g, i): ranks 16 c + i of rows 16 g + 8 half .. + 7, the k of its x values
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int c = 0; c < TQ; ++c) {
                const uint16_t* p = slice + (16 * g + 8 * half + (i >> 2)) * kLd + 16 * c + 4 * (i & 3);
                const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p));
                const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p + 4 * kLd));
                const u32x4_t w = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[c][n] = mfma16<DT>(w, q.x[n][half], acc[c][n]);
            }
    };
    // (a wave's LDS accesses complete in order and its slice is its own: no barrier)
    constexpr int P = TQ <= 2 ? 4 : 2;                      // steps in flight
    Step ring[P];
#pragma unroll
    for (int p = 0; p < P - 1; ++p) load(ring[p], wave + kWaves * p);
    for (int st = wave; st < KS; st += P * kWaves) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (p > 0 && st + kWaves * p >= KS) break;
            load(ring[(p + P - 1) % P], st + kWaves * (p + P - 1));
            stage(ring[p]);
            use(ring[p]);
        }
    }

    // ---- add the waves
    __syncthreads();
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);   // [wave][c][n][lane]
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        uint32_t m = max(top[n] & 0xFFFFu, top[n] >> 16);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lane < 16) am[wave][16 * n + lane] = m;
#pragma unroll
        for (int c = 0; c < TQ; ++c) red[((wave * TQ + c) * NR + n) * 64 + lane] = acc[c][n];
    }
    __syncthreads();
    if (tid < 16 * NR) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = max(m, am[w][tid]);
        rs[tid] = row_scale<DT>(m);
        if (tid < rows) scale[m0 + tid] = rs[tid].scale;
    }
    for (int v = tid; v < TQ * NR * 64; v += kThreads) {
        const int l = v & 63, n = (v >> 6) % NR, c = (v >> 6) / NR;
        f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const f32x4_t z = red[((w * TQ + c) * NR + n) * 64 + l];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += z[e];
        }
        const int m = 16 * n + (l & 15);
        if (m < rows)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * c + 4 * (l >> 4) + e;
                if (j < r) t[(m0 + m) * r + j] = (uint16_t)(pack2<DT>(s * sum[e], 0.0f) & 0xFFFFu);
            }
    }
    __syncthreads();

    // ---- codes
    const int nch = K >> 3;
    for (int row = wave; row < rows; row += kWaves) {
        const RowScale q = rs[row];
        const u32x4_t* xr = reinterpret_cast<const u32x4_t*>(x + (m0 + row) * K);
        u32x2_t* cr = reinterpret_cast<u32x2_t*>(codes + (m0 + row) * K);
        for (int c = lane; c < nch; c += 64 * 8) {
            u32x4_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = xr[min(c + 64 * e, nch - 1)];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + 64 * e < nch) cr[c + 64 * e] = codes8<DT>(v[e], q);
        }
    }
}

// The same for the backward's u = RNE_16(s dy B^T) [M, r]: B [r, N] has consecutive n in its
// rows, so its operands come straight from memory, and there are no codes.  N % 8 == 0.
template <int TQ, int DT>
__global__ __launch_bounds__(kThreads, 2) void int8_u_kernel(const uint16_t* __restrict__ dy,
                                                             const uint16_t* __restrict__ B, float s, int M, int N,
                                                             int r, int per, uint16_t* __restrict__ u) {
    __shared__ __attribute__((aligned(16))) f32x4_t red[kWaves * TQ * 64];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * per;
    const int rows = (int)min((int64_t)per, M - m0), steps = (N + 63) >> 6;
    const rsrc_t drs = buf_rsrc(dy + m0 * N, (uint64_t)rows * N * 2);
    const rsrc_t brs = buf_rsrc(B, (uint64_t)r * N * 2);
    struct Step {
        u32x4_t x[2], b[TQ][2];
    };
    auto load = [&](Step& q, int st) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int n = 64 * st + 16 * g + 8 * c;
            const bool on = n < N;                          // (columns past N would be the next row's)
            q.x[c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                drs, on ? ((uint32_t)i * (uint32_t)N + (uint32_t)n) * 2u : kNone, 0, 0));
#pragma unroll
            for (int t = 0; t < TQ; ++t)                    // (rows past r lie past the buffer)
                q.b[t][c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                    brs, on ? ((uint32_t)(16 * t + i) * (uint32_t)N + (uint32_t)n) * 2u : kNone, 0, 0));
        }
    };
    f32x4_t acc[TQ];
#pragma unroll
    for (int t = 0; t < TQ; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int P = TQ <= 4 ? 4 : 2;                      // steps in flight
    Step ring[P];
#pragma unroll
    for (int p = 0; p < P - 1; ++p) load(ring[p], wave + kWaves * p);
    for (int st = wave; st < steps; st += P * kWaves) {     // steps past N multiply zeros
#pragma unroll
        for (int p = 0; p < P; ++p) {
            load(ring[(p + P - 1) % P], st + kWaves * (p + P - 1));
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int t = 0; t < TQ; ++t) acc[t] = mfma16<DT>(ring[p].b[t][c], ring[p].x[c], acc[t]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int t = 0; t < TQ; ++t) red[(wave * TQ + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int v = tid; v < TQ * 64; v += kThreads) {
        const int l = v & 63, t = v >> 6, m = l & 15;
        f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const f32x4_t z = red[(w * TQ + t) * 64 + l];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += z[e];
        }
        if (m < rows)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * t + 4 * (l >> 4) + e;
                if (j < r) u[(m0 + m) * r + j] = (uint16_t)(pack2<DT>(s * sum[e], 0.0f) & 0xFFFFu);
            }
    }
}

}  // namespace

qlora_status launch_int8_u(const uint16_t* dy, const uint16_t* B, float s, int M, int N, int r, uint16_t* u, int dt,
                           hipStream_t st) {
    const int per = int8_rows_per_wg(M);
    const int64_t grid = ((int64_t)M + per - 1) / per;
    if (grid * kThreads >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_U(TQ) \
    hipLaunchKernelGGL((int8_u_kernel<TQ, DT>), dim3((unsigned)grid), dim3(kThreads), 0, st, dy, B, s, M, N, r, per, u)
        if (r <= 16) QL_U(1);
        else if (r <= 32) QL_U(2);
        else if (r <= 64) QL_U(4);
        else QL_U(8);
#undef QL_U
    });
    return launch_status();
}

qlora_status launch_int8_prep(const uint16_t* x, const uint16_t* A, float s, int M, int K, int r, int8_t* codes,
                              float* scale, uint16_t* t, int dt, hipStream_t st) {
    // (K < 131072: a row group's and A's offsets fit 31 bits)
    const int tq = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
    const bool vec = r % 8 == 0;
    const int per = int8_prep_rows(M, r), nr = per == 32 ? 2 : 1;
    const int64_t grid = ((int64_t)M + per - 1) / per;
    if (grid * kThreads >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_P(TQ, NR, V)                                                                                           \
    hipLaunchKernelGGL((int8_prep_kernel<TQ, NR, V, DT>), dim3((unsigned)grid), dim3(kThreads), (prep_lds<TQ, NR>()), st, x, \
                       A, s, M, K, r, per, codes, scale, t)
#define QL_P1(TQ)                                                        \
    if (nr == 2) { if (vec) QL_P(TQ, 2, true); else QL_P(TQ, 2, false); } \
    else { if (vec) QL_P(TQ, 1, true); else QL_P(TQ, 1, false); }
        switch (tq) {
            case 1: QL_P1(1) break;
            case 2: QL_P1(2) break;
            case 4: QL_P1(4) break;
            default: if (vec) QL_P(8, 1, true); else QL_P(8, 1, false); break;
        }
#undef QL_P1
#undef QL_P
    });
    return launch_status();
}

}  // namespace qlora
