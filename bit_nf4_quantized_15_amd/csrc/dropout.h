// Dropout of the LoRA branch's input ("bitsandbytes deep dive", section 12: LoraConfig's
// lora_dropout), with a mask that is never stored: every kernel that needs mask[m, k]
// makes it again from (seed, offset, m, k / 8).
//
// The generator is Philox-4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011; the fewest rounds of theirs that pass
// their statistical tests).  One call gives 128 bits, 16 for each of 8 consecutive columns
// of a row: the 8 values of a 16-byte load.  A value is kept when its 16 bits are at least
// thr = round(65536 p); kept values count 1 / (1 - thr / 65536) times, as a factor of fp32
// sums, so no 16-bit value is rounded for it.  14 32 x 32 -> 64-bit products per 8 values:
// 0.6 cycles of a SIMD per value.
#pragma once

#include "common.h"

namespace qlora {

struct DropArgs {
    uint32_t k0, k1, o0, o1;   // seed and offset, low words first
    uint32_t thr;              // 0: nothing is dropped
    float inv;                 // 1 / (1 - p)
};

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;
constexpr int kPhiloxRounds = 7;

// The words of columns 8 group .. 8 group + 7 of row m: two columns each, the lower one in
// bits 15..0.
__device__ __forceinline__ u32x4_t drop_words(const DropArgs& d, uint32_t group, uint32_t m) {
    uint32_t c0 = group, c1 = m, c2 = d.o0, c3 = d.o1, k0 = d.k0, k1 = d.k1;
#pragma unroll
    for (int i = 0; i < kPhiloxRounds; ++i) {
        const uint64_t a = (uint64_t)c0 * kPhiloxM0, b = (uint64_t)c2 * kPhiloxM1;
        c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(b >> 32), c1, k0, 0x96);   // (xor of three)
        c1 = (uint32_t)b;
        c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(a >> 32), c3, k1, 0x96);
        c3 = (uint32_t)a;
        k0 += kPhiloxW0;
        k1 += kPhiloxW1;
    }
    return u32x4_t{c0, c1, c2, c3};
}

// All ones in the halves of w that are dropped: the sign of (w - 2^15) - (thr - 2^15), subtracted
// with saturation as signed 16-bit numbers.
__device__ __forceinline__ uint32_t dropped_halves(uint32_t w, uint32_t thr) {
    typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
    const uint32_t t = (thr | (thr << 16)) ^ 0x80008000u;
    const i16x2 d = __builtin_elementwise_sub_sat(__builtin_bit_cast(i16x2, w ^ 0x80008000u), __builtin_bit_cast(i16x2, t));
    return __builtin_bit_cast(uint32_t, (i16x2)(d >> (int16_t)15));
}

// 8 consecutive 16-bit values of row m with the dropped ones zero.
__device__ __forceinline__ u32x4_t drop8(u32x4_t v, const DropArgs& d, uint32_t group, uint32_t m) {
    const u32x4_t w = drop_words(d, group, m);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= ~dropped_halves(w[i], d.thr);
    return v;
}

// drop() of a 32 x 32 MFMA tile whose lane (h, l32) holds, of row m = its token, the columns
// col0 + 8 (v / 4) + 4 h + v % 4.  Each half of the wave makes the words of two of the four
// groups of 8 columns and hands the other half its four.
__device__ __forceinline__ void drop_tile(f32x16_t& f, const DropArgs& d, uint32_t m, uint32_t col0, int h) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const u32x4_t w = drop_words(d, (col0 >> 3) + (uint32_t)(p + 2 * h), m);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // [0]: columns 2 e, 2 e + 1 of the lane's four in group p, [1]: in group p + 2
            const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w[e], w[2 + e], false, false));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float& lo = reinterpret_cast<float*>(&f)[4 * (p + 2 * g) + 2 * e];
                float& hi = reinterpret_cast<float*>(&f)[4 * (p + 2 * g) + 2 * e + 1];
                lo = (s[g] & 0xFFFFu) >= d.thr ? lo * d.inv : 0.0f;
                hi = (s[g] >> 16) >= d.thr ? hi * d.inv : 0.0f;
            }
        }
    }
}

// drop() of a 32 x 32 MFMA tile whose lane (h, l32) holds column col0 + l32 of the rows
// m0 + 8 (v / 4) + 4 h + v % 4.  Lane L makes half of row L % 32's bits; the whole word then
// comes from the row's lane.
__device__ __forceinline__ void drop_tile_rows(f32x16_t& f, const DropArgs& d, uint32_t m0, uint32_t col0, int lane) {
    const int h = lane >> 5, l32 = lane & 31;
    uint32_t bits = 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const u32x4_t w = drop_words(d, (col0 >> 3) + (uint32_t)(2 * h + p), m0 + (uint32_t)l32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bits |= (uint32_t)((w[i] & 0xFFFFu) >= d.thr) << (16 * h + 8 * p + 2 * i);
            bits |= (uint32_t)((w[i] >> 16) >= d.thr) << (16 * h + 8 * p + 2 * i + 1);
        }
    }
    bits |= (uint32_t)__shfl_xor((int)bits, 32);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const uint32_t row = (uint32_t)__shfl((int)bits, 8 * (v >> 2) + 4 * h + (v & 3));
        f[v] = (row >> l32) & 1u ? f[v] * d.inv : 0.0f;
    }
}

// Host side: the generator's arguments; false for a p outside [0, 1) (after its rounding to
// multiples of 2^-16 too).  A null d drops nothing.
bool drop_args(const qlora_dropout* d, DropArgs* out);

// launch_nt_batch (Y natural) with drop[i] (thr > 0) on X of product i
qlora_status launch_nt_batch_dropout(const NtDesc* d, const DropArgs* drop, int count, int r, int dt, hipStream_t s);
// The gradients of layers that drop something: dA = drop(X)^T S into out [D, r], or (dA 0) dB = S^T X into
// out [r, D]; D below kGradMaxWidth.  ws: tn_ws_bytes(M, D, r) bytes that need no clearing.
struct GradDropDesc {
    const uint16_t* X;
    const uint16_t* S;
    void* ws;
    float* out;
    DropArgs drop;
    int M, D, dA;
};
qlora_status launch_grads_dropout(const GradDropDesc* d, int count, int r, int dt, hipStream_t s);
// launch_gemm_bwd_dx and the int8 product with drop (thr > 0) on u A^T
qlora_status launch_gemm_bwd_dx_dropout(const uint16_t* dy, const uint8_t* codes, const uint8_t* q8, const float* a2,
                                        int cb, int dt, const uint16_t* u, const uint16_t* A, const DropArgs& drop,
                                        uint16_t* dx, int M, int N, int K, int r, hipStream_t s);
qlora_status launch_int8_gemm_bwd_dx_dropout(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                             const uint16_t* A, const DropArgs& drop, uint16_t* dx, int M, int N, int K,
                                             int r, int dt, void* ws, hipStream_t s);

}  // namespace qlora
