// Tile loaders and MFMA helpers of the NF4 GEMMs (gemm.hip, gemm_dx_dropout.hip).
#pragma once

#include "common.h"
#include "dequant_tile.h"

namespace qlora {
namespace {

constexpr int kT = 256;             // lanes per workgroup
constexpr int kTM = 256;            // output rows per tile
constexpr int kTN = 256;            // output columns per tile
constexpr int kTK = 64;             // reduction step
constexpr int kTileBytes = kTM * kTK * 2;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4_t v) { return __builtin_bit_cast(bf16x8, v); }

// 32x32x16 MFMA on operands of the compute dtype DT (bf16 or fp16 bit patterns).
template <int DT>
__device__ __forceinline__ f32x16_t mfma32(bf16x8 a, bf16x8 b, f32x16_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Map a linear workgroup id to a tile id so that the workgroups placed on one
// XCD (ids are dealt round-robin over the 8 XCDs) get a contiguous run of
// tiles, i.e. share activation rows and weight columns in that XCD's L2.
__device__ __forceinline__ int xcd_tile(int bid, int total) {
    const int xcd = bid & 7, idx = bid >> 3;
    const int per = total >> 3, rem = total & 7;
    return xcd * per + min(xcd, rem) + idx;
}

// ---- activation tile loader: rows [row0, row0+256) x cols [col0, col0+64) of a
// row-major bf16 matrix with leading dimension ld; rows >= nrows and columns >=
// ncols read as 0.  Lane tid covers row tid/8 + 32p, chunk tid%8 (p = 0..7).
// VEC: ld % 8 == 0 and the base is 16-byte aligned, so whole chunks can be read.
template <bool VEC>
__device__ __forceinline__ void load_tile(u32x4_t (&r)[8], const uint16_t* __restrict__ src, int64_t ld,
                                          int row0, int nrows, int col0, int ncols, int tid) {
    const int lr = tid >> 3, lc = tid & 7;
    const int col = col0 + lc * 8;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int row = row0 + lr + 32 * p;
        if (VEC) {
            if (row < nrows && col < ncols) {
                r[p] = *reinterpret_cast<const u32x4_t*>(src + (int64_t)row * ld + col);
            } else {
                r[p] = u32x4_t{0u, 0u, 0u, 0u};
            }
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c0 = col + 2 * i;
                uint32_t lo = 0, hi = 0;
                if (row < nrows && c0 < ncols) lo = src[(int64_t)row * ld + c0];
                if (row < nrows && c0 + 1 < ncols) hi = src[(int64_t)row * ld + c0 + 1];
                w[i] = lo | (hi << 16);
            }
            r[p] = u32x4_t{w[0], w[1], w[2], w[3]};
        }
    }
}

// Branch-free variant for full-width column steps (col0 + 64 <= ld): rows past
// nrows re-read the last row; the outputs they feed are never stored.
template <bool VEC>
__device__ __forceinline__ void load_tile_clamped(u32x4_t (&r)[8], const uint16_t* __restrict__ src, int64_t ld,
                                                  int row0, int nrows, int col0, int tid) {
    if (!VEC) {
        load_tile<false>(r, src, ld, row0, nrows, col0, (int)ld, tid);
        return;
    }
    const int lr = tid >> 3, lc = tid & 7;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int row = min(row0 + lr + 32 * p, nrows - 1);
        r[p] = *reinterpret_cast<const u32x4_t*>(src + (int64_t)row * ld + col0 + lc * 8);
    }
}

// Forward-kernel tile layout: the XOR swizzle uses only row % 32, so the
// operand reads of rows R + 32 i (i = 0..3) differ by the immediate offset
// 4096 i; 8 or 16 consecutive rows still cover distinct banks.
__device__ __forceinline__ uint32_t ftile_off(int row, int chunk) {
    return (uint32_t)row * 128u + ((uint32_t)(chunk ^ ((row ^ (row >> 3)) & 3 ^ (row & 4))) << 4);
}

__device__ __forceinline__ void store_ftile(uint8_t* lds, const u32x4_t (&r)[8], int tid) {
    const int lr = tid >> 3, lc = tid & 7;
#pragma unroll
    for (int p = 0; p < 8; ++p) *reinterpret_cast<u32x4_t*>(lds + ftile_off(lr + 32 * p, lc)) = r[p];
}

// ---- direct HBM -> LDS tile loads (buffer_load_dwordx4 ... lds).  Lane l of
// an instruction writes 16 bytes at the instruction's LDS base + 16 l, so a
// wave fills 8 consecutive tile rows (1 KB); the swizzle is applied on the
// global side by choosing which 16-byte chunk each lane fetches.  Offsets past
// the buffer's byte range read as zero (rows past M): the range check applies
// to the lane's voffset, so every row offset is kept there.
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
__device__ void raw_buffer_load_lds(i32x4_t rsrc, __attribute__((address_space(3))) uint32_t* lds_ptr, int size,
                                    int voffset, int soffset, int offset, int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

__device__ __forceinline__ i32x4_t buffer_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4_t r;
    r[0] = (int32_t)(uint32_t)(a & 0xffffffffu);
    r[1] = (int32_t)(uint32_t)(a >> 32);   // stride 0
    r[2] = (int32_t)bytes;                 // num_records in bytes
    r[3] = 0x00020000;                     // gfx9 buffer format word
    return r;
}

// One 256 x 64 bf16 tile of a row-major matrix (row stride ld elements) whose
// row 0 is the buffer base: columns [col0, col0 + 64) into `tile` (ftile
// layout).  voff0 = this lane's byte offset of tile row 8*wave + lane/8, its
// logical chunk, column 0.
// An LDS pointer as the address_space(3) pointer the LDS builtins take.  The
// address-space cast keeps the pointer's origin, so the compiler can tell a
// direct load's destination from the tiles a step reads and waits only where
// they may overlap; a round trip through an integer would hide the origin and
// make every LDS read wait for every direct load in flight.
template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* as_lds(const void* p) {
    return (__attribute__((address_space(3))) T*)(p);
}

__device__ __forceinline__ void load_tile_direct(i32x4_t rs, uint8_t* tile, uint32_t voff0, int wave, int col0,
                                                 int64_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        auto* dst = as_lds<uint32_t>(tile + (32 * j + 8 * wave) * 128);
        // the row offset goes in voffset: the buffer range check covers voffset
        // (not soffset), so rows past the end of the buffer read as zero
        raw_buffer_load_lds(rs, dst, 16, (int)(voff0 + (uint32_t)(32 * j * ld * 2)), (int)(col0 * 2), 0, 0);
    }
}

__device__ __forceinline__ void wait_direct_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// In the backward's main loop a step issues the next tile's direct loads and
// then, pinned after them by a scheduling barrier, exactly N ordinary loads of
// codes and scales for two steps ahead.  Loads complete in order, so at most N loads
// in flight means the tile has landed while those N stay outstanding.
constexpr int kAllButVmem = 0x078F;  // sched_barrier mask: every class but VMEM may cross
template <int N>
__device__ __forceinline__ void wait_direct_loads_behind() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier that lets the last N LDS reads of the wave stay in flight
// (every earlier LDS access, reads and writes, has completed when it passes).
template <int N>
__device__ __forceinline__ void barrier_reads_in_flight() {
    asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store_tile(uint8_t* lds, const u32x4_t (&r)[8], int tid) {
    const int lr = tid >> 3, lc = tid & 7;
#pragma unroll
    for (int p = 0; p < 8; ++p) *reinterpret_cast<u32x4_t*>(lds + tile_off(lr + 32 * p, lc)) = r[p];
}

__device__ __forceinline__ bf16x8 lds_operand(const uint8_t* lds, int row, int chunk) {
    return *reinterpret_cast<const bf16x8*>(lds + tile_off(row, chunk));
}

// 8 bf16 from a strided column: src[(j0 + i) * ld + col], i = 0..7, zero when
// j0 + i >= jmax or col is out of range.
__device__ __forceinline__ bf16x8 gather8(const uint16_t* __restrict__ src, int64_t ld, int j0, int jmax, int col,
                                         bool col_ok) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ja = j0 + 2 * i, jb = ja + 1;
        const uint32_t lo = (col_ok && ja < jmax) ? src[(int64_t)ja * ld + col] : 0u;
        const uint32_t hi = (col_ok && jb < jmax) ? src[(int64_t)jb * ld + col] : 0u;
        w[i] = lo | (hi << 16);
    }
    return as_bf16x8(u32x4_t{w[0], w[1], w[2], w[3]});
}

// 8 contiguous bf16 src[row * ld + j0 .. +7], zero past jmax or an invalid row.
__device__ __forceinline__ bf16x8 row8(const uint16_t* __restrict__ src, int64_t ld, int row, bool row_ok, int j0,
                                      int jmax) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ja = j0 + 2 * i, jb = ja + 1;
        const uint32_t lo = (row_ok && ja < jmax) ? src[(int64_t)row * ld + ja] : 0u;
        const uint32_t hi = (row_ok && jb < jmax) ? src[(int64_t)row * ld + jb] : 0u;
        w[i] = lo | (hi << 16);
    }
    return as_bf16x8(u32x4_t{w[0], w[1], w[2], w[3]});
}

// Store an fp32 accumulator tile (this wave: 8 x 32-row tiles times 2 x 32-col
// tiles) as bf16.  Lane l of a 32x32 tile holds column l%32 and rows
// 8*(v/4) + 4*(l/32) + v%4 for v = 0..15.
template <int DT>
__device__ __forceinline__ void store_acc(uint16_t* __restrict__ out, int64_t ld, const f32x16_t (&acc)[8][2],
                                          int m0, int M, const int (&col)[2], const bool (&col_ok)[2], int h) {
    const int l32 = threadIdx.x & 31;
    (void)l32;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (!col_ok[t]) continue;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int m = m0 + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
                if (m < M) out[(int64_t)m * ld + col[t]] = (uint16_t)(pack2<DT>(acc[i][t][v], 0.0f) & 0xFFFFu);
            }
        }
    }
}

}  // namespace
}  // namespace qlora
