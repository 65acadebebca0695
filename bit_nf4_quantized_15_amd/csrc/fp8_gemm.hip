// Products of the 8-bit float layer on MFMA (v_mfma_scale_f32_32x32x64_f8f6f4), gfx950:
//
//   forward         y[m,n]  = RNE_16( sum_k xq[m,k] wq[n,k] + sum_j t[m,j] B[j,n] )
//   input gradient  dx[m,k] = RNE_16( sum_n dyq[m,n] wq[n,k] + drop( sum_j u[m,j] A[k,j] ) )
//
// ("bitsandbytes deep dive", section 8.2: low-bit storage; 8.6 / 12.4: the LoRA branch and the
// frozen base's backward.)  A value is an e4m3 code times the power of two of its block, 1 x 128
// of the activations and 128 x 128 of the weight.  A reduction step is 128 deep, one block of
// both, and the matrix unit multiplies by the two scales itself: the accumulators are the
// result, with no work per block and no epilogue for scales.
//
// The weight's blocks are square, so both products read the one stored weight: the forward
// copies rows n (consecutive k are an operand), the input gradient rows n of a k range, which
// gfx950's transposed byte read (ds_read_b64_tr_b8) turns into operands of consecutive n.
// Tiles are copied HBM -> LDS by direct loads, 16 bytes per lane, XOR-swizzled on the global
// side; the scale bytes of a step travel with its tiles.
//
// Numbers: products of codes are exact and 8 of them are added in the matrix unit with what
// lies 13 bits or more below the largest cut off (measured; on normal data the sum of 4096
// products is 1.6e-5 off in the norm, without bias: a tenth of what rounding to fp16 does);
// the sums of 8 are accumulated in fp32.  The 16-bit matrix unit would keep every bit at half
// the rate.
//
// Bound by the MFMAs and the power they draw (from registers alone the chip reaches 4.0 PFLOP/s).
// 8192 x 28672 x 8192, us: 1285 to 1360 for given codes, r = 0 (3.0 PFLOP/s; a library product of
// these sizes without the blocks' scales 1331), 1570 to 1640 traced with the LoRA term behind the
// preparation.  Input gradient 4096 x 11008 -> 4096, r = 64, dropout 0.05, traced: 150, one round of 256
// tiles (2.5 PFLOP/s), of which the epilogue's masks are 5.  Ragged: 333 x 11008 -> 4096, r = 8: 28
// (split in two); input gradient 777 x 11000 -> 4096, r = 24: 46 (224 of 256 CUs).
// The 256 x 256 input gradient with dropout keeps 260 bytes a lane in scratch memory while its
// epilogue makes masks: outside the main loop, and less than a second pass over the tile would cost.
#include <algorithm>

#include "fp8.h"
#include "split_sync.h"

namespace qlora {

__device__ void raw_buffer_load_lds(i32x4_t rsrc, __attribute__((address_space(3))) uint32_t* lds_ptr, int size,
                                    int voffset, int soffset, int offset, int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

template <int DT>
__device__ __forceinline__ f32x16_t mfma16(u32x4_t a, u32x4_t b, f32x16_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
// (uniform: no loop over lanes around the loads)
__device__ __forceinline__ i32x4_t buffer_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return i32x4_t{__builtin_amdgcn_readfirstlane((int32_t)(uint32_t)a),
                   __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)(a >> 32)),
                   __builtin_amdgcn_readfirstlane((int32_t)bytes), 0x00020000};
}
constexpr uint32_t kNone = 0x80000000u;   // past every buffer here: reads zero, stores nothing

// The cast keeps the pointer's origin, so that the compiler can tell a direct load's
// destination from the buffers a step reads (each ring slot is an object of its own).
template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* as_lds(const void* p) {
    return (__attribute__((address_space(3))) T*)(p);
}

// 8 values p[0 .. 7] of a row of which `left` are left, zero past them.
__device__ __forceinline__ u32x4_t load8(const uint16_t* __restrict__ p, int left) {
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

constexpr int kStep = kFp8Block;   // depth of a step: one block of the reduction

// Byte of 16-byte chunk c of row `row` of a tile with 128-byte rows: any 16 consecutive rows of
// one chunk cover all 64 banks.
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ uint32_t tile_byte(int row, int c) {
    return (uint32_t)row * 128u + ((uint32_t)(c ^ swizzle(row)) << 4);
}
// The input gradient's weight tile: 128 rows of BN bytes; the 8 rows x 32 columns that two lane
// groups read together lie on different banks.
template <int BN>
__device__ __forceinline__ int code_chunk(int row, int c) {
    return BN >= 256 ? c ^ ((row & 7) << 1) : BN == 128 ? c ^ (((row >> 1) & 3) << 1) : c ^ (((row >> 2) & 1) << 1);
}

// Tiles in groups of `gm` row tiles, down the rows first: 32 consecutive tiles (one XCD's
// CUs at a time) then form a block of gm x 32 / gm that shares panels in the XCD's L2.
struct TileMap {
    int tm, tn, gm;
    int splits, per;      // the reduction in `splits` parts of `per` steps
    uint64_t* tags;       // [tile][split]
    uint8_t* part;        // [split][tile]: the fp32 sums of every part but the last
};
__device__ __forceinline__ void tile_of(const TileMap& tp, int bid, int& mt, int& nt) {
    const int total = tp.tm * tp.tn, xcd = bid & 7, idx = bid >> 3, per = total >> 3, rem = total & 7;
    const int id = xcd * per + min(xcd, rem) + idx;   // workgroups are dealt round robin to the 8 XCDs
    const int span = tp.gm * tp.tn, g = id / span, in = id - g * span, rows = min(tp.gm, tp.tm - g * tp.gm);
    nt = in / rows;
    mt = g * tp.gm + in - nt * rows;
}

// Schedule of a depth: its LDS reads spread over the first 1 / PARTS of its MFMAs, its direct loads
// over all of them, so that the matrix unit is fed from the start and the reads are done early.
template <int READS, int LOADS, int MFMAS, int PARTS>
__device__ __forceinline__ void pace() {
    constexpr int kFront = MFMAS / PARTS > 0 ? MFMAS / PARTS : 1;
    constexpr int kR = (READS + kFront - 1) / kFront, kD = (LOADS + MFMAS - 1) / MFMAS;
#pragma unroll
    for (int m = 0; m < MFMAS; ++m) {
        if (m < kFront) __builtin_amdgcn_sched_group_barrier(0x100, kR, 0);
        if (LOADS) __builtin_amdgcn_sched_group_barrier(0x010, kD, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
}

enum Branch { kPlain = 0, kLora = 1, kLoraDrop = 2 };

// NWM x NWN waves, each MT x NT MFMA tiles of 32 tokens x 32 outputs; RING steps' tiles in LDS.
// DX: the input gradient (outputs are the columns k, the reduction runs over n).  VEC: rows of
// t, u, A, B and y are whole 16-byte chunks.  SPLIT: the reduction is split over workgroups; the
// last part's adds the others' partial tiles in order.
template <int NWM, int NWN, int MT, int NT, int RING, bool SPLIT, bool DX, int LORA, bool VEC, int DT>
__global__ __launch_bounds__(64 * NWM * NWN, MT* NT >= 4 ? 1 : 2) void fp8_gemm_kernel(const Fp8Gemm g, TileMap tp) {
    constexpr int kWaves = NWM * NWN, kThreads = 64 * kWaves;
    constexpr int kBM = 32 * MT * NWM, kBN = 32 * NT * NWN;
    constexpr int kXB = kBM * kStep, kWB = kBN * kStep, kSlot = kXB + kWB + 512 * kWaves;   // tiles, scales per wave
    constexpr int kXL = kXB / 1024 / kWaves, kWL = kWB / 1024 / kWaves, kLoads = kXL + kWL + 2;   // loads of a wave
    static_assert(kXL * kWaves * 1024 == kXB && kWL * kWaves * 1024 == kWB, "tiles are whole wave loads");
    static_assert(kBM <= 256 && kBN <= 256, "a wave load holds a tile's scales");
    __shared__ __attribute__((aligned(16))) uint8_t s0[kSlot];
    __shared__ __attribute__((aligned(16))) uint8_t s1[kSlot];
    constexpr int kTwo = RING > 2 ? kSlot : 16;
    __shared__ __attribute__((aligned(16))) uint8_t s2[kTwo], s3[kTwo];
    static_assert(RING == 2 || RING == 4, "slots of the ring");
    const int M = g.M, O = DX ? g.K : g.N, C = DX ? g.N : g.K, K = g.K, r = g.r, ld = g.ld;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % NWM, wn = wave / NWM;
    const int tiles = tp.tm * tp.tn, split = SPLIT ? (int)blockIdx.x / tiles : 0;
    int mt, nt;
    tile_of(tp, (int)blockIdx.x - split * tiles, mt, nt);
    const int m0 = mt * kBM, n0 = nt * kBN;   // (n0: first output, a column k with DX)
    const int steps = (C + kStep - 1) / kStep, first = SPLIT ? split * tp.per : 0;
    const int NS = SPLIT ? min(tp.per, steps - first) : steps;

    // ---- loads of step ks.  Steps past the reduction read as zero and move nothing.
    // Activations: a wave load fills 8 rows; lane: row lane / 8, LDS chunk lane % 8.
    const int lrow = 8 * wave + (lane >> 3), lch = (lane & 7) ^ swizzle(lrow);
    static_assert(8 * kWaves % 16 == 0, "the swizzle of a lane's chunk is the same for its next rows");
    const uint32_t xoff = (uint32_t)lrow * (uint32_t)ld + 16u * (uint32_t)lch;
    const i32x4_t xrs = buffer_rsrc(g.x + (int64_t)m0 * ld, (uint32_t)min(M - m0, kBM) * (uint32_t)ld);
    const uint32_t wvoff = (uint32_t)lrow * (uint32_t)K + 16u * (uint32_t)lch;       // (forward)
    const i32x4_t wrs = DX ? i32x4_t{} : buffer_rsrc(g.w + (int64_t)n0 * K, (uint32_t)min(g.N - n0, kBN) * (uint32_t)K);
    constexpr int kCR = kBN / 16, kRL = 64 / kCR;        // DX: chunks of a row, rows of a wave load
    const int wrow = kRL * wave + lane / kCR;
    const uint32_t dvoff = (uint32_t)wrow * (uint32_t)K + 16u * (uint32_t)code_chunk<kBN>(wrow, lane % kCR);
    static_assert(kRL * kWaves % 8 == 0, "the swizzle of a lane's chunk is the same for its next rows");
    auto load_x = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        const int c = (first + ks) * kStep;
        i32x4_t rs = xrs;
        rs[2] = ks < NS ? rs[2] : 0;
        // what lies past a row's end in a last step that is wider than what is left reads zero
        const uint32_t past = c + 16 * lch < ld ? 0u : kNone;
#pragma unroll
        for (int j = 0; j < kXL; ++j)
            raw_buffer_load_lds(rs, as_lds<uint32_t>(slot + 1024 * (kWaves * j + wave)), 16,
                                (int)((xoff + (uint32_t)(8 * kWaves * j) * (uint32_t)ld) | past), c, 0, 0);
        // scales of the tile's rows, four to a lane, for each wave
        const i32x4_t srs = buffer_rsrc(g.sx + (int64_t)(first + ks) * g.rs + m0,
                                        ks < NS ? (uint32_t)min(g.rs - m0, (int64_t)256) : 0u);
        raw_buffer_load_lds(srs, as_lds<uint32_t>(slot + kXB + kWB + 512 * wave), 4, 4 * lane, 0, 0, 0);
    };
    auto load_w = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        const int c = (first + ks) * kStep;
        uint8_t* const sc = slot + kXB + kWB + 512 * wave + 256;
        if constexpr (DX) {
            // the step's rows of W as a buffer of their own: rows past N read as zero
            const int left = g.N - c;
            const uint32_t bytes = (uint32_t)min(left, kStep) * (uint32_t)K - (uint32_t)n0;
            const i32x4_t rs = buffer_rsrc(g.w + (int64_t)c * K + n0, ks < NS ? bytes : 0u);
#pragma unroll
            for (int j = 0; j < kWL; ++j)
                raw_buffer_load_lds(rs, as_lds<uint32_t>(slot + kXB + 1024 * (kWaves * j + wave)), 16,
                                    (int)(dvoff + (uint32_t)(kRL * kWaves * j) * (uint32_t)K), 0, 0, 0);
            // scales: a lane holds the four bytes around that of columns 4 lane ..
            const i32x4_t srs = buffer_rsrc(g.sw + (int64_t)(first + ks) * g.wrs, ks < NS ? (uint32_t)g.wrs : 0u);
            raw_buffer_load_lds(srs, as_lds<uint32_t>(sc), 4, ((n0 + 4 * lane) >> 7) & ~3, 0, 0, 0);
        } else {
            i32x4_t rs = wrs;
            rs[2] = ks < NS ? rs[2] : 0;
            const uint32_t past = c + 16 * lch < K ? 0u : kNone;
#pragma unroll
            for (int j = 0; j < kWL; ++j)
                raw_buffer_load_lds(rs, as_lds<uint32_t>(slot + kXB + 1024 * (kWaves * j + wave)), 16,
                                    (int)((wvoff + (uint32_t)(8 * kWaves * j) * (uint32_t)K) | past), c, 0, 0);
            const int nb0 = n0 >> 7;
            const i32x4_t srs = buffer_rsrc(
                g.sw + nb0 * g.wrs, ks < NS ? (uint32_t)min((((int64_t)g.N + 127) / 128 - nb0) * g.wrs, (int64_t)0x7FFFFFFF) : 0u);
            raw_buffer_load_lds(srs, as_lds<uint32_t>(sc), 4,
                                (int)((uint32_t)(((n0 + 4 * lane) >> 7) - nb0) * (uint32_t)g.wrs +
                                      ((uint32_t)(first + ks) & ~3u)), 0, 0, 0);
        }
    };

    // ---- operand reads: a lane holds 32 consecutive reduction indices of a row (or column)
    struct Ops {
        u32x8_t x[MT], w[NT];
    };
    struct Scales {
        int x[MT], w[NT];
    };
    uint32_t offX[2][2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) offX[kk][e] = tile_byte(l32, 4 * kk + 2 * h + e);
    uint32_t offD[NT];
    if (DX) {   // lane j of a 16-lane group addresses row j / 2, columns 8 (j % 2) .. of the group's 8 x 16 codes
        const int j = l32 & 15, row = 32 * h + (j >> 1);
#pragma unroll
        for (int e = 0; e < NT; ++e)
            offD[e] = kXB + (uint32_t)(row * kBN + 16 * code_chunk<kBN>(row, 2 * (NT * wn + e) + (l32 >> 4)) + 8 * (j & 1));
    }
    auto join = [](u32x4_t a, u32x4_t b) __attribute__((always_inline)) {
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read = [&](const uint8_t* __restrict__ slot, int kk, Ops& q) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if constexpr (DX) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {   // 8 rows further down the swizzle repeats
                    const u32x2_t c = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        as_lds<__attribute__((ext_vector_type(2))) int>(slot + offD[i] + kBN * (64 * kk + 8 * p))));
                    q.w[i][2 * p] = c[0];
                    q.w[i][2 * p + 1] = c[1];
                }
            } else {
                const uint8_t* p = slot + kXB + 4096 * (NT * wn + i);
                q.w[i] = join(*reinterpret_cast<const u32x4_t*>(p + offX[kk][0]), *reinterpret_cast<const u32x4_t*>(p + offX[kk][1]));
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint8_t* p = slot + 4096 * (MT * wm + i);
            q.x[i] = join(*reinterpret_cast<const u32x4_t*>(p + offX[kk][0]), *reinterpret_cast<const u32x4_t*>(p + offX[kk][1]));
        }
    };
    // (a wave's outputs are in one block of 128 where its width divides 128 and the tile's start is a block's)
    constexpr int kWS = 128 % (32 * NT) == 0 && kBN % 128 == 0 ? 1 : NT;
    auto read_scales = [&](const uint8_t* __restrict__ slot, int ks, Scales& q) __attribute__((always_inline)) {
        const uint8_t* p = slot + kXB + kWB + 512 * wave;
#pragma unroll
        for (int i = 0; i < MT; ++i) q.x[i] = p[32 * (MT * wm + i) + l32];
#pragma unroll
        for (int i = 0; i < kWS; ++i) {   // the byte wanted is brought down to bits 7..0
            const int o = 32 * (NT * wn + i);
            q.w[i] = (int)(*reinterpret_cast<const uint32_t*>(p + 256 + o) >>
                           (8 * (DX ? ((n0 + o) >> 7) & 3 : (first + ks) & 3)));
        }
#pragma unroll
        for (int i = kWS; i < NT; ++i) q.w[i] = q.w[0];
    };
    f32x16_t acc[MT][NT];
    auto multiply = [&](const Ops& q, const Scales& s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    __builtin_bit_cast(i32x8_t, q.w[j]), __builtin_bit_cast(i32x8_t, q.x[i]), acc[i][j], 0, 0, 0, s.w[j], 0,
                    s.x[i]);
    };

    // The products of a depth stay in front of the barrier that follows (nothing else orders them: the
    // compiler moved a whole depth's behind it, 1.2 us per step of 256 x 256 where 0.9 are needed).
    auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    constexpr int kReads = 2 * MT + (DX ? 4 : 2) * NT;   // LDS reads of a depth

    // ---- the LoRA term's operands.  t or u as MFMA operands: a lane holds ranks 16 kk + 8 h .. of its token
    const rsrc_t trs = buf_rsrc(LORA ? g.t + (int64_t)m0 * r : nullptr, (uint64_t)min(M - m0, kBM) * r * 2);
    auto load_t = [&](int i, int kk) __attribute__((always_inline)) {
        const int row = 32 * (MT * wm + i) + l32, j = 16 * kk + 8 * h;
        if (VEC)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   trs, j < r ? (uint32_t)(row * r + j) * 2u : kNone, 0, 0));
        return m0 + row < M && j < r ? load8(g.t + (int64_t)(m0 + row) * r + j, r - j) : u32x4_t{0u, 0u, 0u, 0u};
    };
    // forward: 64 rows of B, 16 bytes along n per lane
    constexpr int kCh = kBN / 8, kBPer = 64 * kCh / kThreads;   // 16-byte chunks of a row; per thread of 64 rows
    const rsrc_t brs = buf_rsrc(LORA && !DX ? g.L + n0 : nullptr, LORA && !DX ? ((uint64_t)r * O - n0) * 2 : 0);
    auto load_b = [&](int j0, int e) __attribute__((always_inline)) {
        const int c = tid + kThreads * e, j = j0 + c / kCh, n = 8 * (c % kCh);
        if (VEC)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   brs, j < r && n0 + n < O ? ((uint32_t)j * O + n) * 2u : kNone, 0, 0));
        return j < r && n0 + n < O ? load8(g.L + (int64_t)j * O + n0 + n, O - n0 - n) : u32x4_t{0u, 0u, 0u, 0u};
    };
    // input gradient: rows k of A as MFMA operands
    const rsrc_t ars = buf_rsrc(LORA && DX ? g.L + (int64_t)n0 * r : nullptr, (uint64_t)min(O - n0, kBN) * r * 2);
    auto load_a = [&](int e, int kk) __attribute__((always_inline)) {
        const int row = 32 * (NT * wn + e) + l32, j = 16 * kk + 8 * h;
        if (VEC)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   ars, j < r ? (uint32_t)(row * r + j) * 2u : kNone, 0, 0));
        return n0 + row < O && j < r ? load8(g.L + (int64_t)(n0 + row) * r + j, r - j) : u32x4_t{0u, 0u, 0u, 0u};
    };

    // chunk tid + kThreads e of rows of 64 ranks, 8 chunks a row
    auto load_row = [&](rsrc_t rs, const uint16_t* p, int rows, int e) __attribute__((always_inline)) {
        const int c = tid + kThreads * e, row = c >> 3, j = 8 * (c & 7);
        if (VEC)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   rs, j < r ? (uint32_t)(row * r + j) * 2u : kNone, 0, 0));
        return row < rows && j < r ? load8(p + (int64_t)row * r + j, r - j) : u32x4_t{0u, 0u, 0u, 0u};
    };

    // ---- main loop
    uint8_t* const slots[4] = {s0, s1, s2, s3};
#pragma unroll
    for (int p = 0; p < (RING == 2 ? 2 : 3); ++p) {
        load_x(slots[p], p);
        load_w(slots[p], p);
    }
    // zeros from the matrix unit while the first tiles are on their way (the compiler's copies of
    // 256 written registers took a microsecond in the int8 kernels)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            u32x4_t z = {0u, 0u, 0u, 0u};
            asm volatile("" : "+v"(z));   // (an operand of its own, or the products become one and its copies)
            acc[i][j] = mfma16<DT>(z, z, f32x16_t{});
        }
    if constexpr (RING == 2) {
        // Two slots (256 x 256 takes 66 KB each).  A tile is in registers after half of its step;
        // the one barrier of a step is there: its tile may then be overwritten, and the next one,
        // requested a whole step before, has landed.
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        Ops a, b;
        Scales sa, sb;
        read(s0, 0, a);
        read_scales(s0, 0, sa);
        auto step = [&](int ks, uint8_t* cur, const uint8_t* next) __attribute__((always_inline)) {
            read(cur, 1, b);
            multiply(a, sa);
            pin();
            pace<kReads, 0, MT * NT, 2>();
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            load_x(cur, ks + 2);
            load_w(cur, ks + 2);
            read(next, 0, a);
            read_scales(next, ks + 1, sb);
            multiply(b, sa);
            sa = sb;
            pin();
            pace<kReads + MT + kWS, kLoads, MT * NT, 2>();
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int ks = 0; ks < NS; ks += 2) {   // whole turns: steps past the end multiply zeros
            step(ks, s0, s1);
            step(ks + 1, s1, s0);
        }
    } else {
        // Four slots, operands two depths ahead: step ks reads tile ks + 1 and requests tile ks + 3;
        // its end waits for tile ks + 2 only.
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");   // tiles 0 and 1 have landed
        Ops a, b;
        Scales sa;
        read(s0, 0, a);
        read(s0, 1, b);
        read_scales(s0, 0, sa);
        auto step = [&](int ks, const uint8_t* __restrict__ next, uint8_t* __restrict__ fill) __attribute__((always_inline)) {
            Ops an, bn;
            Scales sn;
            load_x(fill, ks + 3);
            read(next, 0, an);
            read_scales(next, ks + 1, sn);
            multiply(a, sa);
            pin();
            pace<kReads + MT + kWS, kXL + 1, MT * NT, 1>();
            __builtin_amdgcn_sched_barrier(0);
            load_w(fill, ks + 3);
            read(next, 1, bn);
            multiply(b, sa);
            pin();
            pace<kReads, kWL + 1, MT * NT, 1>();
            a = an;
            b = bn;
            sa = sn;
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int ks = 0; ks < NS; ks += 4) {
            step(ks, s1, s3);
            step(ks + 1, s2, s0);
            step(ks + 2, s3, s1);
            step(ks + 3, s0, s2);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last, empty tiles
    __syncthreads();

    if constexpr (SPLIT) {
        constexpr uint32_t kTileBytes = (uint32_t)MT * NT * 16 * 4 * kThreads;
        const int tile = mt * tp.tn + nt;
        uint64_t* const flags = tp.tags + (size_t)tile * tp.splits;
        auto off = [&](int i, int j, int v4) { return (uint32_t)((((i * NT + j) * 4 + v4) * kThreads + tid) * 16); };
        if (split < tp.splits - 1) {
            const rsrc_t rs = buf_rsrc(tp.part + ((size_t)split * tiles + tile) * kTileBytes, kTileBytes);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        const f32x4_t v = {acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2],
                                           acc[i][j][4 * v4 + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rs, off(i, j, v4), 0,
                                                               kCoherent);
                    }
            publish_tag(flags + split, launch_tag());
            return;
        }
        const bool fail = wait_tags(flags, tp.splits - 1, launch_tag());
        // the parts' sums in order, this one's last
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            f32x4_t tot[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) tot[j][v4] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            for (int p = 0; p < tp.splits - 1; ++p) {
                const rsrc_t rs = buf_rsrc(tp.part + ((size_t)p * tiles + tile) * kTileBytes, kTileBytes);
                u32x4_t gv[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
                        gv[j][v4] = __builtin_amdgcn_raw_buffer_load_b128(rs, off(i, j, v4), 0, kCoherent);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
#pragma unroll
                        for (int c = 0; c < 4; ++c) tot[j][v4][c] += __uint_as_float(gv[j][v4][c]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][j][v] = fail ? __builtin_nanf("") : tot[j][v >> 2][v & 3] + acc[i][j][v];
        }
    }

    // ---- epilogue, 32 tokens of each wave row at a time, in four parts of the ring: B rows go to
    // e1 (0 - 63) and e2 (64 - 127) in their own layout, 16-byte chunks swizzled by row; the
    // outputs leave through e0 and e3 in turn.
    constexpr int kRow = 2 * kBN, kPart = RING == 2 ? (kXB + kWB) / 2 : kXB + kWB;
    static_assert(64 * kRow <= kPart && NWM * 32 * kRow <= kPart, "epilogue tiles fit their parts");
    uint8_t* const e0 = s0;
    uint8_t* const e1 = RING == 2 ? s0 + kPart : s1;
    uint8_t* const e2 = RING == 2 ? s1 : s2;
    uint8_t* const e3 = RING == 2 ? s1 + kPart : s3;
    // t (or u) of up to 64 ranks goes to e2 in rows of 128 bytes, and A's rows to e1 the same way:
    // all of it requested at once.  (Ranks 64 on are read from memory as operands.)
    const bool staged = LORA && r <= 64;
    if constexpr (LORA) {
        constexpr int kTPer = kBM * 8 / kThreads, kAPer = kBN * 8 / kThreads;
        static_assert(kBM * 128 <= kPart && kBN * 128 <= kPart, "operands of 64 ranks fit their parts");
        auto put = [&](uint8_t* slot, int e, u32x4_t v) __attribute__((always_inline)) {
            const int c = tid + kThreads * e;
            *reinterpret_cast<u32x4_t*>(slot + tile_byte(c >> 3, c & 7)) = v;
        };
        u32x4_t tv[kTPer], lv[DX ? kAPer : kBPer];
        if (staged)
#pragma unroll
            for (int e = 0; e < kTPer; ++e) tv[e] = load_row(trs, g.t + (int64_t)m0 * r, min(M - m0, kBM), e);
        if constexpr (DX) {
            if (staged)
#pragma unroll
                for (int e = 0; e < kAPer; ++e) lv[e] = load_row(ars, g.L + (int64_t)n0 * r, min(O - n0, kBN), e);
        } else {
#pragma unroll
            for (int e = 0; e < kBPer; ++e) lv[e] = load_b(0, e);
        }
        if (staged)
#pragma unroll
            for (int e = 0; e < kTPer; ++e) put(e2, e, tv[e]);
        if constexpr (DX) {
            if (staged)
#pragma unroll
                for (int e = 0; e < kAPer; ++e) put(e1, e, lv[e]);
        } else {
            auto put_b = [&](uint8_t* slot, int e, u32x4_t v) __attribute__((always_inline)) {
                const int c = tid + kThreads * e, row = c / kCh, cc = c % kCh;
                *reinterpret_cast<u32x4_t*>(slot + row * kRow + 16 * (cc ^ ((row & 3) << 1))) = v;
            };
#pragma unroll
            for (int e = 0; e < kBPer; ++e) put_b(e1, e, lv[e]);
            if (r > 64)
#pragma unroll
                for (int e = 0; e < kBPer; ++e) put_b(e2, e, load_b(64, e));
        }
        __syncthreads();
    }
    const int tj = l32 & 15, tg = l32 >> 4;
    const rsrc_t ors = buf_rsrc(g.out + (int64_t)m0 * O, DX || VEC ? (uint64_t)min(M - m0, kBM) * O * 2 : 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        // (the sums live in the accumulation registers until their turn)
        if constexpr (MT * NT >= 12)
#pragma unroll
            for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));
        f32x16_t f[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) f[j] = LORA == kLoraDrop ? f32x16_t{} : acc[i][j];
        if constexpr (LORA) {
            auto rank16 = [&](int kk, bool lds) __attribute__((always_inline)) {
                const u32x4_t a = lds ? *reinterpret_cast<const u32x4_t*>(e2 + tile_byte(32 * (MT * wm + i) + l32, 2 * kk + h))
                                      : load_t(i, kk);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    u32x4_t b;
                    if constexpr (DX) {
                        b = lds ? *reinterpret_cast<const u32x4_t*>(e1 + tile_byte(32 * (NT * wn + j) + l32, 2 * kk + h))
                                : load_a(j, kk);
                    } else {   // rows 16 kk + 8 h .. + 7 of B, column l32 of each tile, by two transposed reads
                        const uint8_t* slot = kk < 4 ? e1 : e2;
                        const int row = 16 * (kk & 3) + 8 * h + (tj >> 2), col = 32 * (NT * wn + j) + 16 * tg + 4 * (tj & 3);
                        const uint8_t* p = slot + row * kRow + 16 * ((col >> 3) ^ ((row & 3) << 1)) + 2 * (col & 7);
                        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p));
                        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p + 4 * kRow));
                        b = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    }
                    f[j] = mfma16<DT>(b, a, f[j]);
                }
            };
            if (staged)
                for (int kk = 0; 16 * kk < r; ++kk) rank16(kk, true);
            else
                for (int kk = 0; 16 * kk < r; ++kk) rank16(kk, false);
        }
        if constexpr (LORA == kLoraDrop) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                drop_tile(f[j], g.drop, (uint32_t)(m0 + 32 * (MT * wm + i) + l32), (uint32_t)(n0 + 32 * (NT * wn + j)), h);
#pragma unroll
                for (int v = 0; v < 16; ++v) f[j][v] += acc[i][j][v];
                __builtin_amdgcn_sched_barrier(0);   // (a tile at a time, or their temporaries spill)
            }
        }
        // lane (h, l32): token l32 of the 32, outputs 32 j + 8 v4 + 4 h + 0..3
        if constexpr (!DX && !VEC) {
            const int m = m0 + 32 * (MT * wm + i) + l32;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int n = n0 + 32 * (NT * wn + j) + 8 * (v >> 2) + 4 * h + (v & 3);
                    if (m < M && n < O) g.out[(int64_t)m * O + n] = (uint16_t)(pack2<DT>(f[j][v], 0.0f) & 0xFFFFu);
                }
        } else {
            uint8_t* const slot = (i & 1) ? e3 : e0;
            constexpr int kMask = (kCh < 16 ? kCh : 16) - 1;   // 16-byte chunks of a row are swizzled by the token
            static_assert((kCh & (kCh - 1)) == 0, "");
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const u32x2_t o = {pack2<DT>(f[j][4 * v4], f[j][4 * v4 + 1]),
                                       pack2<DT>(f[j][4 * v4 + 2], f[j][4 * v4 + 3])};
                    const int cc = 4 * (NT * wn + j) + v4;
                    *reinterpret_cast<u32x2_t*>(slot + (32 * wm + l32) * kRow + 16 * (cc ^ (l32 & kMask)) + 8 * h) = o;
                }
            __syncthreads();   // the slot written two rounds ago was read before the last barrier
#pragma unroll
            for (int e = 0; e < NWM * 32 * kCh / kThreads; ++e) {
                const int c = tid + kThreads * e, cc = c % kCh, rr = c / kCh;
                const int row = 32 * (MT * (rr >> 5) + i) + (rr & 31), n = n0 + 8 * cc;
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(slot + rr * kRow + 16 * (cc ^ (rr & kMask)));
                // rows past M lie past the buffer and are dropped, as are columns past the last
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, ors, n < O ? ((uint32_t)row * (uint32_t)O + (uint32_t)n) * 2u : kNone, 0, 0);
            }
        }
    }
}

template <int NWM, int NWN, int MT, int NT, int RING, bool SPLIT>
qlora_status run(const Fp8Gemm& g, bool dx, int splits, void* ws, int dt, hipStream_t s) {
    constexpr int kBM = 32 * MT * NWM, kBN = 32 * NT * NWN, kThreads = 64 * NWM * NWN;
    const int64_t O = dx ? g.K : g.N, C = dx ? g.N : g.K;
    TileMap tp{};
    tp.tm = (int)(((int64_t)g.M + kBM - 1) / kBM);
    tp.tn = (int)((O + kBN - 1) / kBN);
    tp.gm = 4;
    const int64_t tiles = (int64_t)tp.tm * tp.tn;
    if (SPLIT) {
        const int steps = (int)fp8_blocks(C);
        tp.per = (steps + splits - 1) / splits;
        tp.splits = (steps + tp.per - 1) / tp.per;
        tp.tags = static_cast<uint64_t*>(ws);
        tp.part = static_cast<uint8_t*>(ws) + align256((size_t)(tiles * splits) * 8);
    }
    const int64_t total = tiles * (SPLIT ? tp.splits : 1);
    if (total * kThreads >= (int64_t(1) << 32) || (int64_t)tp.gm * tp.tn >= (int64_t(1) << 31))
        return QLORA_ERR_UNSUPPORTED_SHAPE;
    const bool vec = g.r % 8 == 0 && g.N % 8 == 0;
    const int lora = g.r == 0 ? kPlain : dx && g.drop.thr ? kLoraDrop : kLora;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_G(D, L, V) \
    hipLaunchKernelGGL((fp8_gemm_kernel<NWM, NWN, MT, NT, RING, SPLIT, D, L, V, DT>), dim3((unsigned)total), dim3(kThreads), 0, s, g, tp)
        if (dx) {
            if (lora == kPlain) QL_G(true, kPlain, true);
            else if (lora == kLora) { if (g.r % 8 == 0) QL_G(true, kLora, true); else QL_G(true, kLora, false); }
            else { if (g.r % 8 == 0) QL_G(true, kLoraDrop, true); else QL_G(true, kLoraDrop, false); }
        } else if (lora == kPlain) {
            if (vec) QL_G(false, kPlain, true); else QL_G(false, kPlain, false);
        } else {
            if (vec) QL_G(false, kLora, true); else QL_G(false, kLora, false);
        }
#undef QL_G
    });
    return launch_status();
}

}  // namespace

size_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K, bool dx) {
    const Fp8Choice c = fp8_choice(M, dx ? K : N, dx ? N : K, true);
    if (c.splits == 1) return 0;
    const int64_t tiles = ((M + 127) / 128) * (((dx ? K : N) + 127) / 128);
    return align256((size_t)(tiles * c.splits) * 8) + (size_t)(tiles * (c.splits - 1)) * 128 * 128 * 4;
}

qlora_status launch_fp8_gemm(const Fp8Gemm& g, bool dx, int dt, void* ws, hipStream_t s) {
    const Fp8Choice c = fp8_choice(g.M, dx ? g.K : g.N, dx ? g.N : g.K, ws != nullptr);
    switch (c.tile) {
        case kFp8T256x256: return run<2, 2, 4, 4, 2, false>(g, dx, 1, nullptr, dt, s);
        case kFp8T128x128:
            return c.splits > 1 ? run<2, 2, 2, 2, 4, true>(g, dx, c.splits, ws, dt, s)
                                : run<2, 2, 2, 2, 4, false>(g, dx, 1, nullptr, dt, s);
        default: return run<2, 2, 1, 1, 4, false>(g, dx, 1, nullptr, dt, s);
    }
}

}  // namespace qlora
