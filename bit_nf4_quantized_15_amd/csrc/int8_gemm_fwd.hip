// Forward product of the int8 layer on MFMA (v_mfma_i32_32x32x32_i8), gfx950:
//
//   y[m,n] = RNE_16( sx[m] sw[n] sum_k xq[m,k] wq[n,k] + sum_j t[m,j] B[j,n] )
//
// ("bitsandbytes deep dive", section 4: vector-wise int8; sections 8.6 / 12.4: the LoRA
// branch.)  Both operands are int8 rows with consecutive k, so both tiles are copied
// HBM -> LDS by direct loads (16 bytes per lane, XOR-swizzled on the global side) and a
// lane's MFMA operand is one 16-byte LDS read.  Operands are read two MFMA depths ahead and
// tiles are requested one or more steps ahead, so neither latency is exposed: in the main
// loop of a 256 x 256 tile on an otherwise idle chip a step takes its MFMAs' time (0.44 us
// per 64 k).  On the whole chip the clock falls to 1.5 - 1.65 GHz, and what a tile moves
// counts: rows of 128 bytes per step (whole cache lines) measured 6 - 9 % faster than rows
// of 64 (8192 x 28672 x 8192, r = 0, calls: 1592 to 1475 us; the kernel's trace: 1434 us, 2.7 POP/s;
// 128 x 128 tiles 12 - 20 %).  Sums are exact int32; the scales, one after the other (int8.h), t B
// (r more reduction steps of the 16-bit MFMA) and the rounding follow once per tile.
//
// W rows are the MFMA's first operand, so a lane holds one token m and groups of four
// consecutive outputs n: y leaves through LDS in 8-byte writes and 16-byte stores.  t, the
// first 64 rows of B and the scales are fetched before the main loop into registers that it
// has no use for, and the epilogue goes 32 tokens at a time (scale, t B, round, store).
#include <algorithm>

#include "int8.h"
#include "lora_plan.h"
#include "split_sync.h"

namespace qlora {

__device__ void raw_buffer_load_lds(i32x4_t rsrc, __attribute__((address_space(3))) uint32_t* lds_ptr, int size,
                                    int voffset, int soffset, int offset, int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x16_t mfma16(u32x4_t a, u32x4_t b, f32x16_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}


typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}

// 8 values p[i .. i + 7] of a row whose values end at `end`, zero past it.
__device__ __forceinline__ u32x4_t load8(const uint16_t* __restrict__ p, int i, int end) {
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < end) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

__device__ __forceinline__ i32x4_t buffer_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return i32x4_t{(int32_t)(uint32_t)a, (int32_t)(uint32_t)(a >> 32), (int32_t)bytes, 0x00020000};
}

// The cast keeps the pointer's origin, so that the compiler can tell a direct load's
// destination from the buffers a step reads (each ring slot is an object of its own).
template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* as_lds(const void* p) {
    return (__attribute__((address_space(3))) T*)(p);
}


// Byte of 16-byte chunk c of tile row `row`: rows of S bytes, chunks XOR-swizzled so that any
// 16 consecutive rows of one chunk cover all 64 banks.
template <int S>
__device__ __forceinline__ int swizzle(int row) { return S == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
template <int S>
__device__ __forceinline__ uint32_t tile_byte(int row, int c) {
    return (uint32_t)row * S + ((uint32_t)(c ^ swizzle<S>(row)) << 4);
}

// Tiles in groups of `gm` row tiles, down the rows first: 32 consecutive tiles (one XCD's
// CUs at a time) then form a block of gm x 32 / gm that shares panels in the XCD's L2.
struct TileMap {
    int tm, tn, gm;
    int splits, per;      // the reduction in `splits` parts of `per` steps
    uint64_t* tags;       // [tile][split]
    uint8_t* part;        // [split][tile]: the int32 sums of every part but the last
};
__device__ __forceinline__ void tile_of(const TileMap& tp, int bid, int& mt, int& nt) {
    const int total = tp.tm * tp.tn, xcd = bid & 7, idx = bid >> 3, per = total >> 3, rem = total & 7;
    const int id = xcd * per + min(xcd, rem) + idx;   // workgroups are dealt round robin to the 8 XCDs
    const int span = tp.gm * tp.tn, g = id / span, in = id - g * span, rows = min(tp.gm, tp.tm - g * tp.gm);
    nt = in / rows;
    mt = g * tp.gm + in - nt * rows;
}

// NWM x NWN waves, each MT x NT MFMA tiles of 32 tokens x 32 outputs; S k per step, RING
// steps' tiles in LDS.  VEC: r % 8 == 0 and
// N % 8 == 0, so t, B and y are accessed 16 bytes at a time.
// LORA: r > 0.  SPLIT: the reduction is split over workgroups; the last part's adds the others' int32 sums
// (exact, so y does not depend on the split).
template <int NWM, int NWN, int MT, int NT, int S, int RING, bool SPLIT, bool LORA, bool VEC, int DT>
__global__ __launch_bounds__(64 * NWM * NWN, MT* NT >= 4 ? 1 : 2) void int8_gemm_fwd_kernel(
    const int8_t* __restrict__ xq, const float* __restrict__ sx, const int8_t* __restrict__ wq,
    const float* __restrict__ sw, const uint16_t* __restrict__ t, const uint16_t* __restrict__ B,
    uint16_t* __restrict__ y, int M, int N, int K, int r, TileMap tp) {
    constexpr int kWaves = NWM * NWN, kThreads = 64 * kWaves;
    constexpr int kBM = 32 * MT * NWM, kBN = 32 * NT * NWN;
    constexpr int kXB = kBM * S, kWB = kBN * S, kKK = S / 32;      // bytes of a step's tiles
    constexpr int kXL = kXB / 1024 / kWaves, kWL = kWB / 1024 / kWaves;   // loads per wave
    static_assert(kXL * kWaves * 1024 == kXB && kWL * kWaves * 1024 == kWB, "tiles are whole wave loads");
    __shared__ __attribute__((aligned(16))) uint8_t s0[kXB + kWB];
    __shared__ __attribute__((aligned(16))) uint8_t s1[kXB + kWB];
    constexpr int kTwo = RING > 2 ? kXB + kWB : 16, kMore = RING > 4 ? kXB + kWB : 16;
    __shared__ __attribute__((aligned(16))) uint8_t s2[kTwo], s3[kTwo];
    __shared__ __attribute__((aligned(16))) uint8_t s4[kMore], s5[kMore], s6[kMore], s7[kMore];
    uint8_t* const slots[8] = {s0, s1, s2, s3, s4, s5, s6, s7};
    static_assert((RING == 2 && S == 128) || RING == 4 || RING == 8, "slots of the ring");
    constexpr int kInFlight = RING == 2 ? kXL + kWL : (RING - 3) * (kXL + kWL);   // loads that a barrier leaves in flight
    __shared__ __attribute__((aligned(16))) float swt[kBN];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % NWM, wn = wave / NWM;
    const int tiles = tp.tm * tp.tn, split = SPLIT ? (int)blockIdx.x / tiles : 0;
    int mt, nt;
    tile_of(tp, (int)blockIdx.x - split * tiles, mt, nt);
    const int m0 = mt * kBM, n0 = nt * kBN;
    const int steps = (K + S - 1) / S, s_first = SPLIT ? split * tp.per : 0, NS = SPLIT ? min(tp.per, steps - s_first) : steps;

    // panels as buffers: rows past the end read as zero (the range check covers voffset)
    const uint32_t k_first = (uint32_t)(s_first * S);
    const i32x4_t xrs = buffer_rsrc(xq + (int64_t)m0 * K + k_first, (uint32_t)min(M - m0, kBM) * (uint32_t)K - k_first);
    const i32x4_t wrs = buffer_rsrc(wq + (int64_t)n0 * K + k_first, (uint32_t)min(N - n0, kBN) * (uint32_t)K - k_first);
    // a wave load fills kRL whole rows of S bytes; lane: row lane / kCL, LDS chunk lane % kCL
    constexpr int kCL = S / 16, kRL = 64 / kCL;
    const int lrow = lane / kCL, lch = (lane % kCL) ^ swizzle<S>(kRL * wave + lrow);
    static_assert(kRL * kWaves % 16 == 0, "the swizzle of a lane's chunk is the same for its next rows");
    const uint32_t voff = (uint32_t)(kRL * wave + lrow) * (uint32_t)K + 16u * (uint32_t)lch;
    // of a last step that is wider than what is left of K (64 of 128), the rest reads zero
    auto past = [&](int ks) __attribute__((always_inline)) {
        return S == 64 || (int)k_first + ks * S + 16 * lch < K ? 0u : 0x80000000u;
    };
    auto load_x = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        i32x4_t rs = xrs;
        rs[2] = ks < NS ? rs[2] : 0;   // steps past K read as zero and move nothing
#pragma unroll
        for (int j = 0; j < kXL; ++j)
            raw_buffer_load_lds(rs, as_lds<uint32_t>(slot + 1024 * (kWaves * j + wave)), 16,
                                (int)((voff + (uint32_t)(kRL * kWaves * j) * (uint32_t)K) | past(ks)), ks * S, 0, 0);
    };
    auto load_w = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        i32x4_t rs = wrs;
        rs[2] = ks < NS ? rs[2] : 0;
#pragma unroll
        for (int j = 0; j < kWL; ++j)
            raw_buffer_load_lds(rs, as_lds<uint32_t>(slot + kXB + 1024 * (kWaves * j + wave)), 16,
                                (int)((voff + (uint32_t)(kRL * kWaves * j) * (uint32_t)K) | past(ks)), ks * S, 0, 0);
    };
    auto load = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        load_x(slot, ks);
        load_w(slot, ks);
    };
    // operand bytes: chunk 2 kk + h of rows 32 i + l32 (the swizzle has period 16 rows)
    uint32_t offX[kKK], offW[kKK];
#pragma unroll
    for (int kk = 0; kk < kKK; ++kk) {
        offX[kk] = tile_byte<S>(32 * MT * wm + l32, 2 * kk + h);
        offW[kk] = kXB + tile_byte<S>(32 * NT * wn + l32, 2 * kk + h);
    }
    auto read = [&](const uint8_t* __restrict__ slot, int kk, i32x4_t (&a)[MT], i32x4_t (&b)[NT])
                    __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) b[i] = *reinterpret_cast<const i32x4_t*>(slot + offW[kk] + 32u * S * i);
#pragma unroll
        for (int i = 0; i < MT; ++i) a[i] = *reinterpret_cast<const i32x4_t*>(slot + offX[kk] + 32u * S * i);
    };

    // ---- ahead of the main loop: scales, t as MFMA operands (lane: token l32, ranks 8 h .. of
    // each 16) and the first 64 rows of B, 16 bytes along n per lane
    const rsrc_t trs = buf_rsrc(LORA ? t + (int64_t)m0 * r : nullptr, (uint64_t)min(M - m0, kBM) * r * 2);
    auto load_t = [&](int i, int kk) __attribute__((always_inline)) {
        const int row = 32 * (MT * wm + i) + l32, j = 16 * kk + 8 * h;
        if (VEC)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   trs, j < r ? (uint32_t)(row * r + j) * 2u : 0x80000000u, 0, 0));
        return m0 + row < M && j < r ? load8(t + (int64_t)(m0 + row) * r + j, j, r) : u32x4_t{0u, 0u, 0u, 0u};
    };
    const rsrc_t brs = buf_rsrc(LORA ? B + n0 : nullptr, LORA ? ((uint64_t)r * N - n0) * 2 : 0);
    constexpr int kCh = kBN / 8, kBPer = 64 * kCh / kThreads;   // 16-byte chunks of a row; per thread of 64 rows
    auto load_b = [&](int j0, int e) __attribute__((always_inline)) {
        const int c = tid + kThreads * e, j = j0 + c / kCh, n = 8 * (c % kCh);
        if (VEC)
            return __builtin_bit_cast(u32x4_t,
                                      __builtin_amdgcn_raw_buffer_load_b128(
                                          brs, j < r && n0 + n < N ? ((uint32_t)j * N + n) * 2u : 0x80000000u, 0, 0));
        return j < r && n0 + n < N ? load8(B + (int64_t)j * N + n0 + n, n0 + n, N) : u32x4_t{0u, 0u, 0u, 0u};
    };
    u32x4_t tv[MT][4], bv[kBPer];
    load(s0, 0);
    if (RING > 2) load(s1, 1);
    static_assert(kBN <= kThreads, "a scale per thread");
    const float swv = sw[min(n0 + tid, N - 1)];
    float sxv[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) sxv[i] = sx[min(m0 + 32 * (MT * wm + i) + l32, M - 1)];
    if (LORA) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tv[i][kk] = load_t(i, kk);
#pragma unroll
        for (int e = 0; e < kBPer; ++e) bv[e] = load_b(0, e);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (RING == 2) load(s1, 1);
#pragma unroll
    for (int p = 2; p < RING - 1; ++p) load(slots[p], p);
    // zeros from the matrix unit while the first tiles are on their way: writing 256 registers
    // (and the compiler's copies of them) took a microsecond
    i32x16_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const i32x4_t z = {0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(z, z, i32x16_t{}, 0, 0, 0);
        }
    // tiles 0 and 1 (of two slots, 0) have landed
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kInFlight) : "memory");
    i32x4_t xa[2][MT], wb[2][NT];
    read(s0, 0, xa[0], wb[0]);
    read(s0, 1, xa[1], wb[1]);

    auto step = [&](int ks, const uint8_t* __restrict__ cur, const uint8_t* __restrict__ next, uint8_t* __restrict__ fill) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < kKK; ++kk) {
            if (kk == 0) load_x(fill, ks + RING - 1);
            if (kk == kKK / 2) load_w(fill, ks + RING - 1);
            // operands two MFMA depths ahead: an LDS read's latency is longer than a small tile's MFMAs
            i32x4_t xn[MT], wn_[NT];
            if (kk + 2 < kKK) read(cur, kk + 2, xn, wn_);
            else read(next, kk + 2 - kKK, xn, wn_);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wb[kk & 1][j], xa[kk & 1][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < MT; ++i) xa[kk & 1][i] = xn[i];
#pragma unroll
            for (int j = 0; j < NT; ++j) wb[kk & 1][j] = wn_[j];
            // operands are read (and the new tiles requested) between the MFMAs
            constexpr int kReads = MT + NT, kPer = MT * NT / kReads;
#pragma unroll
            for (int g = 0; g < kReads; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (g % 2 == 1 || kReads < 8) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, kPer > 0 ? kPer : 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // tile ks + 2 has landed once only the loads of the RING - 3 after it are in flight
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kInFlight) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Two slots of 128 k (256 x 256: rows of whole 128-byte lines, and no room for a third).  A
    // tile is in registers after half of its step; the one barrier of a step is there: its tile
    // may then be overwritten, and the next one, requested a whole step before, has landed.
    auto step2 = [&](int ks, uint8_t* cur, const uint8_t* next) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < kKK; ++kk) {
            if (kk == 2) load_x(cur, ks + 2);
            if (kk == 3) load_w(cur, ks + 2);
            i32x4_t xn[MT], wn_[NT];
            if (kk < 2) read(cur, (kk + 2) % kKK, xn, wn_);
            else read(next, kk - 2, xn, wn_);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wb[kk & 1][j], xa[kk & 1][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < MT; ++i) xa[kk & 1][i] = xn[i];
#pragma unroll
            for (int j = 0; j < NT; ++j) wb[kk & 1][j] = wn_[j];
            constexpr int kReads = MT + NT, kPer = MT * NT / kReads;
#pragma unroll
            for (int g = 0; g < kReads; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (kk >= 2) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                if (kk == 1) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // reads done by the barrier
                else __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (kk == 1) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // whole turns of the ring: steps past K multiply zeros
    if constexpr (RING == 2) {
        for (int ks = 0; ks < NS; ks += 2) {
            step2(ks, s0, s1);
            step2(ks + 1, s1, s0);
        }
    } else for (int ks = 0; ks < NS; ks += RING) {
#pragma unroll
        for (int p = 0; p < RING; ++p) step(ks + p, slots[p], slots[(p + 1) % RING], slots[(p + RING - 1) % RING]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last, empty tiles
    if (tid < kBN) swt[tid] = swv;
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
                        const u32x4_t v = {(uint32_t)acc[i][j][4 * v4], (uint32_t)acc[i][j][4 * v4 + 1],
                                           (uint32_t)acc[i][j][4 * v4 + 2], (uint32_t)acc[i][j][4 * v4 + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(v, rs, off(i, j, v4), 0, kCoherent);
                    }
            publish_tag(flags + split, launch_tag());
            return;
        }
        bool fail = wait_tags(flags, tp.splits - 1, launch_tag());
        if (fail) for (int i = tid; i < kBN; i += kThreads) swt[i] = __builtin_nanf("");
        for (int p = 0; p < tp.splits - 1; ++p) {
            const rsrc_t rs = buf_rsrc(tp.part + ((size_t)p * tiles + tile) * kTileBytes, kTileBytes);
            u32x4_t g[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
                        g[i][j][v4] = __builtin_amdgcn_raw_buffer_load_b128(rs, off(i, j, v4), 0, kCoherent);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] += (int32_t)g[i][j][v >> 2][v & 3];
        }
        __syncthreads();
    }

    // ---- epilogue, in four parts of the ring.  B rows go to e1 (0 - 63) and e2 (64 - 127) in
    // their own layout, 16-byte chunks swizzled by row; y leaves through e0 and e3 in turn, 32
    // tokens of each wave row.
    constexpr int kBRow = 2 * kBN, kPart = RING == 2 ? (kXB + kWB) / 2 : kXB + kWB;
    static_assert(64 * kBRow <= kPart && NWM * 32 * kBRow <= kPart, "epilogue tiles fit their parts");
    uint8_t* const e0 = s0;
    uint8_t* const e1 = RING == 2 ? s0 + kPart : s1;
    uint8_t* const e2 = RING == 2 ? s1 : s2;
    uint8_t* const e3 = RING == 2 ? s1 + kPart : s3;
    auto put_b = [&](uint8_t* slot, int e, u32x4_t v) __attribute__((always_inline)) {
        const int c = tid + kThreads * e, row = c / kCh, cc = c % kCh;
        *reinterpret_cast<u32x4_t*>(slot + row * kBRow + 16 * (cc ^ ((row & 3) << 1))) = v;
    };
    if (LORA) {
#pragma unroll
        for (int e = 0; e < kBPer; ++e) put_b(e1, e, bv[e]);
        if (r > 64) {
#pragma unroll
            for (int e = 0; e < kBPer; ++e) bv[e] = load_b(64, e);
#pragma unroll
            for (int e = 0; e < kBPer; ++e) put_b(e2, e, bv[e]);
        }
        __syncthreads();
    }
    uint64_t loud[MT];   // lanes whose token has a scale above 2^90
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        loud[i] = __builtin_amdgcn_ballot_w64(loud_scale(sxv[i]));
        if (loud_scale(sxv[i])) sxv[i] *= kLoudDown;
    }
    const int tj = l32 & 15, tg = l32 >> 4;
    const rsrc_t yrs = buf_rsrc(y + (int64_t)m0 * N, VEC ? (uint64_t)min(M - m0, kBM) * N * 2 : 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        f32x16_t f[NT];
        // The sums live in the accumulation registers until their turn (the compiler would move
        // all of them to vector registers at the end of the loop, and spill).
        if constexpr (MT * NT >= 12)
#pragma unroll
            for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                const f32x4_t w4 = *reinterpret_cast<const f32x4_t*>(swt + 32 * (NT * wn + j) + 8 * v4 + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[j][4 * v4 + e] = (float)acc[i][j][4 * v4 + e] * sxv[i] * w4[e];
            }
        if (__builtin_expect(loud[i] != 0, 0)) {
            const float up = (loud[i] >> lane) & 1 ? kLoudUp : 1.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) f[j][v] *= up;
        }
        // t B: rows 16 kk + 8 h .. + 7 of B, column l32 of each tile, by two transposed reads
        auto rank16 = [&](const uint8_t* slot, int kk, u32x4_t a) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int row = 16 * kk + 8 * h + (tj >> 2), col = 32 * (NT * wn + j) + 16 * tg + 4 * (tj & 3);
                const uint8_t* p = slot + row * kBRow + 16 * ((col >> 3) ^ ((row & 3) << 1)) + 2 * (col & 7);
                const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p));
                const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<s16x4_t>(p + 4 * kBRow));
                const u32x4_t b = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                f[j] = mfma16<DT>(b, a, f[j]);
            }
        };
        if (LORA) {   // (ranks past r are zero: 32 at a time, so that the sums keep their registers)
            rank16(e1, 0, tv[i][0]);
            rank16(e1, 1, tv[i][1]);
            if (r > 32) {
                rank16(e1, 2, tv[i][2]);
                rank16(e1, 3, tv[i][3]);
            }
            for (int kk = 4; 16 * kk < r; ++kk) rank16(e2, kk - 4, load_t(i, kk));
        }
        // lane (h, l32): token l32 of the 32, outputs 32 j + 8 v4 + 4 h + 0..3
        if (!VEC) {
            const int m = m0 + 32 * (MT * wm + i) + l32;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int n = n0 + 32 * (NT * wn + j) + 8 * (v >> 2) + 4 * h + (v & 3);
                    if (m < M && n < N) y[(int64_t)m * N + n] = (uint16_t)(pack2<DT>(f[j][v], 0.0f) & 0xFFFFu);
                }
            continue;
        }
        uint8_t* const slot = (i & 1) ? e3 : e0;
        constexpr int kMask = kCh % 16 == 0 ? 15 : 7;   // 16-byte chunks of a row are swizzled by the token
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                const u32x2_t o = {pack2<DT>(f[j][4 * v4], f[j][4 * v4 + 1]),
                                   pack2<DT>(f[j][4 * v4 + 2], f[j][4 * v4 + 3])};
                const int cc = 4 * (NT * wn + j) + v4;
                *reinterpret_cast<u32x2_t*>(slot + (32 * wm + l32) * kBRow + 16 * (cc ^ (l32 & kMask)) + 8 * h) = o;
            }
        __syncthreads();   // the slot written two rounds ago was read before the last barrier
#pragma unroll
        for (int e = 0; e < NWM * 32 * kCh / kThreads; ++e) {
            const int c = tid + kThreads * e, cc = c % kCh, rr = c / kCh;
            const int row = 32 * (MT * (rr >> 5) + i) + (rr & 31), n = n0 + 8 * cc;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(slot + rr * kBRow + 16 * (cc ^ (rr & kMask)));
            // rows past M lie past the buffer and are dropped, as are columns past N
            __builtin_amdgcn_raw_buffer_store_b128(
                v, yrs, n < N ? ((uint32_t)row * (uint32_t)N + (uint32_t)n) * 2u : 0x80000000u, 0, 0);
        }
    }
}

struct Args {
    const int8_t* xq;
    const float* sx;
    const int8_t* wq;
    const float* sw;
    const uint16_t* t;
    const uint16_t* B;
    uint16_t* y;
    int M, N, K, r, dt;
    hipStream_t s;
};

template <int NWM, int NWN, int MT, int NT, int S, int RING, bool SPLIT>
qlora_status run(const Args& a, int splits, void* ws) {
    constexpr int kBM = 32 * MT * NWM, kBN = 32 * NT * NWN, kThreads = 64 * NWM * NWN;
    TileMap tp{};
    tp.tm = (int)(((int64_t)a.M + kBM - 1) / kBM);
    tp.tn = (int)(((int64_t)a.N + kBN - 1) / kBN);
    tp.gm = 4;
    const int64_t tiles = (int64_t)tp.tm * tp.tn;
    if (SPLIT) {
        const int steps = (a.K + S - 1) / S;
        tp.per = (steps + splits - 1) / splits;
        tp.splits = (steps + tp.per - 1) / tp.per;
        tp.tags = static_cast<uint64_t*>(ws);
        tp.part = static_cast<uint8_t*>(ws) + align256((size_t)tiles * splits * 8);
    }
    const int64_t total = tiles * (SPLIT ? tp.splits : 1);
    if (total * kThreads >= (int64_t(1) << 32) || (int64_t)tp.gm * tp.tn >= (int64_t(1) << 31))
        return QLORA_ERR_UNSUPPORTED_SHAPE;
    // (the offsets of B and of a tile's rows of y must fit a buffer's 31 bits)
    const bool vec = a.r % 8 == 0 && a.N % 8 == 0 && (int64_t)std::max(a.r, kBM) * a.N * 2 < (int64_t(1) << 31);
    with_dt(a.dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_F(L, V)                                                                                                   \
    hipLaunchKernelGGL((int8_gemm_fwd_kernel<NWM, NWN, MT, NT, S, RING, SPLIT, L, V, DT>), dim3((unsigned)total),            \
                       dim3(kThreads), 0, a.s, a.xq, a.sx, a.wq, a.sw, a.t, a.B, a.y, a.M, a.N, a.K, a.r, tp)
        if (a.r) {
            if (vec) QL_F(true, true); else QL_F(true, false);
        } else {
            if (vec) QL_F(false, true); else QL_F(false, false);
        }
#undef QL_F
    });
    return launch_status();
}

}  // namespace

size_t int8_gemm_fwd_workspace(int64_t M, int64_t N, int64_t K) {
    const Int8Choice c = int8_fwd_choice(M, N, K, true);
    if (c.splits == 1) return 0;
    const int64_t tiles = tiles_of(M, N, 128, 128);
    return align256((size_t)(tiles * c.splits) * 8) + (size_t)(tiles * (c.splits - 1)) * 128 * 128 * 4;
}

qlora_status launch_int8_gemm_fwd(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                  const uint16_t* t, const uint16_t* B, uint16_t* y, int M, int N, int K, int r, int dt,
                                  void* ws, hipStream_t s) {
    const Args a{xq, sx, wq, sw, t, B, y, M, N, K, r, dt, s};
    const Int8Choice c = int8_fwd_choice(M, N, K, ws != nullptr);
    switch (c.tile) {
        case kFwd256x256: return run<2, 2, 4, 4, 128, 2, false>(a, 1, nullptr);
        case kFwd256x192: return run<2, 2, 4, 3, 128, 2, false>(a, 1, nullptr);
        case kFwd128x128:
            return c.splits > 1 ? run<2, 2, 2, 2, 128, 4, true>(a, c.splits, ws) : run<2, 2, 2, 2, 128, 4, false>(a, 1, nullptr);
        default: return run<2, 2, 1, 1, 64, 8, false>(a, 1, nullptr);
    }
}

}  // namespace qlora
