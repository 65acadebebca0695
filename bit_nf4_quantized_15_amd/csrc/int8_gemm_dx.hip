// Input gradient of the int8 layer on MFMA (v_mfma_f32_32x32x16_{bf16,f16}), gfx950:
//
//   dx[m,k] = RNE_16( sum_n dy[m,n] W_16[n,k] + sum_j u[m,j] A[k,j] ),
//   W_16[n,k] = RNE_16( fl32( sw[n] wq[n,k] ) )
//
// ("bitsandbytes deep dive", section 4: vector-wise int8; 12.4: frozen base, no dW.)  The
// reduction runs down the stored rows n, 64 per step: dy (whole 128-byte lines) and the int8
// weight (64 rows of its codes) are copied HBM -> LDS by direct loads.  An MFMA operand is 8
// consecutive n of one column k: gfx950's transposed byte read (ds_read_b64_tr_b8) hands a
// lane exactly those 8 codes, which it scales (a scale per n, the same for all columns) and
// rounds in registers: 20 VALU instructions per operand.  Each wave owns its columns over all
// rows of the tile, so no weight is expanded twice and the weight's LDS traffic is its one
// byte per element.
//
// While the MFMAs of 16 n run, dy and codes of the 16 n two further on are read and the codes
// read before are expanded for the next 16.  Bound by the MFMAs and the power they draw (the
// expansion's VALU work runs beside them).  4096 x 11008 x 4096, r = 64, traced: 278 us for a given
// u, 1.33 PFLOP/s; 309 us behind the kernel that makes u, 1.19 PFLOP/s.
#include <algorithm>

#include "int8.h"
#include "lora_plan.h"
#include "split_sync.h"

namespace qlora {

__device__ void raw_buffer_load_lds(i32x4_t rsrc, __attribute__((address_space(3))) uint32_t* lds_ptr, int size,
                                    int voffset, int soffset, int offset, int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

template <int DT>
__device__ __forceinline__ f32x16_t mfma16(u32x4_t a, u32x4_t b, f32x16_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ i32x4_t buffer_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return i32x4_t{(int32_t)(uint32_t)a, (int32_t)(uint32_t)(a >> 32), (int32_t)bytes, 0x00020000};
}
__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}

template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* as_lds(const void* p) {
    return (__attribute__((address_space(3))) T*)(p);
}

// 8 values p[i .. i + 7] of a row that ends at `end`, zero past it; p has any alignment
__device__ __forceinline__ u32x4_t load8(const uint16_t* __restrict__ p, int64_t i, int64_t end) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (i + 8 <= end) {
        __builtin_memcpy(&v, p, 16);
        return v;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < end) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

constexpr int kStep = kDxStep;   // rows n per step
constexpr int kKK = 4;      // MFMA depths (16 n) of a step
constexpr int kWaves = 4, kThreads = 256;

// dy tile: 128-byte rows, 16-byte chunks swizzled so that 16 consecutive rows of one chunk
// cover all 64 banks
__device__ __forceinline__ uint32_t tile_byte(int row, int c) {
    return (uint32_t)row * 128u + ((uint32_t)(c ^ ((row >> 1) & 7)) << 4);
}
// code tile: rows of kBN bytes; the 8 rows x 32 columns that two lane groups read together
// lie on different banks
template <int BN>
__device__ __forceinline__ int code_chunk(int row, int c) {
    return BN >= 256 ? c ^ ((row & 7) << 1) : c ^ (((row >> 1) & 3) << 1);
}

// 4 waves side by side, each MT x NT MFMA tiles (32 tokens x 32 columns k).  DYV: dy rows are
// whole 16-byte chunks (direct loads); AV: rows of u and A are.
// RING: steps' tiles in LDS, two or four.  SPLIT: the reduction is split over workgroups; the
// last part's adds the others' partial tiles in order.
struct Split {
    int splits, per;      // parts of `per` steps
    uint64_t* tags;       // [tile][split]
    uint8_t* part;        // [split][tile]: the fp32 sums of every part but the last
};

template <int MT, int NT, int RING, bool SPLIT, bool DYV, bool AV, int DT>
__global__ __launch_bounds__(kThreads, 1) void int8_gemm_dx_kernel(
    const uint16_t* __restrict__ dy, const int8_t* __restrict__ wq, const float* __restrict__ sw,
    const uint16_t* __restrict__ u, const uint16_t* __restrict__ A, uint16_t* __restrict__ dx, int M, int N, int K,
    int r, int tm, int tn, int gm, Split sp) {
    constexpr int kBM = 32 * MT, kBN = 32 * NT * kWaves;
    constexpr int kDB = kBM * 128, kWB = kStep * kBN;
    constexpr int kSlot = kDB + kWB + 256 * kWaves;      // dy, codes, a copy of the scales per wave
    constexpr int kDL = kDB / 1024 / kWaves, kWL = kWB / 1024 / kWaves;
    constexpr int kLoads = (DYV ? kDL : 0) + kWL + 1;
    static_assert(kDL * kWaves * 1024 == kDB && kWL * kWaves * 1024 == kWB, "tiles are whole wave loads");
    __shared__ __attribute__((aligned(16))) uint8_t s0[kSlot];
    __shared__ __attribute__((aligned(16))) uint8_t s1[kSlot];
    constexpr int kTwo = RING > 2 ? kSlot : 16;
    __shared__ __attribute__((aligned(16))) uint8_t s2[kTwo], s3[kTwo];
    static_assert(RING == 4 || (RING == 2 && DYV), "slots of the ring");
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = tm * tn, split = SPLIT ? (int)blockIdx.x / tiles : 0, bid = (int)blockIdx.x - split * tiles;
    int mt, nt;
    {   // tiles in groups of gm row tiles; each XCD (ids dealt round robin) takes a run of them
        const int xcd = bid & 7, idx = bid >> 3, per = tiles >> 3, rem = tiles & 7;
        const int id = xcd * per + min(xcd, rem) + idx, span = gm * tn, g = id / span, in = id - g * span;
        const int rows = min(gm, tm - g * gm);
        nt = in / rows;
        mt = g * gm + in - nt * rows;
    }
    const int m0 = mt * kBM, k0 = nt * kBN;
    const int steps = (N + kStep - 1) / kStep, first = SPLIT ? split * sp.per : 0;
    const int NS = SPLIT ? min(sp.per, steps - first) : steps;
    const int n_end = SPLIT ? min(N, (first + NS) * kStep) : N;   // rows of W past it read as zero

    // ---- loads of step ks
    const i32x4_t drs = buffer_rsrc(dy + (int64_t)m0 * N, (uint32_t)((int64_t)min(M - m0, kBM) * N * 2));
    const i32x4_t srs = buffer_rsrc(sw, (uint32_t)min((int64_t)N * 4, (int64_t)0x7FFFFFFF));
    const int drow = 8 * wave + (lane >> 3), dch = (lane & 7) ^ ((drow >> 1) & 7);   // a wave load: 8 rows
    uint32_t dvoff[kDL];
#pragma unroll
    for (int j = 0; j < kDL; ++j) dvoff[j] = (uint32_t)(((int64_t)(drow + 32 * j) * N + 8 * dch) * 2);
    constexpr int kCR = kBN / 16, kRL = 64 / kCR;        // code chunks of a row, rows of a wave load
    const int wrow = kRL * wave + lane / kCR;
    const uint32_t wvoff = (uint32_t)wrow * (uint32_t)K + 16u * (uint32_t)code_chunk<kBN>(wrow, lane % kCR);
    static_assert(kRL * kWaves % 8 == 0, "the swizzle of a lane's chunk is the same for its next rows");
    u32x4_t dreg[DYV ? 1 : kDL];
    auto load_dy = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        const int n = (first + ks) * kStep;
        if (DYV) {
            // columns past N (in the last step) would be the next row's: read as zero
            const uint32_t past = n + 8 * dch < n_end ? 0u : 0x80000000u;
#pragma unroll
            for (int j = 0; j < kDL; ++j)
                raw_buffer_load_lds(drs, as_lds<uint32_t>(slot + 1024 * (kWaves * j + wave)), 16, (int)(dvoff[j] | past),
                                    n * 2, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < kDL; ++j) {
                const int64_t row = min(m0 + drow + 32 * j, M - 1), c = n + 8 * dch;
                dreg[j] = c < n_end ? load8(dy + row * N + c, c, N) : u32x4_t{0u, 0u, 0u, 0u};
            }
        }
    };
    auto load_w = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        const int n = (first + ks) * kStep;
        // the step's rows of W as a buffer of their own: rows past N read as zero
        const int left = n_end - n;
        const uint32_t bytes = (uint32_t)(left >= kStep ? kStep : left) * (uint32_t)K - (uint32_t)k0;
        i32x4_t wrs = buffer_rsrc(wq + (int64_t)n * K + k0, left > 0 ? bytes : 0u);
#pragma unroll
        for (int i = 0; i < 3; ++i) wrs[i] = __builtin_amdgcn_readfirstlane(wrs[i]);   // (is uniform: no loop over lanes)
#pragma unroll
        for (int j = 0; j < kWL; ++j)
            raw_buffer_load_lds(wrs, as_lds<uint32_t>(slot + kDB + 1024 * (kWaves * j + wave)), 16,
                                (int)(wvoff + (uint32_t)(kRL * kWaves * j) * (uint32_t)K), 0, 0, 0);
        const bool sok = n + lane < n_end;
        raw_buffer_load_lds(srs, as_lds<uint32_t>(slot + kDB + kWB + 256 * wave), 4,
                            (int)(sok ? 4u * (uint32_t)(n + lane) : 0x80000000u), 0, 0, 0);
    };
    auto load = [&](uint8_t* __restrict__ slot, int ks) __attribute__((always_inline)) {
        load_dy(slot, ks);
        load_w(slot, ks);
    };
    auto put_dy = [&](uint8_t* __restrict__ slot) __attribute__((always_inline)) {
        if (!DYV) {
#pragma unroll
            for (int j = 0; j < kDL; ++j)   // the layout a direct load writes: lane l at 16 l of its kilobyte
                *reinterpret_cast<u32x4_t*>(slot + 1024 * (kWaves * j + wave) + 16 * lane) = dreg[j];
        }
    };

    // ---- operand reads
    uint32_t offD[kKK], offC[NT];
#pragma unroll
    for (int kk = 0; kk < kKK; ++kk) offD[kk] = tile_byte(l32, 2 * kk + h);
    {   // lane j of a 16-lane group addresses row j / 2, columns 8 (j % 2) .. of the group's 8 x 16 codes
        const int j = l32 & 15, row = 8 * h + (j >> 1);
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const int c = 2 * (NT * wave + e) + (l32 >> 4);
            offC[e] = kDB + (uint32_t)(row * kBN + 16 * code_chunk<kBN>(row, c) + 8 * (j & 1));
        }
    }
    struct Codes {
        u32x2_t c[NT];
        f32x4_t s[2];
    };
    auto read_dy = [&](const uint8_t* __restrict__ slot, int kk, u32x4_t (&a)[MT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) a[i] = *reinterpret_cast<const u32x4_t*>(slot + offD[kk] + 4096u * i);
    };
    auto read_codes = [&](const uint8_t* __restrict__ slot, int kk, Codes& q) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < NT; ++e)   // 16 rows further down the swizzle repeats
            q.c[e] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                                     as_lds<__attribute__((ext_vector_type(2))) int>(
                                                         slot + offC[e] + 16 * kBN * kk)));
        const float* s = reinterpret_cast<const float*>(slot + kDB + kWB + 256 * wave) + 16 * kk + 8 * h;
        q.s[0] = *reinterpret_cast<const f32x4_t*>(s);
        q.s[1] = *reinterpret_cast<const f32x4_t*>(s + 4);
    };
    auto expand = [&](const Codes& q, u32x4_t (&b)[NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t c = q.c[e][p];
                const float f0 = (float)(int32_t)(int8_t)c * q.s[p][0], f1 = (float)(int32_t)(int8_t)(c >> 8) * q.s[p][1];
                const float f2 = (float)(int32_t)(int8_t)(c >> 16) * q.s[p][2], f3 = (float)((int32_t)c >> 24) * q.s[p][3];
                b[e][2 * p] = pack2<DT>(f0, f1);
                b[e][2 * p + 1] = pack2<DT>(f2, f3);
            }
    };

    // ---- A rows of the LoRA term as MFMA operands, ahead of the main loop (first 64 ranks)
    const rsrc_t ars = buf_rsrc(r ? A + (int64_t)k0 * r : nullptr, (uint64_t)min(K - k0, kBN) * r * 2);
    auto load_a = [&](int e, int kk) __attribute__((always_inline)) {
        const int row = 32 * (NT * wave + e) + l32, j = 16 * kk + 8 * h;
        if (AV)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   ars, j < r ? (uint32_t)(row * r + j) * 2u : 0x80000000u, 0, 0));
        return k0 + row < K && j < r ? load8(A + (int64_t)(k0 + row) * r + j, j, r) : u32x4_t{0u, 0u, 0u, 0u};
    };
    const rsrc_t urs = buf_rsrc(r ? u + (int64_t)m0 * r : nullptr, (uint64_t)min(M - m0, kBM) * r * 2);
    auto load_u = [&](int i, int kk) __attribute__((always_inline)) {
        const int row = 32 * i + l32, j = 16 * kk + 8 * h;
        if (AV)
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   urs, j < r ? (uint32_t)(row * r + j) * 2u : 0x80000000u, 0, 0));
        return m0 + row < M && j < r ? load8(u + (int64_t)(m0 + row) * r + j, j, r) : u32x4_t{0u, 0u, 0u, 0u};
    };
    load(s0, 0);
    put_dy(s0);
    if (RING > 2) {
        load(s1, 1);
        put_dy(s1);
    }
    u32x4_t av[NT][4];
    if (r)
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) av[e][kk] = load_a(e, kk);
    __builtin_amdgcn_sched_barrier(0);
    if (RING == 2) {
        load(s1, 1);
    } else {
        load(s2, 2);
        put_dy(s2);
    }
    // zeros from the matrix unit while the first tiles are on their way (256 register writes,
    // and the compiler's copies of them, took a microsecond)
    f32x16_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const u32x4_t z = {0u, 0u, 0u, 0u};
            acc[i][e] = mfma16<DT>(z, z, f32x16_t{});
        }
    // tiles 0 and 1 (of two slots, 0) have landed
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
    u32x4_t da[2][MT], wb[2][NT];
    Codes q[2];
    read_codes(s0, 0, q[0]);
    read_codes(s0, 1, q[1]);
    read_dy(s0, 0, da[0]);
    read_dy(s0, 1, da[1]);
    expand(q[0], wb[0]);

    // One MFMA depth: dy and codes of two depths on are read, the codes read a depth ago are
    // expanded for the next one.
    auto depth = [&](const uint8_t* __restrict__ from, int at, auto kkc, auto groups) __attribute__((always_inline)) {
        constexpr int p = decltype(kkc)::value & 1;
        u32x4_t dn[MT];
        Codes cn;
        read_dy(from, at, dn);
        read_codes(from, at, cn);
        expand(q[p ^ 1], wb[p ^ 1]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < NT; ++e) acc[i][e] = mfma16<DT>(wb[p][e], da[p][i], acc[i][e]);
#pragma unroll
        for (int i = 0; i < MT; ++i) da[p][i] = dn[i];
        q[p] = cn;
        if constexpr (DYV) {
#pragma unroll
            for (int g = 0; g < MT * NT; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (decltype(groups)::value) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 24 / MT + 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Four slots: step ks requests tile ks + 3; its end waits for tile ks + 2 only.
    auto step = [&](int ks, const uint8_t* __restrict__ cur, const uint8_t* __restrict__ next,
                    uint8_t* __restrict__ fill) __attribute__((always_inline)) {
        load_dy(fill, ks + 3);
        depth(cur, 2, IntC<0>{}, IntC<1>{});
        load_w(fill, ks + 3);
        depth(cur, 3, IntC<1>{}, IntC<1>{});
        depth(next, 0, IntC<2>{}, IntC<0>{});
        depth(next, 1, IntC<3>{}, IntC<0>{});
        put_dy(fill);
        if (DYV) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Two slots (a 256 x 256 tile's take 49 KB each): a tile is in registers after half of its
    // step; the one barrier of a step is there: its tile may then be overwritten, and the next
    // one, requested a whole step before, has landed.
    auto step2 = [&](int ks, uint8_t* cur, const uint8_t* next) __attribute__((always_inline)) {
        depth(cur, 2, IntC<0>{}, IntC<0>{});
        depth(cur, 3, IntC<1>{}, IntC<0>{});
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        load_dy(cur, ks + 2);
        depth(next, 0, IntC<2>{}, IntC<1>{});
        load_w(cur, ks + 2);
        depth(next, 1, IntC<3>{}, IntC<1>{});
    };
    // whole turns of the ring: steps past N multiply zeros
    if constexpr (RING == 2) {
        for (int ks = 0; ks < NS; ks += 2) {
            step2(ks, s0, s1);
            step2(ks + 1, s1, s0);
        }
    } else {
        for (int ks = 0; ks < NS; ks += 4) {
            step(ks, s0, s1, s3);
            step(ks + 1, s1, s2, s0);
            step(ks + 2, s2, s3, s1);
            step(ks + 3, s3, s0, s2);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last, empty tiles
    __syncthreads();

    if constexpr (SPLIT) {
        constexpr uint32_t kTileBytes = (uint32_t)MT * NT * 16 * 4 * kThreads;
        const int tile = mt * tn + nt;
        uint64_t* const flags = sp.tags + (size_t)tile * sp.splits;
        auto off = [&](int i, int e, int v4) { return (uint32_t)((((i * NT + e) * 4 + v4) * kThreads + tid) * 16); };
        if (split < sp.splits - 1) {
            const rsrc_t rs = buf_rsrc(sp.part + ((size_t)split * tiles + tile) * kTileBytes, kTileBytes);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        const f32x4_t v = {acc[i][e][4 * v4], acc[i][e][4 * v4 + 1], acc[i][e][4 * v4 + 2],
                                           acc[i][e][4 * v4 + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rs, off(i, e, v4), 0,
                                                               kCoherent);
                    }
            publish_tag(flags + split, launch_tag());
            return;
        }
        const bool fail = wait_tags(flags, sp.splits - 1, launch_tag());
        // the parts' sums in order, this one's last: tot + acc
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            f32x4_t tot[NT][4];
#pragma unroll
            for (int e = 0; e < NT; ++e)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) tot[e][v4] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            for (int p = 0; p < sp.splits - 1; ++p) {
                const rsrc_t rs = buf_rsrc(sp.part + ((size_t)p * tiles + tile) * kTileBytes, kTileBytes);
                u32x4_t gv[NT][4];
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
                        gv[e][v4] = __builtin_amdgcn_raw_buffer_load_b128(rs, off(i, e, v4), 0, kCoherent);
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
#pragma unroll
                        for (int c = 0; c < 4; ++c) tot[e][v4][c] += __uint_as_float(gv[e][v4][c]);
            }
#pragma unroll
            for (int e = 0; e < NT; ++e)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][e][v] = fail ? __builtin_nanf("") : tot[e][v >> 2][v & 3] + acc[i][e][v];
        }
    }

    // ---- epilogue, 32 tokens at a time: u A^T, rounding, and out through s0 and s1 in turn.
    // Lane (h, l32): token l32, columns 32 e + 8 v4 + 4 h + 0..3 of the wave's.
    constexpr int kRow = 2 * kBN, kCh = kBN / 8, kMask = (kCh < 16 ? kCh : 16) - 1;
    static_assert(32 * kRow <= kSlot, "32 output rows fit a slot");
    const rsrc_t xrs = buf_rsrc(dx + (int64_t)m0 * K, (uint64_t)min(M - m0, kBM) * K * 2);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if constexpr (MT * NT >= 16)
#pragma unroll
            for (int e = 0; e < NT; ++e) asm volatile("" : "+a"(acc[i][e]));
        if (r) {   // (ranks past r are zero: 32 at a time, so that the sums keep their registers)
            auto rank16 = [&](const u32x4_t (&a)[NT], u32x4_t uv) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < NT; ++e) acc[i][e] = mfma16<DT>(a[e], uv, acc[i][e]);
            };
            u32x4_t a[NT];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (kk == 2 && r <= 32) break;
#pragma unroll
                for (int e = 0; e < NT; ++e) a[e] = av[e][kk];
                rank16(a, load_u(i, kk));
            }
            for (int kk = 4; 16 * kk < r; ++kk) {
#pragma unroll
                for (int e = 0; e < NT; ++e) a[e] = load_a(e, kk);
                rank16(a, load_u(i, kk));
            }
        }
        uint8_t* const slot = (i & 1) ? s1 : s0;
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                const u32x2_t o = {pack2<DT>(acc[i][e][4 * v4], acc[i][e][4 * v4 + 1]),
                                   pack2<DT>(acc[i][e][4 * v4 + 2], acc[i][e][4 * v4 + 3])};
                const int cc = 4 * (NT * wave + e) + v4;
                *reinterpret_cast<u32x2_t*>(slot + l32 * kRow + 16 * (cc ^ (l32 & kMask)) + 8 * h) = o;
            }
        __syncthreads();   // the slot written two rounds ago was read before the last barrier
#pragma unroll
        for (int p = 0; p < 32 * kCh / kThreads; ++p) {
            const int c = tid + kThreads * p, cc = c % kCh, rr = c / kCh;
            const int row = 32 * i + rr, k = k0 + 8 * cc;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(slot + rr * kRow + 16 * (cc ^ (rr & kMask)));
            // rows past M lie past the buffer and are dropped, as are columns past K
            __builtin_amdgcn_raw_buffer_store_b128(
                v, xrs, k < K ? ((uint32_t)row * (uint32_t)K + (uint32_t)k) * 2u : 0x80000000u, 0, 0);
        }
    }
}

template <int MT, int NT, int RING, bool SPLIT>
qlora_status run(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u, const uint16_t* A,
                 uint16_t* dx, int M, int N, int K, int r, int dt, bool dyv, int splits, void* ws, hipStream_t s) {
    constexpr int kBM = 32 * MT, kBN = 32 * NT * kWaves;
    const int tm = (int)(((int64_t)M + kBM - 1) / kBM), tn = (int)(((int64_t)K + kBN - 1) / kBN), gm = 4;
    const int64_t tiles = (int64_t)tm * tn;
    Split sp{};
    if (SPLIT) {
        const int steps = (int)(((int64_t)N + kStep - 1) / kStep);
        sp.per = (steps + splits - 1) / splits;
        sp.splits = (steps + sp.per - 1) / sp.per;
        sp.tags = static_cast<uint64_t*>(ws);
        sp.part = static_cast<uint8_t*>(ws) + align256((size_t)(tiles * splits) * 8);
    }
    const int64_t total = tiles * (SPLIT ? sp.splits : 1);
    if (total * kThreads >= (int64_t(1) << 32) || (int64_t)gm * tn >= (int64_t(1) << 31))
        return QLORA_ERR_UNSUPPORTED_SHAPE;
    const bool av = r % 8 == 0;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_DX(V, W)                                                                                            \
    hipLaunchKernelGGL((int8_gemm_dx_kernel<MT, NT, RING, SPLIT, V, W, DT>), dim3((unsigned)total), dim3(kThreads), 0, s, dy, \
                       wq, sw, u, A, dx, M, N, K, r, tm, tn, gm, sp)
        if constexpr (NT == 2) {   // (chosen for direct loads only)
            if (av) QL_DX(true, true); else QL_DX(true, false);
        } else if (dyv) {
            if (av) QL_DX(true, true); else QL_DX(true, false);
        } else {
            if (av) QL_DX(false, true); else QL_DX(false, false);
        }
#undef QL_DX
    });
    return launch_status();
}

}  // namespace

size_t int8_gemm_dx_workspace(int64_t M, int64_t N, int64_t K) {
    const Int8Choice c = int8_dx_choice(M, N, K, true);
    if (c.splits == 1) return 0;
    const int64_t tiles = tiles_of(M, K, 128, 256);
    return align256((size_t)(tiles * c.splits) * 8) + (size_t)(tiles * (c.splits - 1)) * 128 * 256 * 4;
}

qlora_status launch_int8_gemm_bwd_dx(const uint16_t* dy, const int8_t* wq, const float* sw, const uint16_t* u,
                                     const uint16_t* A, uint16_t* dx, int M, int N, int K, int r, int dt, void* ws,
                                     hipStream_t s) {
    const bool dyv = direct_dy(N);
    const Int8Choice c = int8_dx_choice(M, N, K, ws != nullptr);
    switch (c.tile) {
        case kDx256x256: return run<8, 2, 2, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        case kDx128x256:
            return c.splits > 1 ? run<4, 2, 4, true>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, c.splits, ws, s)
                                : run<4, 2, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        case kDx128x128: return run<4, 1, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
        default: return run<2, 1, 4, false>(dy, wq, sw, u, A, dx, M, N, K, r, dt, dyv, 1, nullptr, s);
    }
}

}  // namespace qlora
