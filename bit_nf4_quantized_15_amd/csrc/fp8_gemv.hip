// Decode-size forward of the 8-bit float layer (M <= 16 tokens), one launch:
//
//   y[m,n] = RNE_16( sum_k xq[m,k] wq[n,k] + sum_j t[m,j] B[j,n] ),   t = RNE_16(s x A)
//
// ("bitsandbytes deep dive", section 8.2: low-bit storage; 12.2: the LoRA side path.)  The
// layer is bound by the weight's N K bytes.  A workgroup of 8 waves takes 16 weight rows at a
// time; a wave takes runs of four blocks (512 consecutive bytes of each row), the waves' runs
// round robin, and a lane's 32 bytes of a block are an operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 as they come, the block's two scales included: the byte of
// the weight's block and that of the token's lie, four blocks to a dword, where the
// instruction's byte selectors pick them.  Weights go straight to registers, one run in flight
// behind the one being multiplied, across row tiles.
//
// x is quantized by every workgroup for itself, block by block, where its codes fit beside the
// rest in LDS; larger x come as codes.
//
// LoRA.  t needs all of A; workgroups 0 .. P - 1 each sum a range of K into an fp32 partial and
// publish it with the launch's tag (split_sync.h); the others add the P partials in order, after
// their first row tile's products, while later weights stream.  t B runs on the 16-bit MFMA over
// the same accumulators' layout.  t is rounded to 16 bits, also where the caller keeps none.
//
// Traced, us, weights in the caches after the first call: 1 token 4096 -> 4096, r = 16: 7.9, the hand-off of t and the
// reduction's end (17 MB would stream in 3.3); 13 tokens 4096 -> 11008, r = 64, fp16: 19, where each
// workgroup quantizes x and waits for t before its first row tile ends (47 MB: 9.2).
#include "fp8.h"
#include "split_sync.h"

namespace qlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kNone = 0x80000000u;   // past every buffer here: reads zero

__device__ __forceinline__ u32x4_t load16(rsrc_t rs, uint32_t at) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
}

template <int DT>
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    if (DT == kDtF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

constexpr int kWaves = 8, kThreads = 512, kRows = 16;
constexpr int kProducers = 16;                          // at most
constexpr int kRun = 4;                                 // blocks of a run

struct GemvArgs {
    const uint16_t* x;      // 16-bit x: quantized here, and the producers' operand
    const uint8_t* xq;      // or its codes [M, ld] and scale bytes [block][rs]
    const uint8_t* sx;
    const uint8_t* w;
    const uint8_t* sw;      // [block of rows][wrs]
    const uint16_t* t;      // given, or null with producers
    const uint16_t* A;
    const uint16_t* B;
    uint16_t* y;
    uint16_t* t_out;
    uint64_t* tags;
    float* part;            // [P][16][rp]
    int64_t rs, wrs;
    int M, N, K, ld, r, rp, P, slice, tiles;
    float scale;
};

// LDS: the wait's verdict, a reduction buffer, B's 16 columns and t (rows of their rank, in whole
// 32s, and 8 halves), the scales of x (16 tokens of whole runs), then x's codes.
__host__ __device__ constexpr int runs_of(int K) { return (K + kRun * kFp8Block - 1) / (kRun * kFp8Block); }
constexpr int kOffRed = 16, kOffB = kOffRed + kWaves * 64 * 16;
__host__ __device__ constexpr int t_ld(int r) { return ((r + 31) & ~31) + 8; }
__host__ __device__ constexpr int off_t(int r) { return kOffB + (r ? kRows * t_ld(r) * 2 : 0); }
__host__ __device__ constexpr int off_s(int r) { return off_t(r) + (r ? kRows * t_ld(r) * 2 : 0); }
__host__ __device__ constexpr int off_x(int r, int K) { return off_s(r) + kRows * 4 * (runs_of(K) | 1) + 15 & ~15; }

// Partial products of x A over this producer's range of K: [16][rp] fp32.
template <int DT>
__device__ __forceinline__ void produce(const GemvArgs& a, int p, uint8_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int k0 = p * a.slice, k1 = min(a.K, k0 + a.slice), q_n = a.rp >> 4;
    const rsrc_t xrs = buf_rsrc(a.x, (uint32_t)a.M * (uint32_t)a.K * 2u);
    const rsrc_t ars = buf_rsrc(a.A, (uint32_t)a.K * (uint32_t)a.r * 2u);
    f32x4_t acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = k0 + 32 * wave; k < k1; k += 32 * kWaves) {   // (ranges are whole 32s)
        const u32x4_t xv = load16(xrs, i < a.M ? ((uint32_t)i * (uint32_t)a.K + (uint32_t)(k + 8 * g)) * 2u : kNone);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q >= q_n) break;
            const int j = 16 * q + i;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t o = j < a.r ? ((uint32_t)(k + 8 * g + 2 * e) * (uint32_t)a.r + (uint32_t)j) * 2u : kNone;
                const uint32_t lo = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ars, o, 0, 0);
                const uint32_t hi = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ars, o + 2u * (uint32_t)a.r, 0, 0);
                w[e] = lo | (hi << 16);
            }
            acc[q] = mfma16<DT>(u32x4_t{w[0], w[1], w[2], w[3]}, xv, acc[q]);   // rows: ranks, columns: tokens
        }
    }
    float* const red = reinterpret_cast<float*>(lds);   // [wave][q][lane][4]
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < q_n) *reinterpret_cast<f32x4_t*>(red + ((wave * 8 + q) * 64 + lane) * 4) = acc[q];
    __syncthreads();
    if (wave < q_n) {
        f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const f32x4_t t = *reinterpret_cast<const f32x4_t*>(red + ((v * 8 + wave) * 64 + lane) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += t[e];
        }
        const rsrc_t prs = buf_rsrc(a.part, (uint32_t)(a.P * 16 * a.rp) * 4u);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, s), prs,
                                               (uint32_t)((p * 16 + i) * a.rp + 16 * wave + 4 * g) * 4u, 0, kCoherent);
    }
    publish_tag(a.tags + p, launch_tag());
}

// x's codes and scale bytes into LDS: 16 lanes take a block, 16 bytes each.  `first` holds the
// blocks that a lane's group takes first, requested by the caller.
template <int DT>
struct SelfQuant {
    static constexpr int kHold = 4, kGroups = kThreads / 16;
    u32x4_t first[kHold];
    __device__ __forceinline__ u32x4_t get(const GemvArgs& a, rsrc_t xrs, int b, int nb) const {
        const int row = b / nb, c = (b - row * nb) * kFp8Block + 8 * ((int)threadIdx.x & 15);
        return load16(xrs, ((row < a.M) & (c < a.K)) ? ((uint32_t)row * (uint32_t)a.K + (uint32_t)c) * 2u : kNone);
    }
    __device__ __forceinline__ void request(const GemvArgs& a) {
        const int nb = (a.K + kFp8Block - 1) / kFp8Block;
        const rsrc_t xrs = buf_rsrc(a.x, (uint32_t)a.M * (uint32_t)a.K * 2u);
#pragma unroll
        for (int e = 0; e < kHold; ++e) first[e] = get(a, xrs, ((int)threadIdx.x >> 4) + kGroups * e, nb);
    }
    __device__ __forceinline__ void run(const GemvArgs& a, uint8_t* lds) {
        const int nb = (a.K + kFp8Block - 1) / kFp8Block, all = a.M * nb, l = threadIdx.x & 15;
        const rsrc_t xrs = buf_rsrc(a.x, (uint32_t)a.M * (uint32_t)a.K * 2u);
        uint8_t* const sc = lds + off_s(a.r);
        const int ld = 4 * (runs_of(a.K) | 1);
        auto put = [&](u32x4_t v, int b) __attribute__((always_inline)) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_mag2(m, v[i]);
            const uint32_t byte = fp8_scale_byte<DT>(max_row16(m));
            const int row = b / nb, k = b - row * nb;
            if (b < all) {
                if (l == 0) sc[row * ld + k] = (uint8_t)byte;
                *reinterpret_cast<u32x2_t*>(lds + off_x(a.r, a.K) + row * x_ld(a.K) + k * kFp8Block + 8 * l) =
                    fp8_codes8<DT>(v, byte);
            }
        };
        for (int b0 = 0; b0 < all; b0 += kGroups * kHold) {
            if (b0)
#pragma unroll
                for (int e = 0; e < kHold; ++e) first[e] = get(a, xrs, b0 + ((int)threadIdx.x >> 4) + kGroups * e, nb);
#pragma unroll
            for (int e = 0; e < kHold; ++e) put(first[e], b0 + ((int)threadIdx.x >> 4) + kGroups * e);
        }
    }
    // bytes of a row of codes in LDS: whole runs, and 16 to shift the rows' banks
    static __host__ __device__ constexpr int x_ld(int K) { return runs_of(K) * kRun * kFp8Block + 16; }
};

// (given codes double a run's registers: one workgroup on a CU)
template <bool SELF, int DT>
__global__ __launch_bounds__(kThreads, SELF ? 4 : 2) void fp8_gemv_kernel(const GemvArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    if ((int)blockIdx.x < a.P) {
        produce<DT>(a, blockIdx.x, lds);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)gridDim.x - a.P, runs = runs_of(a.K), nbk = (a.K + kFp8Block - 1) / kFp8Block;
    const int nb = (runs + kWaves - 1) / kWaves;        // runs of a wave
    const uint32_t woff = (uint32_t)i * (uint32_t)a.K + 32u * g;
    const uint32_t xm = (uint32_t)min(i, a.M - 1);      // tokens past M repeat the last: never stored
    const rsrc_t xrs = buf_rsrc(SELF ? nullptr : a.xq, SELF ? 0u : (uint32_t)a.M * (uint32_t)a.ld);
    struct Run {
        u32x4_t w[2 * kRun], x[SELF ? 1 : 2 * kRun];
        uint32_t sw, sx;
    };
    auto load = [&](Run& q, int tile, int b) __attribute__((always_inline)) {
        const int n0 = tile * kRows, s = wave + kWaves * b;
        const uint32_t bytes = tile < a.tiles ? (uint32_t)min(kRows, a.N - n0) * (uint32_t)a.K : 0u;
        const rsrc_t wrs = buf_rsrc(a.w + (int64_t)n0 * a.K, __builtin_amdgcn_readfirstlane(bytes));
        const uint8_t* sp = a.sw + (int64_t)(min(n0, a.N - 1) >> 7) * a.wrs;
        const rsrc_t srs = buf_rsrc(sp, tile < a.tiles ? (uint32_t)a.wrs : 0u);
        q.sw = __builtin_amdgcn_raw_buffer_load_b32(srs, s < runs ? 4u * (uint32_t)s : kNone, 0, 0);
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            const uint32_t k = (uint32_t)(s * kRun + e) * kFp8Block;
#pragma unroll
            for (int c = 0; c < 2; ++c) {   // (what lies past the row's end would be the next row's)
                const bool on = (s < runs) & (k + 32u * g + 16u * c < (uint32_t)a.K);
                q.w[2 * e + c] = load16(wrs, on ? woff + k + 16u * c : kNone);
                if (!SELF) q.x[SELF ? 0 : 2 * e + c] = load16(xrs, on ? xm * (uint32_t)a.ld + 32u * g + k + 16u * c : kNone);
            }
        }
    };

    int tile = (int)blockIdx.x - a.P, b = 0;
    Run q0, q1;
    uint8_t* const sc = lds + off_s(a.r);
    const int s_ld = 4 * (runs | 1);
    if constexpr (SELF) {
        SelfQuant<DT> sq;
        sq.request(a);
        load(q0, tile, 0);
        // blocks of a last run that K does not reach: code 0 (their scales would do for any, but NaN)
        const int used = (a.K + 7) / 8, all = runs * kRun * kFp8Block / 8;
        for (int v = tid; v < a.M * (all - used); v += kThreads) {
            const int row = v / (all - used), c = used + v - row * (all - used);
            *reinterpret_cast<u32x2_t*>(lds + off_x(a.r, a.K) + row * SelfQuant<DT>::x_ld(a.K) + 8 * c) = u32x2_t{0u, 0u};
        }
        for (int v = tid; v < a.M * runs; v += kThreads) *reinterpret_cast<uint32_t*>(sc + (v / runs) * s_ld + 4 * (v % runs)) = 0u;
        __syncthreads();
        sq.run(a, lds);
        __syncthreads();
    } else {
        load(q0, tile, 0);
        for (int v = tid; v < a.M * runs * kRun; v += kThreads) {
            const int row = v / (runs * kRun), k = v - row * (runs * kRun);
            sc[row * s_ld + k] = k < nbk ? a.sx[(int64_t)k * a.rs + row] : 0;
        }
        __syncthreads();
    }

    const int rp32 = (a.r + 31) & ~31;
    const rsrc_t brs = buf_rsrc(a.r ? a.B : nullptr, (uint32_t)a.r * (uint32_t)a.N * 2u);
    const int ld = t_ld(a.r);
    uint16_t* const tl = reinterpret_cast<uint16_t*>(lds + off_t(a.r));
    uint16_t* const bt = reinterpret_cast<uint16_t*>(lds + kOffB);
    uint8_t* const red = lds + kOffRed;
    const uint8_t* const xl = lds + off_x(a.r, a.K) + (SELF ? xm * (uint32_t)SelfQuant<DT>::x_ld(a.K) + 32u * g : 0u);
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    int turn = 0;                                       // row tiles done
    auto finish = [&]() __attribute__((always_inline)) {
        const int n0 = tile * kRows;
        if (turn) __syncthreads();   // (the buffers of the tile before have been read)
        *reinterpret_cast<f32x4_t*>(red + (wave * 64 + lane) * 16) = acc;
        // B's 16 columns, [n][j]: zero past r
        uint16_t bv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = (tid >> 4) + 32 * e, n = n0 + (tid & 15);
            bv[e] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                brs, ((j < a.r) & (n < a.N)) ? ((uint32_t)j * (uint32_t)a.N + (uint32_t)n) * 2u : kNone, 0, 0);
        }
        if (turn == 0 && a.r) {                         // t into LDS, zero past r
            bool fail = false;
            if (a.P) {
                if (wave == 0) {
                    fail = wait_tags(a.tags, a.P, launch_tag());
                    if (lane == 0) *reinterpret_cast<uint32_t*>(lds) = fail;
                }
                __syncthreads();
                fail = *reinterpret_cast<const uint32_t*>(lds) != 0u;
            }
            const rsrc_t prs = buf_rsrc(a.part, a.P ? (uint32_t)(a.P * 16 * a.rp) * 4u : 0u);
            for (int v = tid; v < kRows * rp32; v += kThreads) {
                const int m = v / rp32, j = v - m * rp32;
                uint16_t o = 0;
                if (m < a.M && j < a.r) {
                    if (a.P) {
                        uint32_t pv[kProducers];
#pragma unroll
                        for (int p = 0; p < kProducers; ++p)
                            pv[p] = __builtin_amdgcn_raw_buffer_load_b32(
                                prs, p < a.P ? (uint32_t)((p * 16 + m) * a.rp + j) * 4u : kNone, 0, kCoherent);
                        float s = 0.0f;
#pragma unroll
                        for (int p = 0; p < kProducers; ++p) s += __uint_as_float(pv[p]);
                        o = (uint16_t)(pack2<DT>(fail ? __builtin_nanf("") : a.scale * s, 0.0f) & 0xFFFFu);
                    } else {
                        o = a.t[(int64_t)m * a.r + j];
                    }
                    if (a.t_out && (int)blockIdx.x == a.P) a.t_out[(int64_t)m * a.r + j] = o;
                }
                tl[m * ld + j] = o;
            }
        }
        if (a.r)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (32 * e < rp32) bt[(tid & 15) * ld + (tid >> 4) + 32 * e] = bv[e];
        __syncthreads();
        if (wave == (turn & (kWaves - 1))) {
            f32x4_t f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                const f32x4_t p = *reinterpret_cast<const f32x4_t*>(red + (v * 64 + lane) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] += p[e];
            }
            // lane: token i, outputs n0 + 4 g + e
            const int n = n0 + 4 * g;
            for (int j = 0; j < rp32; j += 32)
                f = mfma16<DT>(*reinterpret_cast<const u32x4_t*>(bt + i * ld + j + 8 * g),
                               *reinterpret_cast<const u32x4_t*>(tl + i * ld + j + 8 * g), f);
            if (i < a.M) {
                uint16_t* o = a.y + (int64_t)i * a.N + n;
                const u32x2_t v = {pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])};
                if ((a.N & 3) == 0) {
                    if (n < a.N) *reinterpret_cast<u32x2_t*>(o) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < a.N) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
        acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        ++turn;
    };
    auto body = [&](const Run& cur, Run& nxt) __attribute__((always_inline)) {
        const bool end = b + 1 == nb;
        load(nxt, end ? tile + G : tile, end ? 0 : b + 1);
        // (blocks and runs past K: codes of w are zero, and so are its scales, whatever pads them)
        const int s = min(wave + kWaves * b, runs - 1), left = nbk - kRun * (wave + kWaves * b);
        const uint32_t sw = left >= kRun ? cur.sw : left > 0 ? cur.sw & ((1u << (8 * left)) - 1u) : 0u;
        const uint32_t sx = *reinterpret_cast<const uint32_t*>(sc + xm * s_ld + 4 * s);
        u32x4_t xv[2 * kRun];
#pragma unroll
        for (int e = 0; e < 2 * kRun; ++e)
            xv[e] = SELF ? *reinterpret_cast<const u32x4_t*>(xl + (uint32_t)s * (kRun * kFp8Block) + 128u * (e >> 1) + 16u * (e & 1))
                         : cur.x[SELF ? 0 : e];
        auto join = [](u32x4_t a, u32x4_t b) __attribute__((always_inline)) {
            return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        };
#define QL_STEP(E)                                                                                                   \
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(cur.w[2 * E], cur.w[2 * E + 1]), join(xv[2 * E], xv[2 * E + 1]), \
                                                           acc, 0, 0, E, (int)sw, E, (int)sx)
        QL_STEP(0);
        QL_STEP(1);
        QL_STEP(2);
        QL_STEP(3);
#undef QL_STEP
        if (end) {
            finish();
            tile += G;
            b = 0;
        } else {
            ++b;
        }
    };
    while (true) {
        body(q0, q1);
        if (tile >= a.tiles) break;
        body(q1, q0);
        if (tile >= a.tiles) break;
    }
}

}  // namespace

static int rank_pad(int r) { return (r + 15) & ~15; }

size_t fp8_gemv_workspace(int r) {
    return r ? align256(kProducers * 8) + align256((size_t)kProducers * 16 * rank_pad(r) * 4) : 0;
}

qlora_status launch_fp8_gemv(const Fp8Gemm& gm, const uint16_t* x, const uint16_t* A, float scale, uint16_t* t_out,
                             void* ws, int dt, hipStream_t s) {
    GemvArgs a{};
    a.x = x;
    a.xq = gm.x;
    a.sx = gm.sx;
    a.w = gm.w;
    a.sw = gm.sw;
    a.t = gm.t;
    a.A = A;
    a.B = gm.L;
    a.y = gm.out;
    a.t_out = t_out;
    a.rs = gm.rs;
    a.wrs = gm.wrs;
    a.M = gm.M;
    a.N = gm.N;
    a.K = gm.K;
    a.ld = gm.ld;
    a.r = gm.r;
    a.rp = rank_pad(gm.r);
    a.scale = scale;
    a.tiles = (int)(((int64_t)gm.N + kRows - 1) / kRows);
    if (a.r && !a.t) {
        a.P = std::min(a.r > 32 ? kProducers : kProducers / 2, (a.K + 255) / 256);
        a.slice = ((a.K + a.P - 1) / a.P + 31) / 32 * 32;
        a.tags = static_cast<uint64_t*>(ws);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(kProducers * 8));
    }
    const bool self = gm.x == nullptr;
    const size_t need = std::max<size_t>(off_x(a.r, a.K) + (self ? (size_t)a.M * SelfQuant<0>::x_ld(a.K) : 0),
                                         a.P ? kWaves * 8 * 64 * 16 : 0);
    // Two workgroups on a CU stream a little better; one quantizes x once where two would twice.
    // 11008 x 4096, r = 64, us, 512 and 256 workgroups: 1 token 15.8, 17.8; 13 tokens 20.6, 18.2.
    const unsigned grid = (unsigned)(a.P + std::min(a.tiles, a.M > 4 ? 256 : 512));
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        if (self) hipLaunchKernelGGL((fp8_gemv_kernel<true, DT>), dim3(grid), dim3(kThreads), need, s, a);
        else hipLaunchKernelGGL((fp8_gemv_kernel<false, DT>), dim3(grid), dim3(kThreads), need, s, a);
    });
    return launch_status();
}

}  // namespace qlora
