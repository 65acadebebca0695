// Decode-size forward of the int8 layer (M <= 16 tokens), one launch:
//
//   y[m,n] = RNE_16( sx[m] sw[n] sum_k xq[m,k] wq[n,k] + sum_j t[m,j] B[j,n] )
//
// ("bitsandbytes deep dive", section 4: vector-wise int8; 12.2: the LoRA side path.)  The
// layer is bound by the weight's N K bytes.  A workgroup of 8 waves takes 16 weight rows at
// a time; its waves deal the 64-wide steps of K round robin, so together they read 512
// consecutive bytes of each row, and a lane's 16 bytes are an operand of
// v_mfma_i32_16x16x64_i8 as they come: no conversion at all.  Weights go straight to
// registers, a batch of steps in flight behind the one being multiplied, across row tiles.
//
// x is quantized by every workgroup for itself where its codes fit beside the rest in LDS
// (M (K + 16) <= 72 KB): 2 M K bytes from L2 next to 16 K of weights, and no launch before
// this one.  Larger x come as codes.
//
// LoRA.  t = RNE_16(s x A) needs all of A; workgroups 0 .. P - 1 each sum a range of K into an
// fp32 partial and publish it with the launch's tag (split_sync.h); the others add the P
// partials in order, after their first row tile's products, while later weights stream.
// t B runs on the 16-bit MFMA over the same accumulators' layout.
//
// t is rounded to 16 bits as everywhere (int8_prep.hip), also where the caller keeps none.
//
// Traced, weights from HBM: 1 token 4096 -> 4096, r = 16: 9.6 us, of which 3.5 are the weight's
// bytes (r = 0: 8.7; t's hand-off and the reduction's end are the rest); 13 tokens 4096 -> 11008,
// r = 64: 22 us; 4 tokens 8192 -> 28672, r = 16: 49 us, 4.8 TB/s.
#include "int8.h"
#include "lora_plan.h"
#include "split_sync.h"

namespace qlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
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

constexpr int kWaves = 8, kThreads = 512, kRows = 16;
constexpr int kProducers = 8;

struct GemvArgs {
    const uint16_t* x;      // 16-bit x: quantized here, and the producers' operand
    const int8_t* xq;       // or its codes and scales
    const float* sx;
    const int8_t* w;
    const float* sw;
    const uint16_t* t;      // given, or null with producers
    const uint16_t* A;
    const uint16_t* B;
    uint16_t* y;
    uint16_t* t_out;
    uint64_t* tags;
    float* part;            // [P][16][rp]
    int M, N, K, r, rp, P, slice, tiles;
    float scale;
};

// LDS: 16 scales and the wait's verdict, a reduction buffer, B's 16 columns and t (rows of
// their rank, in whole 32s, and 8 halves), then x's codes.  16 tokens of 4096 at rank 64 leave
// room for two workgroups on a CU.
constexpr int kOffS = 0, kOffRed = 256, kOffB = kOffRed + kWaves * 64 * 16;
__host__ __device__ constexpr int t_ld(int r) { return ((r + 31) & ~31) + 8; }
__host__ __device__ constexpr int off_t(int r) { return kOffB + (r ? kRows * t_ld(r) * 2 : 0); }
__host__ __device__ constexpr int off_x(int r) { return off_t(r) + (r ? kRows * t_ld(r) * 2 : 0); }

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
        const u32x4_t xv = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
            xrs, i < a.M ? ((uint32_t)i * (uint32_t)a.K + (uint32_t)(k + 8 * g)) * 2u : kNone, 0, 0));
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

// x's codes and scales into LDS.  Each row is shared by G waves; `first` holds a lane's
// chunks of its first row, requested by the caller.
template <int DT>
struct SelfQuant {
    static constexpr int kHold = 8;   // 16-byte chunks of a row a lane keeps
    u32x4_t first[kHold];
    int G, nch;
    __device__ __forceinline__ void request(const GemvArgs& a, int wave, int lane) {
        nch = a.K >> 3;
        G = a.M == 1 ? 8 : a.M == 2 ? 4 : a.M <= 4 ? 2 : 1;
        const int row = wave / G, c0 = (wave % G) * 64 + lane;
        const rsrc_t xrs = buf_rsrc(a.x, (uint32_t)a.M * (uint32_t)a.K * 2u);
#pragma unroll
        for (int e = 0; e < kHold; ++e) {
            const int c = c0 + 64 * G * e;
            first[e] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                xrs, ((row < a.M) & (c < nch)) ? ((uint32_t)row * (uint32_t)nch + (uint32_t)c) * 16u : kNone, 0, 0));
        }
    }
    __device__ __forceinline__ void run(const GemvArgs& a, int wave, int lane, uint8_t* lds) {
        uint32_t* const am = reinterpret_cast<uint32_t*>(lds + kOffRed);   // [wave]
        float* const sxs = reinterpret_cast<float*>(lds + kOffS);
        const int per = kWaves / G, part = wave % G;
        for (int p = 0; p * per < a.M; ++p) {
            const int row = p * per + wave / G;
            const u32x4_t* xr = reinterpret_cast<const u32x4_t*>(a.x) + (int64_t)min(row, a.M - 1) * nch;
            const bool on = row < a.M;
            const int c0 = part * 64 + lane;
            if (p > 0) {
#pragma unroll
                for (int e = 0; e < kHold; ++e) first[e] = xr[min(c0 + 64 * G * e, nch - 1)];
            }
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < kHold; ++e)
                if (c0 + 64 * G * e < nch)
#pragma unroll
                    for (int i = 0; i < 4; ++i) m = max_abs2(m, first[e][i]);
            for (int c = c0 + 64 * G * kHold; c < nch; c += 64 * G) {
                const u32x4_t v = xr[c];
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max_abs2(m, v[i]);
            }
            uint32_t top = max(m & 0xFFFFu, m >> 16);
#pragma unroll
            for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
            if (lane == 0) am[wave] = top;
            __syncthreads();
            for (int e = 0; e < G; ++e) top = max(top, am[wave - part + e]);
            const RowScale rs = row_scale<DT>(top);
            uint8_t* const xl = lds + off_x(a.r) + (size_t)min(row, a.M - 1) * (a.K + 16);
            if (on) {
                if (part == 0 && lane == 0) sxs[row] = rs.scale;
#pragma unroll
                for (int e = 0; e < kHold; ++e) {
                    const int c = c0 + 64 * G * e;
                    if (c < nch) *reinterpret_cast<u32x2_t*>(xl + 8 * c) = codes8<DT>(first[e], rs);
                }
                for (int c = c0 + 64 * G * kHold; c < nch; c += 64 * G)
                    *reinterpret_cast<u32x2_t*>(xl + 8 * c) = codes8<DT>(xr[c], rs);
            }
            __syncthreads();
        }
    }
};

template <bool SELF, int DT>
__global__ __launch_bounds__(kThreads, 4) void int8_gemv_kernel(const GemvArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    if ((int)blockIdx.x < a.P) {
        produce<DT>(a, blockIdx.x, lds);
        return;
    }
    constexpr int D = SELF ? 8 : 4;                     // 64-wide steps per wave and batch
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)gridDim.x - a.P, KS = a.K >> 6;
    const int nb = ((KS + kWaves - 1) / kWaves + D - 1) / D;

    const uint32_t woff = (uint32_t)i * (uint32_t)a.K + 16u * g;
    const uint32_t xm = (uint32_t)min(i, a.M - 1);      // tokens past M repeat the last: never stored
    const uint32_t xoff = SELF ? xm * (uint32_t)(a.K + 16) + 16u * g : xm * (uint32_t)a.K + 16u * g;
    const rsrc_t xrs = buf_rsrc(SELF ? nullptr : a.xq, SELF ? 0u : (uint32_t)a.M * (uint32_t)a.K);
    struct Batch {
        u32x4_t w[D], x[SELF ? 1 : D];
    };
    auto load = [&](Batch& q, int tile, int b) __attribute__((always_inline)) {
        const int n0 = tile * kRows;
        const uint32_t bytes = tile < a.tiles ? (uint32_t)min(kRows, a.N - n0) * (uint32_t)a.K : 0u;
        const rsrc_t wrs = buf_rsrc(a.w + (int64_t)n0 * a.K, __builtin_amdgcn_readfirstlane(bytes));
#pragma unroll
        for (int e = 0; e < D; ++e) {
            const int s = wave + kWaves * (b * D + e);
            const uint32_t so = s < KS ? 64u * (uint32_t)s : kNone;   // steps past K read zero
            q.w[e] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wrs, woff + so, 0, 0));
            if (!SELF) q.x[SELF ? 0 : e] =
                __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xrs, xoff + so, 0, 0));
        }
    };

    int tile = (int)blockIdx.x - a.P, b = 0;
    Batch q0, q1;
    if constexpr (SELF) {
        SelfQuant<DT> sq;
        sq.request(a, wave, lane);
        load(q0, tile, 0);
        sq.run(a, wave, lane, lds);
    } else {
        load(q0, tile, 0);
        if (tid < kRows) reinterpret_cast<float*>(lds + kOffS)[tid] = a.sx[min(tid, a.M - 1)];
    }

    const int rp32 = (a.r + 31) & ~31;
    const rsrc_t brs = buf_rsrc(a.r ? a.B : nullptr, (uint32_t)a.r * (uint32_t)a.N * 2u);
    const int ld = t_ld(a.r), xat = off_x(a.r);
    uint16_t* const tl = reinterpret_cast<uint16_t*>(lds + off_t(a.r));
    uint16_t* const bt = reinterpret_cast<uint16_t*>(lds + kOffB);
    uint8_t* const red = lds + kOffRed;
    i32x4_t acc = {0, 0, 0, 0};
    int turn = 0;                                       // row tiles done
    auto finish = [&]() __attribute__((always_inline)) {
        const int n0 = tile * kRows;
        if (turn) __syncthreads();   // (the buffers of the tile before have been read)
        *reinterpret_cast<i32x4_t*>(red + (wave * 64 + lane) * 16) = acc;
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
                    if (lane == 0) *reinterpret_cast<uint32_t*>(lds + kOffS + 128) = fail;
                }
                __syncthreads();
                fail = *reinterpret_cast<const uint32_t*>(lds + kOffS + 128) != 0u;
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
            i32x4_t s = {0, 0, 0, 0};
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                const i32x4_t p = *reinterpret_cast<const i32x4_t*>(red + (v * 64 + lane) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += p[e];
            }
            // lane: token i, outputs n0 + 4 g + e
            float sx = reinterpret_cast<const float*>(lds + kOffS)[min(i, a.M - 1)];
            const float up = loud_scale(sx) ? kLoudUp : 1.0f;
            if (loud_scale(sx)) sx *= kLoudDown;
            const int n = n0 + 4 * g;
            f32x4_t f;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (float)s[e] * sx * a.sw[min(n + e, a.N - 1)] * up;
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
        acc = i32x4_t{0, 0, 0, 0};
        ++turn;
    };
    auto body = [&](const Batch& cur, Batch& nxt) __attribute__((always_inline)) {
        const bool end = b + 1 == nb;
        load(nxt, end ? tile + G : tile, end ? 0 : b + 1);
#pragma unroll
        for (int e = 0; e < D; ++e) {
            i32x4_t xv;
            if constexpr (SELF) {
                const int s = min(wave + kWaves * (b * D + e), KS - 1);
                xv = *reinterpret_cast<const i32x4_t*>(lds + xat + xoff + 64u * (uint32_t)s);
            } else {
                xv = __builtin_bit_cast(i32x4_t, cur.x[e]);
            }
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, cur.w[e]), xv, acc, 0, 0, 0);
        }
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

size_t int8_gemv_workspace(int r) {
    return r ? align256(kProducers * 8) + align256((size_t)kProducers * 16 * rank_pad(r) * 4) : 0;
}

qlora_status launch_int8_gemv(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                              const uint16_t* t, const uint16_t* A, const uint16_t* B, float scale, uint16_t* y,
                              uint16_t* t_out, void* ws, int M, int N, int K, int r, int dt, hipStream_t s) {
    GemvArgs a{};
    a.x = x;
    a.xq = xq;
    a.sx = sx;
    a.w = wq;
    a.sw = sw;
    a.t = t;
    a.A = A;
    a.B = B;
    a.y = y;
    a.t_out = t_out;
    a.M = M;
    a.N = N;
    a.K = K;
    a.r = r;
    a.rp = rank_pad(r);
    a.scale = scale;
    a.tiles = (int)(((int64_t)N + kRows - 1) / kRows);
    if (r && !t) {
        a.P = std::min(kProducers, (K + 255) / 256);
        a.slice = ((K + a.P - 1) / a.P + 31) / 32 * 32;
        a.tags = static_cast<uint64_t*>(ws);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(kProducers * 8));
    }
    const bool self = xq == nullptr;
    const size_t need = std::max<size_t>(off_x(r) + (self ? (size_t)M * (K + 16) : 0), a.P ? kWaves * 8 * 64 * 16 : 0);
    const unsigned grid = (unsigned)(a.P + std::min(a.tiles, 512));
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        if (self) hipLaunchKernelGGL((int8_gemv_kernel<true, DT>), dim3(grid), dim3(kThreads), need, s, a);
        else hipLaunchKernelGGL((int8_gemv_kernel<false, DT>), dim3(grid), dim3(kThreads), need, s, a);
    });
    return launch_status();
}

}  // namespace qlora
