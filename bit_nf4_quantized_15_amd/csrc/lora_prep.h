// The LoRA products that stream a 16-bit operand X [M, C] once and may do more with it on the way:
// out = RNE_16(scale drop(X) Y) (t of x, u of dy), and X's own 8-bit form, rows in blocks of 128
// (fp8_codes.h).
//
// A workgroup of 4 waves takes 128 tokens and a range of C, in blocks of 128 columns, the next two
// on their way while one is multiplied.  A wave loads whole 256-byte pieces of its 32 rows, 16
// lanes to a row, so that a row's maximum over the block is a rotation within the lanes' DPP row and
// its codes are one 128-byte store; what the mask leaves goes through LDS of the wave's own into
// MFMA operands.  Y's rows go through LDS for all four waves.  Where C is split, the fp32 sums of
// each range go to the workspace and a second kernel adds them in order, on all CUs.  (Adding them in the launch, by the
// workgroup of the last range as lora_body.h does, left that to one CU per 128 tokens: 333 x
// 11008, r = 8 took 24 us, 4096 x 11008, r = 64 38 us.)
//
// Traced, us, the pass and the second kernel: x 8192 x 8192, r = 64, dropout, with codes 50 + 7 (HBM: 4.0
// TB/s in the pass); dy 4096 x 11008, r = 64, with codes 32 + 5; x 333 x 11008, r = 8, dropout, with
// codes 7.9 + 4.7, latencies; t of three layers that share x 4096 x 4096, r = 64, dropout, 24 + 7:
// the generator's 12 us of every SIMD's time in the pass, whose x comes from the caches twice.
#pragma once

#include "fp8.h"
#include "lora_body.h"
#include "prep_plan.h"

namespace qlora {
namespace {

// What becomes of X itself: its codes [M][ld] (zeros from C to ld) and scale bytes [block][rs].
struct PrepCodes {
    uint8_t* codes;
    uint8_t* scale;
    int64_t ld, rs;
};

constexpr int kStreamItems = 8;
struct StreamItem {
    const uint16_t* X;
    const uint16_t* Y;
    uint16_t* out;
    float* part;                      // [split][M][rp], rp = r rounded up to 4
    DropArgs drop;
    float scale;
    int M, C, chunk, tiles, splits;   // chunk: columns of a split, whole blocks
};
// Item i takes workgroups [first[i], first[i + 1]).
struct StreamArgs {
    StreamItem item[kStreamItems];
    int first[kStreamItems + 1];
    PrepCodes q;          // (of the only item)
    int n, r;
};

// What lanes of a wave read from LDS that is the wave's own comes after what its other lanes wrote
// there.  No instruction: a wave's LDS accesses are done in order, and the compiler keeps to it.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// TQ: groups of 32 ranks.  VEC: rows of X and Y are whole 16-byte chunks.  DROP: thr > 0.
template <int TQ, bool VEC, bool YNAT, bool DROP, bool QUANT, int DT>
__device__ __forceinline__ void stream_body(const StreamArgs& args) {
    constexpr int kLdT = 128 + 8, kLdN = slice_ld<TQ>();            // halves of a row of the slice in LDS
    constexpr int kCh = YNAT ? 4 * TQ : 16;                         // 16-byte chunks of a row
    constexpr int kYPer = 2 * TQ;                                   // slice loads per thread
    constexpr int kSlice = YNAT ? 128 * kLdN : 32 * TQ * kLdT;
    constexpr int kLdX = 128 + 8;
    __shared__ __attribute__((aligned(16))) uint16_t ys[2][kSlice];
    __shared__ __attribute__((aligned(16))) uint16_t xs[4][32 * kLdX];
    int it = 0;
    while (it + 1 < args.n && (int)blockIdx.x >= args.first[it + 1]) ++it;
    const StreamItem a = args.item[it];
    const int id = (int)blockIdx.x - args.first[it], tile = id % a.tiles, split = id / a.tiles;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, l32 = lane & 31;
    const int tj = l32 & 15, tg = l32 >> 4;
    const int M = a.M, C = a.C, r = args.r;
    const int bm0 = tile * 128, row0 = bm0 + 32 * wave + (lane >> 4), ch8 = 8 * (lane & 15);   // a lane: rows row0 + 4 p, 8 columns
    const int c_begin = split * a.chunk, c_end = min(C, c_begin + a.chunk), n = (c_end - c_begin + 127) >> 7;
    const rsrc_t xrs = buf_rsrc(a.X + (int64_t)bm0 * C, (uint64_t)min(128, M - bm0) * C * 2);
    [[maybe_unused]] constexpr uint32_t kNone = 0x80000000u;   // past every buffer here: stores nothing
    [[maybe_unused]] const rsrc_t qrs = buf_rsrc(QUANT ? args.q.codes + (int64_t)bm0 * args.q.ld : nullptr,
                                                 QUANT ? (uint64_t)min(128, M - bm0) * args.q.ld : 0);

    struct Cols {
        bf16x8 x[8];
    };
    auto load_x = [&](Cols& q, int b) __attribute__((always_inline)) {
        const int c = c_begin + 128 * b + ch8;
        // (rows past M lie past the buffer, and so does whatever is added to kNone)
        const uint32_t at = c < c_end ? 2u * ((uint32_t)(row0 - bm0) * (uint32_t)C + (uint32_t)c) : kNone;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (VEC) q.x[p] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(xrs, at + 8u * (uint32_t)p * (uint32_t)C, 0, 0));
            else q.x[p] = load8_row<false>(a.X, C, row0 + 4 * p, M, c, c_end);
        }
    };
    bf16x8 yv[kYPer];
    auto load_y = [&](int b) __attribute__((always_inline)) {
        const int c0 = c_begin + 128 * b;
        if constexpr (YNAT) {
            const rsrc_t rs = buf_rsrc(a.Y + (int64_t)c0 * r, c0 < c_end ? (uint64_t)min(128, c_end - c0) * r * 2 : 0);
#pragma unroll
            for (int e = 0; e < kYPer; ++e) {
                const int idx = tid + 256 * e, row = idx / kCh, ch = idx % kCh;
                yv[e] = VEC ? bload8(rs, 8 * ch < r, (uint32_t)(row * r + 8 * ch))
                            : load8_row<false>(a.Y, r, c0 + row, c_end, 8 * ch, r);
            }
        } else {
            const rsrc_t rs = buf_rsrc(a.Y, (uint64_t)r * C * 2);
#pragma unroll
            for (int e = 0; e < kYPer; ++e) {
                const int idx = tid + 256 * e, row = idx / kCh, c = c0 + 8 * (idx % kCh);
                yv[e] = VEC ? bload8(rs, row < r && c < c_end, (uint32_t)(row * C + c))
                            : load8_row<false>(a.Y, C, row, r, c, c_end);
            }
        }
    };
    auto store_y = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < kYPer; ++e) {
            const int idx = tid + 256 * e, row = idx / kCh, ch = idx % kCh;
            *reinterpret_cast<bf16x8*>(&ys[buf][row * (YNAT ? kLdN : kLdT) + 8 * ch]) = yv[e];
        }
    };
    f32x16_t acc[TQ];
#pragma unroll
    for (int q = 0; q < TQ; ++q)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[q][v] = 0.0f;
    auto use = [&](const Cols& q, int b, int buf) __attribute__((always_inline)) {
        const int c0 = c_begin + 128 * b;
        uint16_t* const xw = xs[wave];
        [[maybe_unused]] const uint32_t to = c0 + ch8 < args.q.ld ? (uint32_t)(row0 - bm0) * (uint32_t)args.q.ld + (uint32_t)(c0 + ch8) : kNone;
        [[maybe_unused]] uint32_t mine = 0;   // the scale byte of row row0 + 4 (lane % 8)
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            u32x4_t v = __builtin_bit_cast(u32x4_t, q.x[p]);
            if constexpr (DROP) v = drop8(v, a.drop, (uint32_t)(c0 + ch8) >> 3, (uint32_t)(row0 + 4 * p));
            *reinterpret_cast<u32x4_t*>(&xw[((lane >> 4) + 4 * p) * kLdX + ch8]) = v;
        }
        auto read_y = [&](int i, int t) __attribute__((always_inline)) {   // columns 16 i + 8 h .. of ranks 32 t ..
            const int c = 16 * i + 8 * h;
            return YNAT ? slice_col8(ys[buf], kLdN, c, 32 * t + 16 * tg, tj)
                        : *reinterpret_cast<const bf16x8*>(&ys[buf][(32 * t + l32) * kLdT + c]);
        };
        bf16x8 y[2][TQ], xo[2];   // operands: 16 columns' are read while the 16 before are multiplied
#pragma unroll
        for (int t = 0; t < TQ; ++t) y[0][t] = read_y(0, t);
        // No memory access moves across the order point: the codes are stored behind it, beside the
        // products, and Y's first operands are read in front.  (With the codes in front, and operands
        // read as they are used, it cost up to 4 %, r = 128.)  What lanes read for block b - 1 lies
        // behind the barrier before this block.
        wave_lds_order();
        auto read_x = [&](int i) __attribute__((always_inline)) {
            return *reinterpret_cast<const bf16x8*>(&xw[l32 * kLdX + 16 * i + 8 * h]);
        };
        xo[0] = read_x(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < 7) {
                xo[(i + 1) & 1] = read_x(i + 1);
#pragma unroll
                for (int t = 0; t < TQ; ++t) y[(i + 1) & 1][t] = read_y(i + 1, t);
            }
            if constexpr (QUANT) {
                const u32x4_t v = __builtin_bit_cast(u32x4_t, q.x[i]);
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) top = max_mag2(top, v[w]);
                const uint32_t byte = fp8_scale_byte<DT>(max_row16(top));
                mine = (lane & 7) == i ? byte : mine;
                // (rows past M lie past the buffer and are dropped)
                __builtin_amdgcn_raw_buffer_store_b64(fp8_codes8<DT>(v, byte), qrs,
                                                      to + 4u * (uint32_t)i * (uint32_t)args.q.ld, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < TQ; ++t) acc[t] = mfma32<DT>(xo[i & 1], y[i & 1][t], acc[t]);
        }
        if constexpr (QUANT) {
            const int row = row0 + 4 * (lane & 7);
            const rsrc_t srs = buf_rsrc(args.q.scale + (int64_t)(c0 >> 7) * args.q.rs + bm0, (uint64_t)min(128, M - bm0));
            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)mine, srs, (lane & 15) < 8 ? (uint32_t)(row - bm0) : kNone, 0, 0);
        }
    };
    Cols q0, q1;
    load_y(0);
    load_x(q0, 0);
    load_x(q1, 1);
    store_y(0);
    for (int b = 0; b < n; b += 2) {
        load_y(b + 1);
        __syncthreads();     // the slice of block b is there
        use(q0, b, 0);
        load_x(q0, b + 2);
        store_y(1);          // (read for block b - 1, before this turn's barrier)
        if (b + 1 >= n) break;
        load_y(b + 2);
        __syncthreads();
        use(q1, b + 1, 1);
        load_x(q1, b + 3);
        store_y(0);
    }
    const int m0 = 32 * wave, rp = (r + 3) & ~3, rows = min(128, M - bm0);
    if (a.splits > 1) {
        const rsrc_t prs = buf_rsrc(a.part + ((int64_t)split * M + bm0) * rp, (uint64_t)rows * rp * 4);
#pragma unroll
        for (int q = 0; q < TQ; ++q) {
            const int j = 32 * q + l32;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int m = m0 + 8 * (v >> 2) + 4 * h + (v & 3);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[q][v]), prs, j < rp ? (uint32_t)(m * rp + j) * 4u : kNone, 0, 0);
            }
        }
        return;
    }
    const rsrc_t ors = buf_rsrc(a.out + (int64_t)bm0 * r, (uint64_t)rows * r * 2);
#pragma unroll
    for (int q = 0; q < TQ; ++q) {
        const int j = 32 * q + l32;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int m = m0 + 8 * (v >> 2) + 4 * h + (v & 3);
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pack2<DT>(a.scale * acc[q][v], 0.0f) & 0xFFFFu), ors,
                                                  j < r ? (uint32_t)(m * r + j) * 2u : kNone, 0, 0);
        }
    }
}

// out[m, 4 c ..] = RNE_16(scale sum over splits of part), 8 lanes to each four ranks: lane k adds the
// splits k, k + 8, .., then the lanes' sums are added pairwise.
template <int DT>
__device__ __forceinline__ void reduce_body(const StreamArgs& args) {
    const StreamItem a = args.item[blockIdx.y];
    const int r = args.r, rp = (r + 3) & ~3, k = threadIdx.x & 7;
    if (a.splits <= 1) return;
    const int64_t quads = (int64_t)a.M * (rp / 4);
    for (int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); i < quads; i += (int64_t)gridDim.x * 32) {
        const float* p = a.part + 4 * i;
        const int64_t step = (int64_t)a.M * rp;
        f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
        int d = k;
        for (; d + 24 < a.splits; d += 32) {   // four in flight
            f32x4_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const f32x4_t*>(p + (d + 8 * e) * step);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] += v[e][c];
        }
        for (; d < a.splits; d += 8) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + d * step);
#pragma unroll
            for (int c = 0; c < 4; ++c) s[c] += v[c];
        }
#pragma unroll
        for (int x = 1; x < 8; x *= 2)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[c] += __shfl_xor(s[c], x);
        if (k == 0) {
            const int64_t m = i / (rp / 4);
            const int j = 4 * (int)(i - m * (rp / 4));
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (j + c < r) a.out[m * r + j + c] = (uint16_t)(pack2<DT>(a.scale * s[c], 0.0f) & 0xFFFFu);
        }
    }
}
template <int DT>
__global__ __launch_bounds__(256) void prep_reduce_kernel(const StreamArgs args) { reduce_body<DT>(args); }

// The second launch, where some product is split.
inline qlora_status launch_reduce(const StreamArgs& a, int dt, hipStream_t s) {
    int64_t wgs = 0;
    for (int i = 0; i < a.n; ++i)
        if (a.item[i].splits > 1) wgs = std::max(wgs, ((int64_t)a.item[i].M * ((a.r + 3) / 4) + 31) / 32);
    if (!wgs) return QLORA_OK;
    const dim3 grid((unsigned)std::min<int64_t>(wgs, 1 << 16), (unsigned)a.n);
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        hipLaunchKernelGGL((prep_reduce_kernel<DT>), grid, dim3(256), 0, s, a);
    });
    return launch_status();
}

inline StreamItem stream_item(const uint16_t* X, const uint16_t* Y, uint16_t* out, void* ws, const DropArgs& drop,
                              float scale, int M, int C, const SplitPlan& sp) {
    return StreamItem{X, Y, out, static_cast<float*>(ws), drop, scale * drop.inv, M, C, sp.chunk,
                      (int)(((int64_t)M + 127) / 128), sp.splits};
}

}  // namespace
}  // namespace qlora
