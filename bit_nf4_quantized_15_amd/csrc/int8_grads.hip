// LoRA weight gradients with x given as its 8-bit checkpoint (MFMA, gfx950):
//
//   dA [K, r] = x_16^T u,   x_16[m,k] = RNE_16( fl32( x_scale[m] x[m,k] ) )
//   dB [r, N] = t^T dy
//
// ("bitsandbytes deep dive" 12.2 and 12.4: the rank-r side path's gradients, the base
// frozen; section 4: absmax int8 rows.)  Both are out[d, j] = sum_m X[m, d] S[m, j]: one wide
// operand X (codes, or dy) read once from HBM and one narrow one S (u, or t) from L2.
//
// An MFMA operand is 8 consecutive m of one column.  A lane loads 4 neighbouring columns of
// 8 rows (a wave: 128 columns x 16 rows, whole 128-byte runs) and builds the operands of its
// four columns in registers: codes are converted, scaled by their row and rounded pairwise;
// dy pairs rows with one byte permute.  Which column an MFMA row stands for is free, so its
// row l of product c is column 4 l + c, and no transpose through LDS is needed; S, whose
// lane holds 1, 2 or 4 neighbouring ranks, the same.  Loads run several 16-row steps ahead
// in registers; there is no barrier in the main loop.
//
// The four waves of a workgroup share 128 columns and take a quarter of its rows each; their
// sums are added through LDS in a fixed order.  Long reductions are split over workgroups
// as in the other LoRA products (split_sync.h): the last split adds the others' partial
// tiles in order, so results do not depend on timing.
//
// Bound by HBM: the seven layers of a 7B-size block, 4096 tokens, r = 64, traced: 117 us, 4.2 TB/s of
// codes and dy; one layer of 500 tokens, 4096 -> 11008, r = 16: 10.6 us, mostly one tile's latency.
#include <cstring>

#include "int8.h"
#include "lora_plan.h"
#include "split_sync.h"

namespace qlora {
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

__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
constexpr uint32_t kNone = 0x80000000u;   // past every buffer here: reads zero

constexpr int kGrThreads = 256, kGrCols = 128;
constexpr int kTable = kInt8GradChunk + 64;   // row scales in LDS

struct GradProb {
    const void* X;        // codes [M, D] with scale, or 16-bit values [M, D] without
    const float* scale;
    const uint16_t* S;    // [M, r]
    uint64_t* tags;
    float* part;
    float* out;           // codes: [D, r]; values: [r, D]
    int M, D, chunk, tiles, splits;
};
struct GradBatch {
    GradProb p[2 * kInt8GradLayers];
    int first[2 * kInt8GradLayers + 1];
    int n, r;
};

// Operand word of rows (m, m + 1) from two rows' 16-bit pairs: their low or their high halves.
__device__ __forceinline__ uint32_t rows2(uint32_t m0, uint32_t m1, int high) {
    return __builtin_amdgcn_perm(m1, m0, high ? 0x07060302u : 0x05040100u);
}

// CW: ranks per lane (1, 2, 4: r up to 32, 64, 128).  SV: r % CW == 0 (a lane's ranks are one
// load).  XV: D % 4 == 0 (dy: a lane's columns are one load).
template <int CW, bool SV, bool XV, bool I8, int DT>
__device__ __forceinline__ void grad_body(const GradProb& pr, int r, int tile, int split, float* __restrict__ lds) {
    constexpr int P = I8 ? 4 : (CW == 4 ? 2 : 3);      // 16-row steps in flight
    constexpr int kXW = I8 ? 1 : 2, kSW = CW == 4 ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int d0 = tile * kGrCols, D = pr.D;
    const int b0 = split * pr.chunk, b1 = min(pr.M, b0 + pr.chunk);
    const int quarter = (((b1 - b0) + 63) >> 6) * 16;  // rows per wave, whole 16-row steps
    const int m0 = b0 + wave * quarter, rows = max(0, min(b1 - m0, quarter)), steps = (rows + 15) >> 4;

    // row scales of the workgroup's chunk in LDS, zero past its end (the steps in flight past
    // it read them too)
    float* const st = lds;
    if (I8) {
        for (int i = tid; i < 4 * quarter + 16 * P; i += kGrThreads) st[i] = b0 + i < b1 ? pr.scale[b0 + i] : 0.0f;
        __syncthreads();
    }

    // Row 16 k + e of the wave's rows starts at the scalar base of a buffer of its own, whose
    // range is what is left from there: one lane offset each for X and S (rows e and e + 8),
    // rows past the end read zero, and the addresses cost scalar instructions only.
    const uint32_t ld = (uint32_t)D * (I8 ? 1u : 2u), lds_ = (uint32_t)r * 2u;   // bytes of a row of X, of S
    const uint8_t* xb = static_cast<const uint8_t*>(pr.X) + (int64_t)(rows ? m0 : b0) * ld + (int64_t)d0 * (I8 ? 1 : 2);
    const uint8_t* sb = reinterpret_cast<const uint8_t*>(pr.S) + (int64_t)(rows ? m0 : b0) * lds_;
    int32_t xleft = rows ? (int32_t)((uint32_t)rows * ld - (uint32_t)d0 * (I8 ? 1u : 2u)) : 0;
    int32_t sleft = (int32_t)((uint32_t)rows * lds_);
    const uint32_t xoff = 8u * h * ld + (I8 ? 4u : 8u) * l32;
    const bool jok = CW * l32 < r;
    const uint32_t soff = (jok || !SV) ? 8u * h * lds_ + (uint32_t)(CW * l32) * 2u : kNone;
    struct Step {
        uint32_t x[8][kXW], s[8][kSW];
    };
    // Requests the next 16 rows.
    auto load = [&](Step& q) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const rsrc_t xrs = buf_rsrc(xb, (uint32_t)max(xleft, 0)), srs = buf_rsrc(sb, (uint32_t)max(sleft, 0));
            if (I8) {
                q.x[e][0] = __builtin_amdgcn_raw_buffer_load_b32(xrs, xoff, 0, 0);
            } else if (XV) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(xrs, xoff, 0, 0);
                q.x[e][0] = v[0];
                q.x[e][kXW - 1] = v[1];
            } else {
#pragma unroll
                for (int i = 0; i < kXW; ++i) {
                    const uint32_t lo = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(xrs, xoff + 4 * i, 0, 0);
                    const uint32_t hi = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(xrs, xoff + 4 * i + 2, 0, 0);
                    q.x[e][i] = lo | (hi << 16);
                }
            }
            if (SV && CW == 1) {
                q.s[e][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(srs, soff, 0, 0);
            } else if (SV && CW == 2) {
                q.s[e][0] = __builtin_amdgcn_raw_buffer_load_b32(srs, soff, 0, 0);
            } else if (SV) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(srs, soff, 0, 0);
                q.s[e][0] = v[0];
                q.s[e][kSW - 1] = v[1];
            } else {
#pragma unroll
                for (int i = 0; i < kSW; ++i) {
                    const int j = CW * l32 + 2 * i;
                    const uint32_t lo =
                        (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(srs, j < r ? soff + 4 * i : kNone, 0, 0);
                    const uint32_t hi =
                        (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(srs, j + 1 < r ? soff + 4 * i + 2 : kNone, 0, 0);
                    q.s[e][i] = lo | (hi << 16);
                }
            }
            // the next row, or past the 8 rows of the other lane half
            const uint32_t skip = e == 7 ? 9u : 1u;
            xb += (int64_t)skip * ld;
            sb += (int64_t)skip * lds_;
            xleft -= (int32_t)(skip * ld);
            sleft -= (int32_t)(skip * lds_);
        }
    };

    f32x16_t acc[4][CW];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < CW; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[c][j][v] = 0.0f;
    auto use = [&](int st_, const Step& q) __attribute__((always_inline)) {
        u32x4_t xo[4], so[CW];
        f32x4_t sc[2];
        if (I8) {
            sc[0] = *reinterpret_cast<const f32x4_t*>(st + wave * quarter + 16 * st_ + 8 * h);
            sc[1] = *reinterpret_cast<const f32x4_t*>(st + wave * quarter + 16 * st_ + 8 * h + 4);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {                  // rows 2p, 2p + 1
#pragma unroll
            for (int j = 0; j < CW; ++j) so[j][p] = rows2(q.s[2 * p][j >> 1], q.s[2 * p + 1][j >> 1], j & 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (I8) {
                    const float a = (float)(int32_t)(int8_t)(q.x[2 * p][0] >> (8 * c)) * sc[p >> 1][2 * (p & 1)];
                    const float b = (float)(int32_t)(int8_t)(q.x[2 * p + 1][0] >> (8 * c)) * sc[p >> 1][2 * (p & 1) + 1];
                    xo[c][p] = pack2<DT>(a, b);
                } else {
                    xo[c][p] = rows2(q.x[2 * p][(c >> 1) & (kXW - 1)], q.x[2 * p + 1][(c >> 1) & (kXW - 1)], c & 1);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)   // codes: rows of the product are columns d; values: ranks j
                acc[c][j] = I8 ? mfma16<DT>(xo[c], so[j], acc[c][j]) : mfma16<DT>(so[j], xo[c], acc[c][j]);
    };

    Step ring[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        load(ring[p]);
        __builtin_amdgcn_sched_barrier(0);             // in order, so that a wait for one leaves the next in flight
    }
    for (int k = 0; k < steps; k += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            use(k + p, ring[p]);                       // steps past the end multiply zeros
            load(ring[p]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // ---- add the waves: wave w keeps product rows 8 w + 4 h + e of every (c, j)
    f32x4_t res[4][CW];
    float* const ex = lds + (I8 ? kTable : 0);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int j = 0; j < CW; ++j)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                *reinterpret_cast<f32x4_t*>(ex + (((wave * CW + j) * 4 + v4) * 64 + lane) * 4) =
                    f32x4_t{acc[c][j][4 * v4], acc[c][j][4 * v4 + 1], acc[c][j][4 * v4 + 2], acc[c][j][4 * v4 + 3]};
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CW; ++j) {
            f32x4_t t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t*>(ex + (((w * CW + j) * 4 + wave) * 64 + lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] += v[e];
            }
            res[c][j] = t;
        }
        __syncthreads();
    }

    // ---- add the splits
    const uint64_t tag = launch_tag();
    uint64_t* const flags = pr.tags + (size_t)tile * pr.splits;
    constexpr uint32_t kTile = 4u * 4u * CW * 64u * 16u;   // bytes of a partial tile
    auto poff = [&](int c, int j) { return (uint32_t)((((wave * 4 + c) * CW + j) * 64 + lane) * 16); };
    if (split < pr.splits - 1) {
        const rsrc_t rs = buf_rsrc(reinterpret_cast<uint8_t*>(pr.part) + ((size_t)split * pr.tiles + tile) * kTile, kTile);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, res[c][j]), rs, poff(c, j), 0, kCoherent);
        publish_tag(flags + split, tag);
        return;
    }
    if (pr.splits > 1) {
        const bool fail = wait_tags(flags, pr.splits - 1, tag);
        f32x4_t tot[4][CW];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j) tot[c][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        // several splits' tiles in flight at a time: each load comes from the device-coherent level
        constexpr int kRound = CW == 4 ? 2 : 4;
        const int last = pr.splits - 1;
        for (int s = 0; s < last; s += kRound) {
            u32x4_t g[kRound][4][CW];
#pragma unroll
            for (int k = 0; k < kRound; ++k) {
                const int from = min(s + k, last - 1);
                const rsrc_t rs = buf_rsrc(reinterpret_cast<uint8_t*>(pr.part) + ((size_t)from * pr.tiles + tile) * kTile,
                                           s + k < last ? kTile : 0u);   // past the last: zeros
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        g[k][c][j] = __builtin_amdgcn_raw_buffer_load_b128(rs, poff(c, j), 0, kCoherent);
            }
#pragma unroll
            for (int k = 0; k < kRound; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < CW; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) tot[c][j][e] += __uint_as_float(g[k][c][j][e]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) res[c][j][e] = fail ? __builtin_nanf("") : tot[c][j][e] + res[c][j][e];
    }

#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = 8 * wave + 4 * h + e;          // of the 32 product rows
        if (I8) {                                      // out [D, r]: columns 4 row + c, ranks CW l32 + 0 ..
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int d = d0 + 4 * row + c;
                if (d >= D) continue;
                float* o = pr.out + (int64_t)d * r + CW * l32;
                if (SV && CW == 2) {
                    if (jok) *reinterpret_cast<f32x2_t*>(o) = f32x2_t{res[c][0][e], res[c][CW - 1][e]};
                } else {
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        if (CW * l32 + j < r) o[j] = res[c][j][e];
                }
            }
        } else {                                       // out [r, D]: ranks CW row + j, columns 4 l32 + 0..3
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                const int jj = CW * row + j, d = d0 + 4 * l32;
                if (jj >= r) continue;
                float* o = pr.out + (int64_t)jj * D + d;
                if (XV) {
                    if (d < D) *reinterpret_cast<f32x4_t*>(o) = f32x4_t{res[0][j][e], res[1][j][e], res[2][j][e], res[3][j][e]};
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (d + c < D) o[c] = res[c][j][e];
                }
            }
        }
    }
}

// Problem i takes workgroups [first[i], first[i + 1]), numbered split by split, so that a
// waiting workgroup only waits for lower ids.
template <int CW, bool SV, bool XV, int DT>
__global__ __launch_bounds__(kGrThreads, CW <= 2 ? 2 : 1) void int8_grads_kernel(const GradBatch bt) {
    __shared__ __attribute__((aligned(16))) float lds[kTable + 4 * CW * 16 * 64];
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.n && b >= bt.first[i + 1]) ++i;
    const GradProb& p = bt.p[i];
    const int c = b - bt.first[i];
    if (p.scale) grad_body<CW, SV, XV, true, DT>(p, bt.r, c % p.tiles, c / p.tiles, lds);
    else grad_body<CW, SV, XV, false, DT>(p, bt.r, c % p.tiles, c / p.tiles, lds);
}

inline int ranks_per_lane(int r) { return r <= 32 ? 1 : r <= 64 ? 2 : 4; }

}  // namespace

Int8GradPlan plan_int8_grad(int64_t M, int64_t D, int r, int64_t all_tiles) {
    Int8GradPlan p;
    p.tiles = (D + kGrCols - 1) / kGrCols;
    // a wave's rows (a quarter of a chunk) are addressed with 31 bits
    const int64_t most = std::min<int64_t>(kInt8GradChunk, (int64_t(1) << 30) / (2 * D) / 16 * 64);
    // One workgroup per CU is enough to stream, and a split costs a partial tile written and
    // read again (32 KB at r = 64 against 128 bytes a row of codes): split only to fill the
    // 256 CUs, and not below 256 rows.  M = 4096, K = N = 4096, r = 64: 4 splits 20.9 us, 2
    // splits 28.6, 8 splits 25.1; M = 500, N = 11008: 1 split 10.4 us, 2 splits 11.5, 3 13.0.
    const int64_t s = std::max<int64_t>((M + most - 1) / most, std::min<int64_t>(256 / all_tiles, M / 256));
    p.chunk = ((M + std::max<int64_t>(s, 1) - 1) / std::max<int64_t>(s, 1) + 63) / 64 * 64;
    p.splits = (M + p.chunk - 1) / p.chunk;
    p.ws_tags = align256((size_t)(p.tiles * p.splits) * 8);
    p.ws = p.ws_tags + align256((size_t)((p.splits - 1) * p.tiles) * 4 * 4 * ranks_per_lane(r) * 64 * 16);
    return p;
}

qlora_status launch_int8_grads(const Int8GradDesc* d, int count, int r, int dt, hipStream_t s) {
    GradBatch b;
    std::memset(&b, 0, sizeof b);
    b.r = r;
    bool xv = true;
    int64_t total = 0;
    // the 16-bit operands first: their workgroups stream twice the bytes
    for (int pass = 0; pass < 2; ++pass)
        for (int i = 0; i < count; ++i) {
            if ((d[i].scale != nullptr) != (pass == 1)) continue;
            GradProb& p = b.p[b.n];
            p.X = d[i].X;
            p.scale = d[i].scale;
            p.S = d[i].S;
            p.out = d[i].out;
            p.tags = static_cast<uint64_t*>(d[i].ws);
            p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(d[i].ws) + d[i].plan.ws_tags);
            p.M = d[i].M;
            p.D = d[i].D;
            p.chunk = (int)d[i].plan.chunk;
            p.tiles = (int)d[i].plan.tiles;
            p.splits = (int)d[i].plan.splits;
            xv = xv && d[i].D % 4 == 0;
            b.first[b.n++] = (int)total;
            total += d[i].plan.tiles * d[i].plan.splits;
            if (total * kGrThreads >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
        }
    b.first[b.n] = (int)total;
    if (total == 0) return QLORA_OK;
    const int cw = ranks_per_lane(r);
    const bool sv = r % cw == 0;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_GR(CW, SV, XV) \
    hipLaunchKernelGGL((int8_grads_kernel<CW, SV, XV, DT>), dim3((unsigned)total), dim3(kGrThreads), 0, s, b)
#define QL_GR1(CW)                                                                                \
    if (sv) { if (xv) QL_GR(CW, true, true); else QL_GR(CW, true, false); }                       \
    else { if (xv) QL_GR(CW, false, true); else QL_GR(CW, false, false); }
        if (cw == 1) {   // one rank per lane: always whole
            if (xv) QL_GR(1, true, true); else QL_GR(1, true, false);
        } else if (cw == 2) {
            QL_GR1(2)
        } else {
            QL_GR1(4)
        }
#undef QL_GR1
#undef QL_GR
    });
    return launch_status();
}

}  // namespace qlora
