// LoRA weight gradients of layers with dropout (MFMA, gfx950), several layers in one launch:
//
//   dA [K, r] = drop(x)^T u,   dB [r, N] = t^T dy
//
// ("bitsandbytes deep dive", 12.2 and 12.4: the rank-r side path's gradients, the base frozen;
// dropout.h: the mask.)  Both are out[d, j] = sum_m X[m, d] S[m, j]: one wide operand X (x, or dy)
// read once from HBM and one narrow one S (u, or t) from the caches.
//
// An MFMA operand is 8 consecutive m of one column.  A lane loads 4 neighbouring columns of 8
// rows (a wave: 128 columns x 16 rows) and pairs rows with one byte permute; which column an MFMA
// row stands for is free, so no transpose through LDS is needed.  S the same: a lane holds 1, 2
// or 4 neighbouring ranks.  Loads run several 16-row steps ahead in registers; there is no barrier
// in the main loop.  The generator's unit is 8 columns of a row, which two neighbouring lanes
// hold: each makes the masks of half of the 8 rows and hands the other its four columns (DPP).
//
// The four waves of a workgroup share 128 columns and take a quarter of its rows each; their sums
// are added through LDS in a fixed order, and the splits of a long reduction by the last one's
// workgroup (split_sync.h), so results do not depend on timing.
//
// Seven layers of a 7B-size block, 4096 tokens, r = 64, traced: 139 us, 4.1 TB/s of x and dy; the generator
// takes 36 us of every SIMD's time beside it.  (Tiles of 64 rows through LDS, as the gradients
// without dropout go, took 189 us.)  One layer of 500 tokens, 4096 -> 11008, r = 16: 11.4 us (15.4), a
// tile's latency.
#include <cstring>

#include "dropout.h"
#include "grads_plan.h"
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
constexpr int kThreads = 256;

struct GradProb {
    const uint16_t* X;    // [M, D]
    const uint16_t* S;    // [M, r]
    uint64_t* tags;       // [tile][split]
    float* part;
    float* out;           // dA [D, r], or dB [r, D]
    DropArgs drop;        // of dA's X
    int M, D, chunk, tiles, splits, dA;
};
constexpr int kGradProbs = 16;
struct GradBatch {
    GradProb p[kGradProbs];
    int first[kGradProbs + 1];
    int n, r;
};

// Operand word of rows (m, m + 1) from two rows' 16-bit pairs: their low or their high halves.
__device__ __forceinline__ uint32_t rows2(uint32_t m0, uint32_t m1, int high) {
    return __builtin_amdgcn_perm(m1, m0, high ? 0x07060302u : 0x05040100u);
}

// CW: ranks per lane (1, 2, 4: r up to 32, 64, 128).  SV: r % CW == 0 (a lane's ranks are one
// load).  XV: D % 4 == 0 (a lane's columns are one load).
template <int CW, bool SV, bool XV, bool DA, int DT>
__device__ __forceinline__ void grad_body(const GradProb& pr, int r, int tile, int split, float* __restrict__ lds) {
    constexpr int P = CW == 4 || (CW == 2 && !(SV && XV)) ? 2 : 3;   // 16-row steps in flight (in registers)
    constexpr int kSW = CW == 4 ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int d0 = tile * kGradCols, D = pr.D;
    const int64_t b0 = (int64_t)split * pr.chunk, b1 = min((int64_t)pr.M, b0 + pr.chunk);
    const int quarter = (int)((b1 - b0 + 63) >> 6) * 16;   // rows per wave, whole 16-row steps
    const int64_t m0 = b0 + wave * quarter;
    const int rows = (int)max((int64_t)0, min(b1 - m0, (int64_t)quarter)), steps = (rows + 15) >> 4;

    // Row 16 k + e of the wave's rows starts at the scalar base of a buffer of its own, whose
    // range is what is left from there: one lane offset each for X and S (rows e and e + 8),
    // rows past the end read zero, and the addresses cost scalar instructions only.
    const uint32_t ld = 2u * (uint32_t)D, lds_ = 2u * (uint32_t)r;
    const uint8_t* xb = reinterpret_cast<const uint8_t*>(pr.X) + (rows ? m0 : b0) * ld + 2 * (int64_t)d0;
    const uint8_t* sb = reinterpret_cast<const uint8_t*>(pr.S) + (rows ? m0 : b0) * lds_;
    int32_t xleft = rows ? (int32_t)((uint32_t)rows * ld - 2u * (uint32_t)d0) : 0;
    int32_t sleft = (int32_t)((uint32_t)rows * lds_);
    const uint32_t xoff = 8u * h * ld + 8u * l32;
    const bool jok = CW * l32 < r;
    const uint32_t soff = (jok || !SV) ? 8u * h * lds_ + (uint32_t)(CW * l32) * 2u : kNone;
    struct Step {
        uint32_t x[8][2], s[8][kSW];
    };
    auto load = [&](Step& q) __attribute__((always_inline)) {   // the next 16 rows
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const rsrc_t xrs = buf_rsrc(xb, (uint32_t)max(xleft, 0)), srs = buf_rsrc(sb, (uint32_t)max(sleft, 0));
            if (XV) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(xrs, xoff, 0, 0);
                q.x[e][0] = v[0];
                q.x[e][1] = v[1];
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
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
    const bool odd = (lane & 1) != 0;                  // the upper four columns of a unit of 8
    auto use = [&](int st, Step& q) __attribute__((always_inline)) {
        if constexpr (DA) {
            const uint32_t group = (uint32_t)(d0 + 4 * l32) >> 3, m = (uint32_t)(m0 + 16 * st + 8 * h) + (odd ? 4u : 0u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {              // this lane: row e of the 8, or row e + 4
                const u32x4_t w = drop_words(pr.drop, group, m + (uint32_t)e);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t lo = dropped_halves(w[i], pr.drop.thr), hi = dropped_halves(w[2 + i], pr.drop.thr);
                    const uint32_t own = odd ? hi : lo;
                    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? lo : hi), 0xB1, 0xF, 0xF, true);
                    q.x[e][i] &= ~(odd ? got : own);
                    q.x[4 + e][i] &= ~(odd ? own : got);
                }
            }
        }
        u32x4_t xo[4], so[CW];
#pragma unroll
        for (int p = 0; p < 4; ++p) {                  // rows 2p, 2p + 1
#pragma unroll
            for (int j = 0; j < CW; ++j) so[j][p] = rows2(q.s[2 * p][j >> 1], q.s[2 * p + 1][j >> 1], j & 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) xo[c][p] = rows2(q.x[2 * p][c >> 1], q.x[2 * p + 1][c >> 1], c & 1);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)   // dA: rows of the product are columns d; dB: ranks j
                acc[c][j] = DA ? mfma16<DT>(xo[c], so[j], acc[c][j]) : mfma16<DT>(so[j], xo[c], acc[c][j]);
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
    float* const ex = lds;
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

    if (DA)                                            // what is kept counts 1 / (1 - p) times
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) res[c][j][e] *= pr.drop.inv;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = 8 * wave + 4 * h + e;          // of the 32 product rows
        if (DA) {                                      // out [D, r]: columns 4 row + c, ranks CW l32 + 0 ..
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
__global__ __launch_bounds__(kThreads, CW <= 2 ? 2 : 1) void grads_dropout_kernel(const GradBatch bt) {
    __shared__ __attribute__((aligned(16))) float lds[4 * CW * 16 * 64];
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.n && b >= bt.first[i + 1]) ++i;
    const GradProb& p = bt.p[i];
    const int c = b - bt.first[i];
    if (p.dA) grad_body<CW, SV, XV, true, DT>(p, bt.r, c % p.tiles, c / p.tiles, lds);
    else grad_body<CW, SV, XV, false, DT>(p, bt.r, c % p.tiles, c / p.tiles, lds);
}

// n <= kGradProbs contractions
qlora_status grads_dropout(const GradDropDesc* d, int n, int r, int dt, hipStream_t s) {
    GradBatch b;
    std::memset(&b, 0, sizeof b);
    b.r = r;
    b.n = n;
    int64_t all = 0, total = 0;
    for (int i = 0; i < n; ++i) all += grad_tiles(d[i].D);
    bool xv = true;
    for (int i = 0; i < n; ++i) {
        const SplitPlan sp = plan_grad_dropout(d[i].M, d[i].D, r, all);
        GradProb& p = b.p[i];
        p.X = d[i].X;
        p.S = d[i].S;
        p.out = d[i].out;
        p.drop = d[i].drop;
        p.dA = d[i].dA;
        p.M = d[i].M;
        p.D = d[i].D;
        p.tiles = (int)grad_tiles(d[i].D);
        p.chunk = sp.chunk;
        p.splits = sp.splits;
        p.tags = static_cast<uint64_t*>(d[i].ws);
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(d[i].ws) + split_tags_bytes(p.tiles, sp));
        xv = xv && d[i].D % 4 == 0;
        b.first[i] = (int)total;
        total += (int64_t)p.tiles * p.splits;
        if (total * kThreads >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    }
    b.first[n] = (int)total;
    const int cw = ranks_per_lane(r);
    const bool sv = r % cw == 0;
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_GR(CW, SV, XV) \
    hipLaunchKernelGGL((grads_dropout_kernel<CW, SV, XV, DT>), dim3((unsigned)total), dim3(kThreads), 0, s, b)
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

}  // namespace

qlora_status launch_grads_dropout(const GradDropDesc* d, int count, int r, int dt, hipStream_t s) {
    for (int i = 0; i < count; i += kGradProbs) {
        const qlora_status st = grads_dropout(d + i, std::min(kGradProbs, count - i), r, dt, s);
        if (st != QLORA_OK) return st;
    }
    return QLORA_OK;
}

}  // namespace qlora
