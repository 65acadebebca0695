// LoRA side-path kernels (MFMA v_mfma_f32_32x32x16_bf16, gfx950).
//
// The rank-r products of the layer ("bitsandbytes deep dive" 12.2:
// Y = XW + s X A B, A [Din, r], B [r, Dout], s = lora_alpha / r; the chain
// rule through the same graph for the backward, base frozen):
//   t  = s x A        [M, r]   (forward, kept for the backward)
//   u  = s dy B^T     [M, r]
//   dA = x^T u        [K, r]
//   dB = t^T dy       [r, N]
// The small operands (A, B, t, u) are read in their own layouts: a slice of
// each is staged in LDS and transposed, where needed, by the LDS reads.
// All four stream one large operand (x or dy) once and are HBM bound.  The
// reductions are split over the long dimension for parallelism; partial sums
// go to a workspace and are added in a fixed order (deterministic results).
#include "lora_body.h"

namespace qlora {
namespace {

template <int TQ, bool VEC, bool YNAT, int NST, int DT>
__global__ __launch_bounds__(256) void nt_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ Y,
                                                 uint64_t* __restrict__ tags, float* __restrict__ part,
                                                 uint16_t* __restrict__ out, float scale, int M, int C, int r,
                                                 int chunk) {
    nt_body<TQ, VEC, YNAT, NST, DT>(X, Y, tags, part, out, scale, M, C, r, chunk, (int)blockIdx.x, (int)blockIdx.y,
                                    (int)gridDim.x, (int)gridDim.y);
}

template <int TQ, bool VEC, bool YNAT, int NST, int DT>
__global__ __launch_bounds__(256) void ntb_kernel(const NtBatch bt) {
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.n && b >= bt.first[i + 1]) ++i;
    const NtProb& p = bt.p[i];
    const int c = b - bt.first[i];
    nt_body<TQ, VEC, YNAT, NST, DT>(p.X, p.Y, p.tags, p.part, p.out, p.scale, p.M, p.C, bt.r, p.chunk, c % p.tiles,
                                    c / p.tiles, p.tiles, p.splits);
}

// two workgroups per CU where r <= 64 on the buffer-load path (80 KB of LDS, at most 256 VGPRs)
template <int TQ, bool VEC, int NST, int DT>
__global__ __launch_bounds__(256, TQ <= 2 && VEC ? 2 : 1) void tn_kernel(const TnProb pr) {
    tn_body<TQ, VEC, NST, DT>(pr, blockIdx.x, blockIdx.y);
}

// Two independent contractions in one grid (dA and dB of a layer): workgroups
// [0, tiles0 x splits0) run the first and the rest the second, each numbered split
// by split, so that the last split of every tile is dispatched after the tile's
// other splits.  The second contraction's workgroups take the CUs that the first
// one's finished splits leave while its last splits add up their tiles.
template <int TQ, bool VEC, int NST, int DT>
__global__ __launch_bounds__(256, TQ <= 2 && VEC ? 2 : 1) void tn2_kernel(const TnProb p0, const TnProb p1) {
    const int n0 = p0.tiles * p0.splits, b = blockIdx.x;
    if (b < n0) {
        tn_body<TQ, VEC, NST, DT>(p0, b % p0.tiles, b / p0.tiles);
    } else {
        const int c = b - n0;
        tn_body<TQ, VEC, NST, DT>(p1, c % p1.tiles, c / p1.tiles);
    }
}

template <int TQ, bool VEC, int NST, int DT>
__global__ __launch_bounds__(256, TQ <= 2 && VEC ? 2 : 1) void tnb_kernel(const TnBatch bt) {
    const int b = blockIdx.x;
    int i = 0;
    while (i + 1 < bt.n && b >= bt.first[i + 1]) ++i;
    const int c = b - bt.first[i];
    tn_body<TQ, VEC, NST, DT>(bt.p[i], c % bt.p[i].tiles, c / bt.p[i].tiles);
}

// QA-LoRA pooled branch ("LoRA, QLoRA, QA-LoRA explained", sections 3-5):
// pool(x) A = x A~ with A~[k, j] = A[k / g, j] / g, exact in bf16 for g a power
// of two (a shift of the exponent) unless it underflows, so the plain kernels run on A~; the
// gradient of A sums each group of g rows of the gradient of A~:
// dA[i, j] = (1/g) sum_{q < g} dA~[g i + q, j], q ascending, in fp32.
template <int DT>
__global__ void expand_pooled_kernel(const uint16_t* __restrict__ A, int64_t count, int r, int g_log2,
                                     uint16_t* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= count) return;
    const int64_t k = i / r, j = i - k * r;
    const float v = h16_to_f32<DT>(A[(k >> g_log2) * r + j]) * __uint_as_float((uint32_t)(127 - g_log2) << 23);
    out[i] = (uint16_t)(pack2<DT>(v, 0.0f) & 0xFFFFu);
}

__global__ void pool_rows_kernel(const float* __restrict__ in, int64_t count, int r, int g, int g_log2,
                                 float* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;  // output element [K/g, r]
    if (i >= count) return;
    const int64_t p = i / r, j = i - p * r;
    float acc = 0.0f;
    for (int q = 0; q < g; ++q) acc += in[(p * g + q) * r + j];
    out[i] = acc * __uint_as_float((uint32_t)(127 - g_log2) << 23);
}

__global__ void fill_f32_kernel(float* __restrict__ out, int64_t count, float v) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < count) out[i] = v;
}

// Grid and arguments of a launch over the n <= kNtBatch products d.  vec: the conditions of
// launch_nt's vector path, for every product of the launch.
qlora_status nt_batch(const NtDesc* d, int n, bool y_natural, int r, NtBatch& b, bool& vec, int& chunk,
                      unsigned& total) {
    b.n = n;
    b.r = r;
    vec = !y_natural || r % 8 == 0;
    int64_t sum = 0;
    for (int i = 0; i < n; ++i) {
        const NtDesc& e = d[i];
        const SplitPlan sp = plan_nt(e.M, e.C, r);
        NtProb& p = b.p[i];
        p.X = e.X;
        p.Y = e.Y;
        p.tiles = (e.M + 127) / 128;
        p.splits = sp.splits;
        p.chunk = sp.chunk;
        p.tags = static_cast<uint64_t*>(e.ws);
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(e.ws) + split_tags_bytes(p.tiles, sp));
        p.out = e.out;
        p.scale = e.scale;
        p.M = e.M;
        p.C = e.C;
        vec = vec && (e.C % 8 == 0) && ((reinterpret_cast<uintptr_t>(e.X) & 15u) == 0) &&
              ((reinterpret_cast<uintptr_t>(e.Y) & 15u) == 0) && (int64_t)e.C * 128 * 2 < (int64_t(1) << 30);
        chunk = std::max(chunk, sp.chunk);
        b.first[i] = (int)sum;
        sum += (int64_t)p.tiles * p.splits;
        if (sum >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    }
    b.first[n] = (int)sum;
    total = (unsigned)sum;
    return QLORA_OK;
}

// The same over the n <= kTnBatch contractions d.
qlora_status tn_batch(const TnDesc* d, int n, int r, TnBatch& b, bool& vec, int& chunk, unsigned& total) {
    b.n = n;
    vec = true;
    int64_t sum = 0;
    for (int i = 0; i < n; ++i) {
        const TnDesc& e = d[i];
        bool v = false;
        b.p[i] = tn_prob(e.X, e.S, e.ws, e.out, e.M, e.D, r, e.ld_d, e.ld_j, v);
        vec = vec && v;
        chunk = std::max(chunk, b.p[i].chunk);
        b.first[i] = (int)sum;
        sum += (int64_t)b.p[i].tiles * b.p[i].splits;
        if (sum >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    }
    b.first[n] = (int)sum;
    total = (unsigned)sum;
    return QLORA_OK;
}

inline unsigned blocks_for(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

qlora_status launch_nt(const uint16_t* X, const uint16_t* Y, bool y_natural, void* ws, uint16_t* out, float scale,
                       int M, int C, int r, int dt, hipStream_t s) {
    const SplitPlan sp = plan_nt(M, C, r);
    const int tiles = (M + 127) / 128;
    const dim3 grid((unsigned)tiles, (unsigned)sp.splits);
    uint64_t* tags = static_cast<uint64_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + split_tags_bytes(tiles, sp));
    // vector path: 16-byte aligned rows, and one workgroup's rows (128 of X, r of
    // Yt) under 1 GiB of buffer offsets
    const bool vec = (C % 8 == 0) && (!y_natural || r % 8 == 0) && ((reinterpret_cast<uintptr_t>(X) & 15u) == 0) &&
                     ((reinterpret_cast<uintptr_t>(Y) & 15u) == 0) && (int64_t)C * 128 * 2 < (int64_t(1) << 30);
    const int tq = (r + 31) / 32, nst = steps_template(sp.chunk);
#define QL_NT(TQ, V, NAT, NST) \
    hipLaunchKernelGGL((nt_kernel<TQ, V, NAT, NST, DT>), grid, dim3(256), 0, s, X, Y, tags, part, out, scale, M, C, r, \
                       sp.chunk);
#define QL_NT1(TQ, V, NAT)                                  \
    if (nst == 2) { QL_NT(TQ, V, NAT, 2) }                  \
    else if (nst == 4) { QL_NT(TQ, V, NAT, 4) }             \
    else { QL_NT(TQ, V, NAT, (TQ == 4 ? 4 : 8)) }
#define QL_NT2(TQ)                                                               \
    if (y_natural) {                                                             \
        if (vec) { QL_NT1(TQ, true, true) } else { QL_NT1(TQ, false, true) }    \
    } else {                                                                     \
        if (vec) { QL_NT1(TQ, true, false) } else { QL_NT1(TQ, false, false) }  \
    }
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        switch (tq) {
            case 1: QL_NT2(1) break;
            case 2: QL_NT2(2) break;
            case 3: QL_NT2(3) break;
            default: QL_NT2(4) break;
        }
    });
#undef QL_NT2
#undef QL_NT1
#undef QL_NT
    return launch_status();
}

namespace {

struct TnLaunch1 {
    const TnProb& p;
    dim3 grid;
    hipStream_t s;
    template <int TQ, bool V, int NST, int DT>
    void operator()() const {
        hipLaunchKernelGGL((tn_kernel<TQ, V, NST, DT>), grid, dim3(256), 0, s, p);
    }
};

struct TnLaunch2 {
    const TnProb& p0;
    const TnProb& p1;
    unsigned n;
    hipStream_t s;
    template <int TQ, bool V, int NST, int DT>
    void operator()() const {
        hipLaunchKernelGGL((tn2_kernel<TQ, V, NST, DT>), dim3(n), dim3(256), 0, s, p0, p1);
    }
};

}  // namespace

qlora_status launch_tn(const uint16_t* X, const uint16_t* S, void* ws, float* out, int M, int D, int r, int64_t ld_d,
                       int64_t ld_j, int dt, hipStream_t s) {
    bool vec = false;
    const TnProb p = tn_prob(X, S, ws, out, M, D, r, ld_d, ld_j, vec);
    const dim3 grid((unsigned)p.tiles, (unsigned)p.splits);
        const TnLaunch1 go{p, grid, s};
    tn_dispatch(r, vec, p.chunk, dt, go);
    return launch_status();
}

qlora_status launch_tn2(const uint16_t* X0, const uint16_t* S0, void* ws0, float* out0, int D0, int64_t ld_d0,
                        int64_t ld_j0, const uint16_t* X1, const uint16_t* S1, void* ws1, float* out1, int D1,
                        int64_t ld_d1, int64_t ld_j1, int M, int r, int dt, hipStream_t s) {
    bool vec0 = false, vec1 = false;
    const TnProb p0 = tn_prob(X0, S0, ws0, out0, M, D0, r, ld_d0, ld_j0, vec0);
    const TnProb p1 = tn_prob(X1, S1, ws1, out1, M, D1, r, ld_d1, ld_j1, vec1);
    const int64_t n = (int64_t)p0.tiles * p0.splits + (int64_t)p1.tiles * p1.splits;
    if (n >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
        const TnLaunch2 go{p0, p1, (unsigned)n, s};
    tn_dispatch(r, vec0 && vec1, std::max(p0.chunk, p1.chunk), dt, go);
    return launch_status();
}

qlora_status launch_nt_batch(const NtDesc* d, int count, bool y_natural, int r, int dt, hipStream_t s) {
    const int tq = (r + 31) / 32;
    for (int i0 = 0; i0 < count; i0 += kNtBatch) {
        NtBatch b{};
        bool vec = false;
        int chunk = 64;
        unsigned total = 0;
        const qlora_status bs = nt_batch(d + i0, std::min(kNtBatch, count - i0), y_natural, r, b, vec, chunk, total);
        if (bs != QLORA_OK) return bs;
        const int nst = steps_template(chunk);
#define QL_NTB(TQ, V, NAT, NST) \
    hipLaunchKernelGGL((ntb_kernel<TQ, V, NAT, NST, DT>), dim3(total), dim3(256), 0, s, b);
#define QL_NTB1(TQ, V, NAT)                                  \
    if (nst == 2) { QL_NTB(TQ, V, NAT, 2) }                  \
    else if (nst == 4) { QL_NTB(TQ, V, NAT, 4) }             \
    else { QL_NTB(TQ, V, NAT, (TQ == 4 ? 4 : 8)) }
#define QL_NTB2(TQ)                                                                \
    if (y_natural) {                                                               \
        if (vec) { QL_NTB1(TQ, true, true) } else { QL_NTB1(TQ, false, true) }    \
    } else {                                                                       \
        if (vec) { QL_NTB1(TQ, true, false) } else { QL_NTB1(TQ, false, false) }  \
    }
        with_dt(dt, [&](auto dtc) {
            constexpr int DT = decltype(dtc)::value;
            switch (tq) {
                case 1: QL_NTB2(1) break;
                case 2: QL_NTB2(2) break;
                case 3: QL_NTB2(3) break;
                default: QL_NTB2(4) break;
            }
        });
#undef QL_NTB2
#undef QL_NTB1
#undef QL_NTB
        const qlora_status st = launch_status();
        if (st != QLORA_OK) return st;
    }
    return QLORA_OK;
}

namespace {
struct TnLaunchB {
    const TnBatch& b;
    unsigned n;
    hipStream_t s;
    template <int TQ, bool V, int NST, int DT>
    void operator()() const {
        hipLaunchKernelGGL((tnb_kernel<TQ, V, NST, DT>), dim3(n), dim3(256), 0, s, b);
    }
};
}  // namespace

qlora_status launch_tn_batch(const TnDesc* d, int count, int r, int dt, hipStream_t s) {
    for (int i0 = 0; i0 < count; i0 += kTnBatch) {
        TnBatch b{};
        bool vec = false;
        int chunk = 64;
        unsigned total = 0;
        const qlora_status bs = tn_batch(d + i0, std::min(kTnBatch, count - i0), r, b, vec, chunk, total);
        if (bs != QLORA_OK) return bs;
        const TnLaunchB go{b, total, s};
        tn_dispatch(r, vec, chunk, dt, go);
        const qlora_status st = launch_status();
        if (st != QLORA_OK) return st;
    }
    return QLORA_OK;
}

qlora_status launch_expand_pooled(const uint16_t* A, int K, int r, int g, int dt, uint16_t* out, hipStream_t s) {
    const int64_t count = (int64_t)K * r;
    const int g_log2 = __builtin_ctz((unsigned)g);
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        hipLaunchKernelGGL(expand_pooled_kernel<DT>, dim3(blocks_for(count, 256)), dim3(256), 0, s, A, count, r, g_log2,
                           out);
    });
    return launch_status();
}

qlora_status launch_pool_rows(const float* in, int K, int r, int g, float* out, hipStream_t s) {
    const int64_t count = (int64_t)(K / g) * r;
    const int g_log2 = __builtin_ctz((unsigned)g);
    hipLaunchKernelGGL(pool_rows_kernel, dim3(blocks_for(count, 256)), dim3(256), 0, s, in, count, r, g, g_log2, out);
    return launch_status();
}

qlora_status launch_fill(float* out, int64_t count, float v, hipStream_t s) {
    if (count > 0) hipLaunchKernelGGL(fill_f32_kernel, dim3(blocks_for(count, 256)), dim3(256), 0, s, out, count, v);
    return launch_status();
}

}  // namespace qlora
