// C ABI of the 8-bit float layer: argument validation and dispatch (declared in include/qlora.h,
// section "fp8").
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fp8.h"
#include "lora_plan.h"

using namespace qlora;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline uint8_t* at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }
inline int dt_of(int dtype) { return dtype == QLORA_DTYPE_F16 ? kDtF16 : kDtBf16; }
inline bool is16(int dtype) { return dtype == QLORA_DTYPE_BF16 || dtype == QLORA_DTYPE_F16; }

// A tile's panels (256 rows of codes or of 16-bit outputs) lie within 31-bit offsets.
constexpr int64_t kMaxWidth = int64_t(1) << 22;
// Rows are counted in 32 bits up to a tile past the last.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 16384;

inline int64_t scale_stride(int64_t rows, int64_t cols, int block_rows) {
    return pad4(block_rows == 1 ? rows : fp8_blocks(cols));
}

// Elements of a tensor that the codes are made of, or restored to: 16 a thread of a grid.
constexpr int64_t kMaxElements = int64_t(1) << 36;

// A weight (min_rows 1) or activations (min_rows 0, where an empty one needs no pointers).
qlora_status check_fp8(const qlora_fp8* q, int64_t min_rows) {
    if (!q || q->rows < min_rows || q->cols < 1 || !is16(q->dtype)) return QLORA_ERR_INVALID_ARG;
    if (q->block_rows != 1 && q->block_rows != kFp8Block) return QLORA_ERR_INVALID_ARG;
    if (q->cols % kBlock || q->cols >= kMaxWidth || q->rows > kMaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (q->rows == 0) return QLORA_OK;
    if (!q->codes || !q->scale) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(q->codes) || !aligned16(q->scale)) return QLORA_ERR_MISALIGNED;
    return QLORA_OK;
}
qlora_status check_weight(const qlora_fp8* w) {
    const qlora_status st = check_fp8(w, 1);
    if (st != QLORA_OK) return st;
    if (w->block_rows != kFp8Block) return QLORA_ERR_INVALID_ARG;
    return w->rows >= kMaxWidth ? QLORA_ERR_UNSUPPORTED_SHAPE : QLORA_OK;
}

inline bool bad_rank(int r) { return r < 0 || r > 128; }
inline bool bad_m(int64_t M) { return M < 0 || M > INT32_MAX; }
inline bool bad_sizes(int64_t M, int64_t N, int64_t K, int r) {
    return bad_m(M) || M > kMaxRows || N < 1 || K < 1 || N >= kMaxWidth || K >= kMaxWidth || K % kBlock || bad_rank(r);
}

// The 8-bit operand [M, C]: codes in rows of whole blocks, its scales, then t (where the caller
// keeps none), the split sums of t or u, and the product's own.
struct Ws {
    size_t scale, tbuf, prep, part, total;
    int64_t ld, rs;
};
Ws layer_ws(int64_t M, int64_t N, int64_t K, int r, bool dx) {
    const int64_t C = dx ? N : K;
    Ws w{};
    w.ld = fp8_blocks(C) * kFp8Block;
    w.rs = pad4(M);
    w.scale = align256((size_t)M * w.ld);
    w.tbuf = w.scale + align256((size_t)fp8_blocks(C) * w.rs);
    w.prep = w.tbuf + (dx ? 0 : align256((size_t)M * r * 2));
    w.part = w.prep + (r ? align256(fp8_prep_ws(M, C, r)) : 0);
    w.total = w.part + (!dx && fp8_gemv_supported(M, K) ? fp8_gemv_workspace(r) : fp8_gemm_workspace(M, N, K, dx));
    return w;
}

}  // namespace

extern "C" {

size_t qlora_fp8_scale_bytes(int64_t rows, int64_t cols, int block_rows) {
    if (rows < 0 || cols < 1 || (block_rows != 1 && block_rows != kFp8Block)) return 0;
    return (size_t)scale_stride(rows, cols, block_rows) *
           (size_t)(block_rows == 1 ? fp8_blocks(cols) : fp8_blocks(rows));
}

qlora_status qlora_fp8_quantize(const uint16_t* x, const qlora_fp8* out, void* stream) {
    const qlora_status st = check_fp8(out, 0);
    if (st != QLORA_OK) return st;
    if (out->rows == 0) return QLORA_OK;
    if (out->rows * out->cols >= kMaxElements) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (!x) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(x)) return QLORA_ERR_MISALIGNED;
    const int64_t rs = scale_stride(out->rows, out->cols, out->block_rows);
    if (out->block_rows == 1)
        return launch_fp8_quantize_rows(x, out->rows, out->cols, out->codes, out->cols, out->scale, rs, dt_of(out->dtype),
                                        (hipStream_t)stream);
    return launch_fp8_quantize_blocks(x, out->rows, out->cols, out->codes, out->scale, rs, dt_of(out->dtype),
                                      (hipStream_t)stream);
}

qlora_status qlora_fp8_dequantize(const qlora_fp8* q, uint16_t* out, void* stream) {
    const qlora_status st = check_fp8(q, 0);
    if (st != QLORA_OK) return st;
    if (q->rows == 0) return QLORA_OK;
    if (q->rows * q->cols >= kMaxElements) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (!out) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(out)) return QLORA_ERR_MISALIGNED;
    return launch_fp8_dequantize(q->codes, q->scale, q->rows, q->cols, scale_stride(q->rows, q->cols, q->block_rows),
                                 q->block_rows == 1, dt_of(q->dtype), out, (hipStream_t)stream);
}

size_t qlora_fp8_fwd_workspace(int64_t M, int64_t N, int64_t K, int r) {
    return bad_sizes(M, N, K, r) || M == 0 ? 0 : layer_ws(M, N, K, r, false).total;
}

qlora_status qlora_fp8_linear_fwd(const qlora_fp8* w, const uint16_t* x, int64_t M, const uint16_t* A,
                                  const uint16_t* B, int r, float alpha, const qlora_dropout* drop, uint16_t* y,
                                  uint16_t* t_out, void* ws, size_t ws_bytes, void* stream) {
    qlora_status st = check_weight(w);
    if (st != QLORA_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    DropArgs d;
    if (bad_m(M) || bad_rank(r) || (r && !std::isfinite(alpha)) || !drop_args(drop, &d)) return QLORA_ERR_INVALID_ARG;
    if (M > kMaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return QLORA_OK;
    if (!x || !y || (r && (!A || !B)) || (!r && (A || B || drop || t_out))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(A) || !aligned16(B) || !aligned16(t_out))
        return QLORA_ERR_MISALIGNED;
    const Ws W = layer_ws(M, N, K, r, false);
    if (!ws || ws_bytes < W.total) return QLORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return QLORA_ERR_MISALIGNED;
    hipStream_t s = (hipStream_t)stream;
    const int dt = dt_of(w->dtype);
    uint8_t *xq = at(ws, 0), *sx = at(ws, W.scale);
    uint16_t* t = t_out ? t_out : reinterpret_cast<uint16_t*>(at(ws, W.tbuf));
    Fp8Gemm g{xq, sx, w->codes, w->scale, r ? t : nullptr, B, y, (int)M, (int)N, (int)K, r, (int)W.ld, W.rs,
              scale_stride(N, K, kFp8Block), DropArgs{}};
    const bool few = fp8_gemv_supported(M, K);
    if (few && !d.thr) {   // t and, where there is room, the codes of x in the launch itself
        if (fp8_gemv_quantizes(M, K)) g.x = nullptr;
        else if ((st = launch_fp8_quantize_rows(x, M, K, xq, W.ld, sx, W.rs, dt, s)) != QLORA_OK) return st;
        g.t = nullptr;
        return launch_fp8_gemv(g, x, A, r ? alpha / (float)r : 0.0f, t_out, at(ws, W.part), dt, s);
    }
    st = r ? launch_fp8_prep(x, A, true, d, alpha / (float)r, (int)M, (int)K, r, xq, W.ld, sx, W.rs, t, at(ws, W.prep), dt, s)
           : launch_fp8_quantize_rows(x, M, K, xq, W.ld, sx, W.rs, dt, s);
    if (st != QLORA_OK) return st;
    if (few) return launch_fp8_gemv(g, nullptr, nullptr, 0.0f, nullptr, nullptr, dt, s);
    return launch_fp8_gemm(g, false, dt, at(ws, W.part), s);
}

qlora_status qlora_fp8_gemm_fwd(const qlora_fp8* w, const qlora_fp8* x, const uint16_t* t, const uint16_t* B, int r,
                                uint16_t* y, void* stream) {
    qlora_status st = check_weight(w);
    if (st != QLORA_OK || (st = check_fp8(x, 0)) != QLORA_OK) return st;
    if (x->block_rows != 1 || x->cols != w->cols || x->dtype != w->dtype || bad_rank(r)) return QLORA_ERR_INVALID_ARG;
    if (x->rows == 0) return QLORA_OK;
    if (!y || (r && (!t || !B)) || (!r && (t || B))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(y) || !aligned16(t) || !aligned16(B)) return QLORA_ERR_MISALIGNED;
    const Fp8Gemm g{x->codes, x->scale, w->codes, w->scale, t, B, y, (int)x->rows, (int)w->rows, (int)w->cols, r,
                    (int)x->cols, pad4(x->rows), scale_stride(w->rows, w->cols, kFp8Block), DropArgs{}};
    if (fp8_gemv_supported(g.M, g.K))
        return launch_fp8_gemv(g, nullptr, nullptr, 0.0f, nullptr, nullptr, dt_of(w->dtype), (hipStream_t)stream);
    return launch_fp8_gemm(g, false, dt_of(w->dtype), nullptr, (hipStream_t)stream);
}

size_t qlora_fp8_linear_bwd_dx_workspace(int64_t M, int64_t N, int64_t K, int r) {
    return bad_sizes(M, N, K, r) || M == 0 ? 0 : layer_ws(M, N, K, r, true).total;
}

qlora_status qlora_fp8_linear_bwd_dx(const qlora_fp8* w, int64_t M, const uint16_t* A, const uint16_t* B, int r,
                                     float alpha, const qlora_dropout* drop, const uint16_t* dy, uint16_t* u,
                                     uint16_t* dx, void* ws, size_t ws_bytes, void* stream) {
    qlora_status st = check_weight(w);
    if (st != QLORA_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    DropArgs d;
    if (bad_m(M) || bad_rank(r) || (r && !std::isfinite(alpha)) || !drop_args(drop, &d)) return QLORA_ERR_INVALID_ARG;
    if (M > kMaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return QLORA_OK;
    if (!dy || !dx || (r && (!A || !B || !u)) || (!r && (A || B || drop || u))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(dy) || !aligned16(u) || !aligned16(dx))
        return QLORA_ERR_MISALIGNED;
    const Ws W = layer_ws(M, N, K, r, true);
    if (!ws || ws_bytes < W.total) return QLORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return QLORA_ERR_MISALIGNED;
    hipStream_t s = (hipStream_t)stream;
    const int dt = dt_of(w->dtype);
    uint8_t *dq = at(ws, 0), *sd = at(ws, W.scale);
    const DropArgs none{0u, 0u, 0u, 0u, 0u, 1.0f};
    st = r ? launch_fp8_prep(dy, B, false, none, alpha / (float)r, (int)M, (int)N, r, dq, W.ld, sd, W.rs, u, at(ws, W.prep),
                             dt, s)
           : launch_fp8_quantize_rows(dy, M, N, dq, W.ld, sd, W.rs, dt, s);
    if (st != QLORA_OK) return st;
    const Fp8Gemm g{dq, sd, w->codes, w->scale, u, A, dx, (int)M, (int)N, (int)K, r, (int)W.ld, W.rs,
                    scale_stride(N, K, kFp8Block), d};
    return launch_fp8_gemm(g, true, dt, at(ws, W.part), s);
}

}  // extern "C"
