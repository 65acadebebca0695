// C ABI of the int8 layer: argument validation and dispatch (declared in include/qlora.h,
// section "int8").
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "int8.h"
#include "lora_plan.h"

using namespace qlora;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline uint8_t* at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }
inline int dt_of(int dtype) { return dtype == QLORA_DTYPE_F16 ? kDtF16 : kDtBf16; }
inline bool is16(int dtype) { return dtype == QLORA_DTYPE_BF16 || dtype == QLORA_DTYPE_F16; }

// A weight (min_rows 1) or activations (min_rows 0, where an empty one needs no pointers).
qlora_status check_int8(const qlora_int8* q, int64_t min_rows) {
    if (!q || q->rows < min_rows || q->cols < 1 || !is16(q->dtype)) return QLORA_ERR_INVALID_ARG;
    if (q->cols % kBlock || q->rows > INT32_MAX || q->cols > INT32_MAX) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (q->rows == 0) return QLORA_OK;
    if (!q->codes || !q->scale) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(q->codes) || !aligned16(q->scale)) return QLORA_ERR_MISALIGNED;
    return QLORA_OK;
}

inline bool bad_rank(int r) { return r < 0 || r > 128; }
inline bool bad_m(int64_t M) { return M < 0 || M > INT32_MAX; }
inline bool bad_sizes(int64_t M, int64_t N, int64_t K, int r) {
    return bad_m(M) || N < 1 || K < 1 || N > INT32_MAX || K > INT32_MAX || bad_rank(r);
}

struct FwdWs {
    size_t codes, scale, tbuf, part, total;  // x in 8 bits; t when the caller keeps none; the products' own
};
inline FwdWs fwd_ws(int64_t M, int64_t N, int64_t K, int r) {
    FwdWs w{};
    if (int8_gemv_supported(M, N, K, r)) {   // one launch; codes only where it does not make them itself
        w.scale = align256((size_t)M * K);
        w.part = w.scale + align256((size_t)M * 4);
        w.total = w.part + int8_gemv_workspace(r);
        return w;
    }
    w.codes = 0;
    w.scale = align256((size_t)M * K);
    w.tbuf = w.scale + align256((size_t)M * 4);
    w.part = w.tbuf + align256((size_t)M * r * 2);
    w.total = w.part + int8_gemm_fwd_workspace(M, N, K);
    return w;
}

}  // namespace

extern "C" {

qlora_status qlora_int8_quantize(const uint16_t* x, const qlora_int8* out, void* stream) {
    const qlora_status st = check_int8(out, 0);
    if (st != QLORA_OK) return st;
    if (out->rows == 0) return QLORA_OK;
    if (!x) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(x)) return QLORA_ERR_MISALIGNED;
    return launch_int8_quantize(x, out->rows, out->cols, out->codes, out->scale, dt_of(out->dtype),
                                (hipStream_t)stream);
}

qlora_status qlora_int8_dequantize(const qlora_int8* q, uint16_t* out, void* stream) {
    const qlora_status st = check_int8(q, 0);
    if (st != QLORA_OK) return st;
    if (q->rows == 0) return QLORA_OK;
    if (!out) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(out)) return QLORA_ERR_MISALIGNED;
    return launch_int8_dequantize(q->codes, q->scale, q->rows, q->cols, dt_of(q->dtype), out, (hipStream_t)stream);
}

size_t qlora_int8_fwd_workspace(int64_t M, int64_t N, int64_t K, int r) {
    if (bad_sizes(M, N, K, r) || M == 0 || K % kBlock) return 0;
    return fwd_ws(M, N, K, r).total;
}

qlora_status qlora_int8_linear_fwd(const qlora_int8* w, const uint16_t* x, int64_t M, const uint16_t* A,
                                   const uint16_t* B, int r, float alpha, uint16_t* y, uint16_t* t_out,
                                   const qlora_int8* x_keep, void* ws, size_t ws_bytes, void* stream) {
    qlora_status st = check_int8(w, 1);
    if (st != QLORA_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    if (bad_m(M) || bad_rank(r) || (r && !std::isfinite(alpha))) return QLORA_ERR_INVALID_ARG;
    if (K >= kInt8MaxK || N > kInt8MaxRows || M > kInt8MaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (x_keep) {
        if ((st = check_int8(x_keep, 0)) != QLORA_OK) return st;
        if (x_keep->rows != M || x_keep->cols != K || x_keep->dtype != w->dtype) return QLORA_ERR_INVALID_ARG;
    }
    if (M == 0) return QLORA_OK;
    if (!x || !y || (r && (!A || !B)) || (!r && (A || B || t_out))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(A) || !aligned16(B) || !aligned16(t_out))
        return QLORA_ERR_MISALIGNED;
    const FwdWs W = fwd_ws(M, N, K, r);
    if (!ws || ws_bytes < W.total) return QLORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return QLORA_ERR_MISALIGNED;
    hipStream_t s = (hipStream_t)stream;
    const int dt = dt_of(w->dtype);
    int8_t* xq = x_keep ? x_keep->codes : reinterpret_cast<int8_t*>(at(ws, W.codes));
    float* sx = x_keep ? x_keep->scale : reinterpret_cast<float*>(at(ws, W.scale));
    uint16_t* t = t_out ? t_out : reinterpret_cast<uint16_t*>(at(ws, W.tbuf));
    const float scale = r ? alpha / (float)r : 0.0f;
    if (int8_gemv_supported(M, N, K, r)) {
        if (!x_keep && int8_gemv_quantizes(M, K)) xq = nullptr;
        else if ((st = launch_int8_quantize(x, M, K, xq, sx, dt, s)) != QLORA_OK) return st;
        return launch_int8_gemv(x, xq, sx, w->codes, w->scale, nullptr, A, B, scale, y, t_out, at(ws, W.part), (int)M,
                                (int)N, (int)K, r, dt, s);
    }
    st = r ? launch_int8_prep(x, A, scale, (int)M, (int)K, r, xq, sx, t, dt, s)
           : launch_int8_quantize(x, M, K, xq, sx, dt, s);
    if (st != QLORA_OK) return st;
    return launch_int8_gemm_fwd(xq, sx, w->codes, w->scale, r ? t : nullptr, B, y, (int)M, (int)N, (int)K, r, dt,
                                at(ws, W.part), s);
}

qlora_status qlora_int8_gemm_fwd(const qlora_int8* w, const qlora_int8* x, const uint16_t* t, const uint16_t* B,
                                 int r, uint16_t* y, void* stream) {
    qlora_status st = check_int8(w, 1);
    if (st != QLORA_OK || (st = check_int8(x, 0)) != QLORA_OK) return st;
    if (x->cols != w->cols || x->dtype != w->dtype || bad_rank(r)) return QLORA_ERR_INVALID_ARG;
    if (w->cols >= kInt8MaxK || w->rows > kInt8MaxRows || x->rows > kInt8MaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (x->rows == 0) return QLORA_OK;
    if (!y || (r && (!t || !B)) || (!r && (t || B))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(y) || !aligned16(t) || !aligned16(B)) return QLORA_ERR_MISALIGNED;
    if (int8_gemv_supported(x->rows, w->rows, w->cols, r))
        return launch_int8_gemv(nullptr, x->codes, x->scale, w->codes, w->scale, t, nullptr, B, 0.0f, y, nullptr, nullptr,
                                (int)x->rows, (int)w->rows, (int)w->cols, r, dt_of(w->dtype), (hipStream_t)stream);
    return launch_int8_gemm_fwd(x->codes, x->scale, w->codes, w->scale, t, B, y, (int)x->rows, (int)w->rows,
                                (int)w->cols, r, dt_of(w->dtype), nullptr, (hipStream_t)stream);
}

// the split sums of u, in front of the product's own
static size_t dx_product_ws(int64_t M, int64_t N, int r) { return r ? align256(nt_ws_bytes(M, N, r)) : 0; }

size_t qlora_int8_linear_bwd_dx_workspace(int64_t M, int64_t N, int64_t K, int r) {
    if (bad_sizes(M, N, K, r) || M == 0 || K % kBlock) return 0;
    return dx_product_ws(M, N, r) + int8_gemm_dx_workspace(M, N, K);
}

qlora_status qlora_int8_linear_bwd_dx(const qlora_int8* w, int64_t M, const uint16_t* A, const uint16_t* B, int r,
                                      float alpha, const uint16_t* dy, uint16_t* u, uint16_t* dx, void* ws,
                                      size_t ws_bytes, void* stream) {
    qlora_status st = check_int8(w, 1);
    if (st != QLORA_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    if (bad_m(M) || bad_rank(r) || (r && !std::isfinite(alpha))) return QLORA_ERR_INVALID_ARG;
    if (K >= kInt8DxMaxK || N >= kInt8DxMaxN || M > kInt8MaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return QLORA_OK;
    if (!dy || !dx || (r && (!A || !B || !u)) || (!r && (A || B || u))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(dy) || !aligned16(u) || !aligned16(dx))
        return QLORA_ERR_MISALIGNED;
    const size_t need = qlora_int8_linear_bwd_dx_workspace(M, N, K, r);
    if (need && (!ws || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
    if (need && !aligned16(ws)) return QLORA_ERR_MISALIGNED;
    hipStream_t s = (hipStream_t)stream;
    const int dt = dt_of(w->dtype);
    if (r) {
        st = int8_u_supported(M, N, r) ? launch_int8_u(dy, B, alpha / (float)r, (int)M, (int)N, r, u, dt, s)
                                       : launch_nt(dy, B, false, ws, u, alpha / (float)r, (int)M, (int)N, r, dt, s);
        if (st != QLORA_OK) return st;
    }
    return launch_int8_gemm_bwd_dx(dy, w->codes, w->scale, u, A, dx, (int)M, (int)N, (int)K, r, dt,
                                   need ? at(ws, dx_product_ws(M, N, r)) : nullptr, s);
}

qlora_status qlora_int8_gemm_bwd_dx(const qlora_int8* w, const uint16_t* dy, int64_t M, const uint16_t* u,
                                    const uint16_t* A, int r, uint16_t* dx, void* stream) {
    const qlora_status st = check_int8(w, 1);
    if (st != QLORA_OK) return st;
    if (bad_m(M) || bad_rank(r)) return QLORA_ERR_INVALID_ARG;
    if (w->cols >= kInt8DxMaxK || w->rows >= kInt8DxMaxN || M > kInt8MaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return QLORA_OK;
    if (!dy || !dx || (r && (!u || !A)) || (!r && (u || A))) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(dx) || !aligned16(u) || !aligned16(A)) return QLORA_ERR_MISALIGNED;
    return launch_int8_gemm_bwd_dx(dy, w->codes, w->scale, u, A, dx, (int)M, (int)w->rows, (int)w->cols, r,
                                   dt_of(w->dtype), nullptr, (hipStream_t)stream);
}

// Tiles of one launch of the gradient kernel: the layers [i0, i0 + n) of a batch.
static int64_t grads_tiles(const qlora_lora_grads_int8* layers, int n) {
    int64_t t = 0;
    for (int i = 0; i < n; ++i)
        if (layers[i].M > 0) t += (layers[i].K + 127) / 128 + (layers[i].N + 127) / 128;
    return t;
}

size_t qlora_lora_grads_batch_int8_workspace(const qlora_lora_grads_int8* layers, int count, int r) {
    if (!layers || count <= 0 || r < 1 || r > 128) return 0;
    for (int i = 0; i < count; ++i)
        if (bad_sizes(layers[i].M, layers[i].N, layers[i].K, r)) return 0;
    size_t total = 0;
    for (int i0 = 0; i0 < count; i0 += kInt8GradLayers) {
        const int n = std::min(kInt8GradLayers, count - i0);
        const int64_t tiles = grads_tiles(layers + i0, n);
        for (int i = i0; i < i0 + n; ++i) {
            const qlora_lora_grads_int8& g = layers[i];
            if (g.M > 0) total += plan_int8_grad(g.M, g.K, r, tiles).ws + plan_int8_grad(g.M, g.N, r, tiles).ws;
        }
    }
    return total;
}

qlora_status qlora_lora_grads_batch_int8(const qlora_lora_grads_int8* layers, int count, int r, int dtype, void* ws,
                                         size_t ws_bytes, void* stream) {
    if (count < 0 || r < 1 || r > 128 || !is16(dtype)) return QLORA_ERR_INVALID_ARG;
    if (count == 0) return QLORA_OK;
    if (!layers) return QLORA_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {  // every entry is checked before anything is launched
        const qlora_lora_grads_int8& g = layers[i];
        if (bad_sizes(g.M, g.N, g.K, r) || !g.dA || !g.dB) return QLORA_ERR_INVALID_ARG;
        // rows of at most 8 MB: the kernel counts what is left of a wave's rows, and the steps in
        // flight past their end, in 32 signed bits
        if (g.K % kBlock || g.K > (int64_t(1) << 22) || g.N > (int64_t(1) << 22) || g.M > kInt8MaxRows)
            return QLORA_ERR_UNSUPPORTED_SHAPE;
        if (!aligned16(g.dA) || !aligned16(g.dB)) return QLORA_ERR_MISALIGNED;
        if (g.M == 0) continue;
        if (!g.x || !g.x_scale || !g.t || !g.u || !g.dy) return QLORA_ERR_INVALID_ARG;
        if (!aligned16(g.x) || !aligned16(g.x_scale) || !aligned16(g.t) || !aligned16(g.u) || !aligned16(g.dy))
            return QLORA_ERR_MISALIGNED;
    }
    const size_t need = qlora_lora_grads_batch_int8_workspace(layers, count, r);
    if (need && (!ws || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
    if (need && !aligned16(ws)) return QLORA_ERR_MISALIGNED;
    hipStream_t s = (hipStream_t)stream;
    size_t off = 0;
    qlora_status st;
    for (int i0 = 0; i0 < count; i0 += kInt8GradLayers) {
        const int n = std::min(kInt8GradLayers, count - i0);
        const int64_t tiles = grads_tiles(layers + i0, n);
        Int8GradDesc d[2 * kInt8GradLayers];
        int m = 0;
        for (int i = i0; i < i0 + n; ++i) {
            const qlora_lora_grads_int8& g = layers[i];
            if (g.M == 0) {  // empty sums
                if ((st = launch_fill(g.dA, g.K * r, 0.0f, s)) != QLORA_OK) return st;
                if ((st = launch_fill(g.dB, (int64_t)r * g.N, 0.0f, s)) != QLORA_OK) return st;
                continue;
            }
            d[m] = Int8GradDesc{g.x, g.x_scale, g.u, g.dA, at(ws, off), (int)g.M, (int)g.K,
                                plan_int8_grad(g.M, g.K, r, tiles)};
            off += d[m++].plan.ws;
            d[m] = Int8GradDesc{g.dy, nullptr, g.t, g.dB, at(ws, off), (int)g.M, (int)g.N,
                                plan_int8_grad(g.M, g.N, r, tiles)};
            off += d[m++].plan.ws;
        }
        if ((st = launch_int8_grads(d, m, r, dt_of(dtype), s)) != QLORA_OK) return st;
    }
    return QLORA_OK;
}

}  // extern "C"
