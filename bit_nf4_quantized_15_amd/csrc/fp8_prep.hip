// What the 8-bit float layer needs of its 16-bit operand, in one pass: the operand's codes and
// scales (rows in blocks of 128), and the LoRA branch's product with it ("bitsandbytes deep
// dive", section 8.2; 12.2: the LoRA side path):
//   forward         x:  codes, t = RNE_16(s drop(x) A)
//   input gradient  dy: codes, u = RNE_16(s dy B^T)
// (the kernels of lora_prep.h).  A block needs nothing beyond its own 128 columns, so the pass
// that has them in registers for the product writes their codes too.
#include "lora_prep.h"

namespace qlora {
namespace {

template <int TQ, bool VEC, bool YNAT, bool DROP, int DT>
__global__ __launch_bounds__(256, TQ <= 2 ? 2 : 1) void fp8_prep_stream_kernel(const StreamArgs a) {
    stream_body<TQ, VEC, YNAT, DROP, true, DT>(a);
}

}  // namespace

size_t fp8_prep_ws(int64_t M, int64_t C, int r) { return stream_ws_bytes(M, C, r); }

qlora_status launch_fp8_prep(const uint16_t* X, const uint16_t* Y, bool y_natural, const DropArgs& drop, float scale,
                             int M, int C, int r, uint8_t* codes, int64_t ld, uint8_t* sx, int64_t rs, uint16_t* out,
                             void* ws, int dt, hipStream_t s) {
    const bool vec = C % 8 == 0 && (!y_natural || r % 8 == 0);
    StreamArgs a{};
    a.item[0] = stream_item(X, Y, out, ws, drop, scale, M, C, plan_stream(M, C, 1, C));
    a.q = PrepCodes{codes, sx, ld, rs};
    a.n = 1;
    a.r = r;
    const int64_t wgs = (int64_t)a.item[0].tiles * a.item[0].splits;
    if (wgs * 256 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    const dim3 grid((unsigned)wgs);
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
#define QL_S(TQ, V, NAT, DROP) \
    hipLaunchKernelGGL((fp8_prep_stream_kernel<TQ, V, NAT, DROP, DT>), grid, dim3(256), 0, s, a)
#define QL_S1(TQ)                                                                                        \
    if (!y_natural) { if (vec) QL_S(TQ, true, false, false); else QL_S(TQ, false, false, false); }       \
    else if (drop.thr) { if (vec) QL_S(TQ, true, true, true); else QL_S(TQ, false, true, true); }        \
    else { if (vec) QL_S(TQ, true, true, false); else QL_S(TQ, false, true, false); }
        switch ((r + 31) / 32) {
            case 1: QL_S1(1) break;
            case 2: QL_S1(2) break;
            case 3: QL_S1(3) break;
            default: QL_S1(4) break;
        }
#undef QL_S1
#undef QL_S
    });
    const qlora_status st = launch_status();
    return st == QLORA_OK ? launch_reduce(a, dt, s) : st;
}

}  // namespace qlora
