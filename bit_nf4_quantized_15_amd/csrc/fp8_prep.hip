// What the 8-bit float layer needs of its 16-bit operand, in one pass: the operand's codes and
// scales (rows in blocks of 128), and the LoRA branch's product with it ("bitsandbytes deep
// dive", section 8.2; 12.2: the LoRA side path):
//   forward         x:  codes, t = RNE_16(s drop(x) A)
//   input gradient  dy: codes, u = RNE_16(s dy B^T)
// A block needs nothing beyond its own 128 columns, so the pass of lora_body.h (128 rows, a split
// of the columns in whole blocks, split sums of the product) writes the codes of what it holds in
// registers anyway.
#include "fp8.h"
#include "lora_body.h"

namespace qlora {
namespace {

template <int TQ, bool VEC, bool YNAT, int NST, int DT>
__global__ __launch_bounds__(256) void fp8_prep_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ Y,
                                                       uint64_t* __restrict__ tags, float* __restrict__ part,
                                                       uint16_t* __restrict__ out, float scale, int M, int C, int r,
                                                       int chunk, const NtMore more) {
    nt_body<TQ, VEC, YNAT, NST, DT, YNAT, true>(X, Y, tags, part, out, scale, M, C, r, chunk, (int)blockIdx.x,
                                                (int)blockIdx.y, (int)gridDim.x, (int)gridDim.y, more);
}

}  // namespace

size_t fp8_prep_ws(int64_t M, int64_t C, int r) { return split_ws_bytes((M + 127) / 128, plan_fp8_prep(M, C, r), r); }

qlora_status launch_fp8_prep(const uint16_t* X, const uint16_t* Y, bool y_natural, const DropArgs& drop, float scale,
                             int M, int C, int r, uint8_t* codes, int64_t ld, uint8_t* sx, int64_t rs, uint16_t* out,
                             void* ws, int dt, hipStream_t s) {
    const SplitPlan sp = plan_fp8_prep(M, C, r);
    const int tiles = (int)(((int64_t)M + 127) / 128);
    const dim3 grid((unsigned)tiles, (unsigned)sp.splits);
    if ((int64_t)tiles * 256 >= (int64_t(1) << 32) || sp.splits > 65535) return QLORA_ERR_UNSUPPORTED_SHAPE;
    uint64_t* tags = static_cast<uint64_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + split_tags_bytes(tiles, sp));
    // vector path: 16-byte aligned rows, and one workgroup's rows under 1 GiB of buffer offsets
    const bool vec = C % 8 == 0 && (!y_natural || r % 8 == 0) && (int64_t)C * 128 * 2 < (int64_t(1) << 30);
    const NtMore more{drop, codes, sx, ld, rs};
    const float f = scale * drop.inv;
    const int tq = (r + 31) / 32, nst = steps_template(sp.chunk);
#define QL_P(TQ, V, NAT, NST) \
    hipLaunchKernelGGL((fp8_prep_kernel<TQ, V, NAT, NST, DT>), grid, dim3(256), 0, s, X, Y, tags, part, out, f, M, C, r, \
                       sp.chunk, more);
#define QL_P1(TQ, V, NAT)                                  \
    if (nst == 2) { QL_P(TQ, V, NAT, 2) }                  \
    else if (nst == 4) { QL_P(TQ, V, NAT, 4) }             \
    else { QL_P(TQ, V, NAT, (TQ == 4 ? 4 : 8)) }
#define QL_P2(TQ)                                                                \
    if (y_natural) {                                                             \
        if (vec) { QL_P1(TQ, true, true) } else { QL_P1(TQ, false, true) }       \
    } else {                                                                     \
        if (vec) { QL_P1(TQ, true, false) } else { QL_P1(TQ, false, false) }     \
    }
    with_dt(dt, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        switch (tq) {
            case 1: QL_P2(1) break;
            case 2: QL_P2(2) break;
            case 3: QL_P2(3) break;
            default: QL_P2(4) break;
        }
    });
#undef QL_P2
#undef QL_P1
#undef QL_P
    return launch_status();
}

}  // namespace qlora
