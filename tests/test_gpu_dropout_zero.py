"""A Dropout that drops nothing, on the GPU: every output is the call's without it, bit for bit, at decode sizes (one
launch) and past them."""
import pytest

from bit_nf4_quantized_15_amd import workloads

from gpu_util import dev_bf16, dev_f16, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base", ["nf4", "fp4", "int8", "fp8"])
@pytest.mark.parametrize("fmt,M,N,K,r", [("bf16", 1, 512, 1024, 16), ("f16", 8, 264, 512, 8), ("bf16", 16, 200, 2048, 24),
                                         ("bf16", 17, 320, 512, 64), ("f16", 100, 257, 704, 7)])
def test_outputs_are_those_without_dropout(base, fmt, M, N, K, r):
    import torch
    from bit_nf4_quantized_15_amd import qlora as q
    say(f"[dropout zero] {base} {fmt} M={M} N={N} K={K} r={r}")
    make, dev = (workloads.normal_bf16, dev_bf16) if fmt == "bf16" else (workloads.normal_f16, dev_f16)
    x, W, A, B, dy = (dev(make(11 + i, s, std)) for i, (s, std) in enumerate(
        [((M, K), 1.0), ((N, K), 0.02), ((K, r), r ** -0.5), ((r, N), 0.05), ((M, N), 0.5)]))
    w = {"int8": q.int8_quantize, "fp8": q.fp8_quantize}.get(base, lambda v: q.quantize(v, quant_type=base))(W)
    fwd = {"int8": q.int8_linear_fwd, "fp8": q.fp8_linear_fwd}.get(base, q.linear_fwd)
    dx = {"int8": q.int8_linear_bwd_dx, "fp8": q.fp8_linear_bwd_dx}.get(base, q.linear_bwd_dx)

    def outputs(drop):
        got = list(fwd(w, x, A, B, 16.0, dropout=drop)) + list(dx(w, A, B, 16.0, dy, dropout=drop))
        got.append(q.lora_down(x, A, 16.0, dropout=drop))
        if base in ("nf4", "fp4"):
            got += q.linear_bwd(w, x, A, B, 16.0, dy, dropout=drop)
            got += q.linear_bwd(w, x, A, B, 16.0, dy, t=got[1], need_dx=False, dropout=drop)[1:]
        return got

    plain = outputs(None)
    for p in (0.0, 0.4 / 65536):
        for i, (a, b) in enumerate(zip(outputs(q.Dropout(p, 5, 6)), plain)):
            assert torch.equal(a, b), i
