"""Gradients with dropout against float64 in every form of their kernel: ranks of each class and their remainders, widths
that are no whole 4 columns (of x too: the generator's units of 8 then end inside a row), one split and many, rows that
end inside a step; and what lies behind the outputs."""
import numpy as np
import pytest

from oracle import dropout
from test_gpu_dropout import FMT, OFFSET, SEED, bits, close, f64

from gpu_util import say

pytestmark = pytest.mark.gpu

# dtype, r, M, N, K
CASES = [
    ("bf16", 1, 1, 1, 1), ("f16", 2, 15, 3, 9), ("bf16", 31, 17, 130, 131), ("f16", 32, 129, 64, 128),
    ("bf16", 33, 300, 134, 190), ("f16", 34, 257, 131, 64), ("bf16", 63, 700, 66, 129), ("f16", 64, 513, 260, 132),
    ("bf16", 65, 1029, 127, 136), ("f16", 68, 640, 128, 260), ("bf16", 96, 2050, 140, 65), ("f16", 126, 511, 70, 257),
    ("bf16", 127, 1300, 37, 70), ("f16", 128, 2047, 256, 384), ("bf16", 8, 9000, 64, 64), ("f16", 5, 6001, 30, 200),
    ("bf16", 64, 5000, 1000, 2056), ("f16", 16, 4100, 8200, 520),
]


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


@pytest.mark.parametrize("fmt,r,M,N,K", CASES)
def test_gradients(q, fmt, r, M, N, K):
    import torch
    say(f"[dropout grads] {fmt} r={r} M={M} N={N} K={K}")
    m, dev, _, _ = FMT[fmt]
    p, guard = 0.3, 64
    host = [bits(fmt, 11 * r + j, s) for j, s in enumerate([(M, K), (M, r), (M, r), (M, N)])]
    x, t, u, dy = (m.to_f64(b) for b in host)
    rec = tuple(dev(b) for b in host)
    drop = q.Dropout(p, SEED, OFFSET)
    bufs = [torch.full((n + 2 * guard,), 7.0, dtype=torch.float32, device="cuda:0") for n in (K * r, r * N)]
    dA, dB = bufs[0][guard:-guard].view(K, r), bufs[1][guard:-guard].view(r, N)
    q.lora_grads_batch([rec], dA=[dA], dB=[dB], dropout=[drop])
    X = dropout.drop(x, p, SEED, OFFSET)
    for name, g, a, s in (("dA", dA, X, u), ("dB", dB, t, dy)):
        # M products added one after the other, the factor's rounding and that of its product
        close(f64(g), a.T @ s, (M + 10) * 2.0 ** -23 * (np.abs(a).T @ np.abs(s)) + 2.0 ** -149, name)
    for b in bufs:
        assert bool((b[:guard] == 7.0).all()) and bool((b[-guard:] == 7.0).all())
    again = q.lora_grads_batch([rec], dropout=[drop])
    assert torch.equal(again[0][0], dA) and torch.equal(again[1][0], dB)


def test_a_column_that_is_not_finite_stays_alone(q):
    """A NaN of x reaches its own column's gradients only, and not even those where it is dropped."""
    import torch
    say("[dropout grads] not finite")
    M, N, K, r = 200, 64, 192, 24
    x, t, u, dy = (torch.randn(s, device="cuda:0").to(torch.bfloat16) for s in [(M, K), (M, r), (M, r), (M, N)])
    drop = q.Dropout(0.5, SEED, OFFSET)
    want = q.lora_grads_batch([(x, t, u, dy)], dropout=[drop])[0][0]
    mask = dropout.mask(M, K, 0.5, SEED, OFFSET)
    for kept in (True, False):
        m, k = np.argwhere(mask == kept)[77]
        bad = x.clone()
        bad[m, k] = float("nan")
        got = q.lora_grads_batch([(bad, t, u, dy)], dropout=[drop])[0][0]
        assert bool(torch.isnan(got[k]).all()) == kept
        got[k] = want[k]
        assert torch.equal(got, want)


def test_no_tokens(q):
    """An empty batch through the layers with dropout: empty outputs, zero gradients."""
    import torch
    say("[dropout] M=0")
    N, K, r = 128, 192, 8
    bf = lambda *s: torch.randn(s, device="cuda:0").to(torch.bfloat16)
    A, B, W, x, dy = bf(K, r), bf(r, N), bf(N, K), bf(0, K), bf(0, N)
    drop = q.Dropout(0.1, SEED, OFFSET)
    w4, w8, wf = q.quantize(W), q.int8_quantize(W), q.fp8_quantize(W)
    for fwd, w in ((q.linear_fwd, w4), (q.int8_linear_fwd, w8), (q.fp8_linear_fwd, wf)):
        y, t = fwd(w, x, A, B, 16.0, dropout=drop)
        assert tuple(y.shape) == (0, N) and tuple(t.shape) == (0, r)
    for bwd, w in ((q.linear_bwd_dx, w4), (q.int8_linear_bwd_dx, w8), (q.fp8_linear_bwd_dx, wf)):
        u, dx = bwd(w, A, B, 16.0, dy, dropout=drop)
        assert tuple(u.shape) == (0, r) and tuple(dx.shape) == (0, K)
    dx, dA, dB = q.linear_bwd(w4, x, A, B, 16.0, dy, dropout=drop)
    assert tuple(dx.shape) == (0, K) and not dA.any() and not dB.any()
