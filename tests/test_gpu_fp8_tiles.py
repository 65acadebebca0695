"""Every tile, split and decode form of the fp8 layer against float64, at the sizes of fp8_sizes.py (their kernels are
checked in test_fp8_plan.py), with the bounds of test_gpu_fp8.py; and the split preparation."""
import numpy as np
import pytest

import fp8_sizes
from oracle import fp8
from test_gpu_fp8 import FMT, OFFSET, SEED, Layer, bits, close, code_bits, f64

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


@pytest.mark.parametrize("tile,splits,fmt,M,N,K,r", fp8_sizes.FWD)
def test_forward(q, tile, splits, fmt, M, N, K, r):
    import torch
    say(f"[fp8 fwd] {tile}/{splits} {fmt} M={M} N={N} K={K} r={r}")
    L = Layer(q, fmt, 20 + M, M, N, K, r)
    y, t = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)
    if r:
        L.check_t(t)
    L.check_y(y, t)
    again, _ = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)
    assert torch.equal(y, again)                                    # sums in one order
    L.check_y(q.fp8_gemm_fwd(L.w, q.fp8_quantize_rows(L.x), t, L.B), t)   # (without a workspace: no splits)


@pytest.mark.parametrize("tile,splits,fmt,M,N,K,r,p", fp8_sizes.DX)
def test_input_gradient(q, tile, splits, fmt, M, N, K, r, p):
    import torch
    say(f"[fp8 dx] {tile}/{splits} {fmt} M={M} N={N} K={K} r={r} p={p}")
    L = Layer(q, fmt, 40 + M, M, N, K, r)
    drop = q.Dropout(p, SEED, OFFSET) if p else None
    u, dx = q.fp8_linear_bwd_dx(L.w, L.A, L.B, L.alpha, L.dy, dropout=drop)
    if r:
        L.check_u(u)
    L.check_dx(dx, u, drop)
    assert torch.equal(dx, q.fp8_linear_bwd_dx(L.w, L.A, L.B, L.alpha, L.dy, dropout=drop)[1])


@pytest.mark.parametrize("own,turns,fmt,M,N,K,r", fp8_sizes.DECODE)
def test_decode(q, own, turns, fmt, M, N, K, r):
    import torch
    say(f"[fp8 decode] own={own} {fmt} M={M} N={N} K={K} r={r}")
    L = Layer(q, fmt, 60 + M, M, N, K, r)
    y, t = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)
    if r:
        L.check_t(t)
    L.check_y(y, t)
    assert torch.equal(y, q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)[0])
    L.check_y(q.fp8_gemm_fwd(L.w, q.fp8_quantize_rows(L.x), t, L.B), t)
    if r:                                                           # with dropout: t and codes made before
        drop = q.Dropout(0.3, SEED, OFFSET)
        y, t = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha, dropout=drop)
        L.check_t(t, drop)
        L.check_y(y, t)


@pytest.mark.parametrize("splits,fmt,M,C,r", fp8_sizes.PREP)
def test_preparation(q, splits, fmt, M, C, r):
    """t and u of few outputs and inputs: the sums over C alone, and the codes through a product with the identity."""
    import torch
    say(f"[fp8 prep] splits={splits} {fmt} M={M} C={C} r={r}")
    m, dev, h, sub = FMT[fmt]
    xb, Ab, Bb = bits(fmt, 7 + M, (M, C)), bits(fmt, 8 + C, (C, r), r ** -0.5), bits(fmt, 9 + C, (r, C), 0.05)
    x, xf = dev(xb), m.to_f64(xb)
    # a weight whose first outputs pick single inputs: y is the value that a code stands for
    picks = np.random.default_rng(C).choice(C, size=min(C, 96), replace=False)
    eye = torch.zeros((len(picks), C), dtype=x.dtype, device="cuda:0")
    eye[torch.arange(len(picks)), torch.from_numpy(picks)] = 1.0
    w = q.fp8_quantize(eye)
    B0 = torch.zeros((r, len(picks)), dtype=x.dtype, device="cuda:0")
    y, t = q.fp8_linear_fwd(w, x, dev(Ab), B0, 16.0)
    s = 16.0 / r
    want, mag = s * (xf @ m.to_f64(Ab)), s * (np.abs(xf) @ np.abs(m.to_f64(Ab)))
    close(f64(t), want, (h * np.abs(want) + sub + (C + 10) * 2.0 ** -23 * mag) * (1 + h), "t")
    rows = np.unique(np.linspace(0, M - 1, 40).astype(int))
    codes, e = fp8.quantize(xb[rows], fmt, 1)
    assert np.array_equal(f64(y)[rows], fp8.values(codes, e, 1)[:, picks])   # (exact in 16 bits: 4 significant bits)
    # the same operand as a gradient (its rows are C outputs wide)
    w = q.fp8_quantize(eye.t().contiguous() if len(picks) % 64 == 0 else
                       torch.nn.functional.pad(eye.t(), (0, -len(picks) % 64)).contiguous())
    A0 = torch.zeros((w.cols, r), dtype=x.dtype, device="cuda:0")
    u, dx = q.fp8_linear_bwd_dx(w, A0, dev(Bb), 16.0, x)
    want, mag = s * (xf @ m.to_f64(Bb).T), s * (np.abs(xf) @ np.abs(m.to_f64(Bb).T))
    close(f64(u), want, (h * np.abs(want) + sub + (C + 10) * 2.0 ** -23 * mag) * (1 + h), "u")
    assert np.array_equal(f64(dx)[rows][:, :len(picks)], fp8.values(codes, e, 1)[:, picks])


def test_codes_of_a_layer_are_those_of_the_quantizer(q):
    """A rank-r layer's own preparation and fp8_quantize_rows give the product the same operand."""
    import torch
    say("[fp8] one operand")
    L = Layer(q, "bf16", 5, 200, 520, 1088, 24)
    y, t = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)
    xq = q.fp8_quantize_rows(L.x)
    assert np.array_equal(code_bits(xq), fp8.quantize(L.xb, "bf16", 1)[0])
    y2, _ = q.fp8_linear_fwd(L.w, L.x)
    assert torch.equal(q.fp8_gemm_fwd(L.w, xq), y2)
    assert torch.equal(q.fp8_gemm_fwd(L.w, xq, t, L.B), y)


def test_split_products_in_graphs_that_share_a_workspace(q):
    """Two layers whose products are split, a graph each, on one workspace, replayed in turn; and at once on two
    streams with a workspace each."""
    import torch
    say("[fp8] split products: graphs on one workspace, two streams")
    Ls = [Layer(q, "bf16", 71, 649, 1728, 5312, 64), Layer(q, "bf16", 72, 464, 5120, 2112, 24)]
    size = max(max(q.lib.qlora_fp8_fwd_workspace(L.M, L.N, L.K, L.r), q.lib.qlora_fp8_linear_bwd_dx_workspace(L.M, L.N, L.K, L.r))
               for L in Ls)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda:0")
    drop = q.Dropout(0.1, SEED, OFFSET)

    def call(L, ws):
        y, t = q.fp8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha, ws=ws, dropout=drop)
        u, dx = q.fp8_linear_bwd_dx(L.w, L.A, L.B, L.alpha, L.dy, ws=ws, dropout=drop)
        return y, t, u, dx
    want = [call(L, ws) for L in Ls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for L in Ls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(L, ws))
        graphs.append(g)
    for rep in range(3):
        for i, g in enumerate(graphs):
            for v in outs[i]:
                v.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), (rep, i)
        call(Ls[rep % 2], ws)
        torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in Ls], [ws, torch.empty_like(ws)]
    got = [[], []]
    for _ in range(3):
        for i, L in enumerate(Ls):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(L, spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
