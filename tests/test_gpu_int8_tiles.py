"""Every kernel of the int8 layer (int8_sizes.py: each tile, split, row grouping and row tile) on the GPU, against
float64 products of torch on the device.  Codes and scales are compared bit for bit.  The bounds are those of
test_gpu_int8.py: h = eps / 2 of the 16-bit type for each rounding to it (and half its smallest subnormal), and
(n + 8) 2^-23 of the sum of the magnitudes for n fp32 products in any order.  Every output lies inside a larger
buffer that has to keep its values on both sides."""
import math

import pytest
import torch

import int8_sizes
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 2.0 ** -134), "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}
F32, I8, F64 = torch.float32, torch.int8, torch.float64
PAD = 4096


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


def mm(a, b):
    return torch.mm(a.contiguous(), b.contiguous())


def close(got, want, tol, what):
    bad = ~((got.to(F64) - want).abs() <= tol)
    n = int(bad.sum())
    if n:
        i = torch.nonzero(bad)[0].tolist()
        at = tuple(i)
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {i}: {float(got[at])} for {float(want[at])}, "
                             f"tolerance {float(tol[at])}")


def codes_of(x):
    """Codes and scales by the definition; 254 |x| and (2 j + 1) a are exact in float64."""
    v = x.to(F64)
    a = v.abs().amax(dim=1, keepdim=True)
    d = torch.where(a > 0, a, torch.ones_like(a))
    j = torch.floor(127.0 * v.abs() / d)
    c = j + (254.0 * v.abs() > (2.0 * j + 1.0) * d)
    return torch.where(v < 0, -c, c).to(I8), (a / 127.0).squeeze(1).to(F32)


class Guarded:
    """Outputs inside larger buffers."""

    def __init__(self):
        self.held = []

    def __call__(self, dtype, *shape):
        n = math.prod(shape)
        buf = torch.full((n + 2 * PAD,), 77, dtype=dtype, device="cuda:0")
        self.held.append((buf, n))
        return buf[PAD:PAD + n].view(*shape)

    def check(self):
        for i, (buf, n) in enumerate(self.held):
            assert bool((buf[:PAD] == 77).all()) and bool((buf[PAD + n:] == 77).all()), f"output {i}: written around it"


class Layer:
    def __init__(self, q, fmt, seed, M, N, K, r, alpha=24.0):
        self.dt, self.h, self.sub = TYPES[fmt]
        self.M, self.N, self.K, self.r, self.alpha, self.s = M, N, K, r, alpha, alpha / r if r else 0.0
        g = torch.Generator(device="cuda:0")
        g.manual_seed(seed)

        def normal(std, *shape):
            return (torch.randn(shape, generator=g, device="cuda:0") * std).to(self.dt)

        self.x, self.dy, self.w16 = normal(1.0, M, K), normal(0.5, M, N), normal(0.02, N, K)
        if M >= 3:
            self.x[M // 2] = 0                                     # a padded token
        self.A, self.B = (normal(r ** -0.5, K, r), normal(0.05, r, N)) if r else (None, None)
        self.q, self.w = q, q.int8_quantize(self.w16)
        self.cw, self.sw = codes_of(self.w16)
        assert torch.equal(self.w.codes, self.cw) and torch.equal(self.w.scale, self.sw)

    def forward(self, g, ws=None):
        keep = self.q.Int8Tensor(g(I8, self.M, self.K), g(F32, self.M), self.dt)
        y, t = g(self.dt, self.M, self.N), g(self.dt, self.M, self.r) if self.r else None
        self.q.int8_linear_fwd(self.w, self.x, self.A, self.B, self.alpha, y=y, t=t, keep=keep, ws=ws)
        return y, t, keep

    def check_t(self, t):
        x, A = self.x.to(F64), self.A.to(F64)
        want = self.s * mm(x, A)
        tol = self.h * want.abs() + self.sub + (self.K + 8) * 2.0 ** -23 * self.s * mm(x.abs(), A.abs())
        close(t, want, tol * (1 + self.h), "t")

    def check_y(self, y, t, keep):
        cx, sx = codes_of(self.x)
        assert torch.equal(keep.codes, cx), "codes of x"
        assert torch.equal(keep.scale, sx), "scales of x"
        want = mm(cx.to(F64), self.cw.to(F64).t()) * sx.to(F64)[:, None] * self.sw.to(F64)[None, :]
        mag = want.abs()
        if self.r:
            want = want + mm(t.to(F64), self.B.to(F64))
            mag = mag + mm(t.to(F64).abs(), self.B.to(F64).abs())
        tol = (self.r + 8) * 2.0 ** -23 * mag
        close(y, want, (tol + self.h * want.abs() + self.sub) * (1 + 2 * self.h), "y")

    def backward(self, g, ws=None):
        u, dx = g(self.dt, self.M, self.r) if self.r else None, g(self.dt, self.M, self.K)
        self.q.int8_linear_bwd_dx(self.w, self.A, self.B, self.alpha, self.dy, u=u, dx=dx, ws=ws)
        return u, dx

    def check_u(self, u):
        dy, B = self.dy.to(F64), self.B.to(F64)
        want = self.s * mm(dy, B.t())
        tol = self.h * want.abs() + self.sub + (self.N + 8) * 2.0 ** -23 * self.s * mm(dy.abs(), B.abs().t())
        close(u, want, tol * (1 + self.h), "u")

    def check_dx(self, dx, u):
        w = (self.cw.to(F64) * self.sw.to(F64)[:, None]).to(F32).to(self.dt).to(F64)
        dy = self.dy.to(F64)
        want, mag = mm(dy, w), mm(dy.abs(), w.abs())
        if self.r:
            want = want + mm(u.to(F64), self.A.to(F64).t())
            mag = mag + mm(u.to(F64).abs(), self.A.to(F64).abs().t())
        tol = (self.N + self.r + 8) * 2.0 ** -23 * mag
        close(dx, want, (tol + self.h * want.abs() + self.sub) * (1 + 2 * self.h), "dx")


def run_forward(q, fmt, seed, M, N, K, r):
    L, g = Layer(q, fmt, seed, M, N, K, r), Guarded()
    y, t, keep = L.forward(g)
    if r:
        L.check_t(t)
    L.check_y(y, t, keep)
    y2, t2 = q.int8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha, want_t=False)   # nothing kept: the same y
    assert t2 is None and torch.equal(y2, y)
    y3 = g(L.dt, M, N)                                                      # the product for given codes and t
    q.int8_gemm_fwd(L.w, keep, t, L.B, y=y3)
    L.check_y(y3, t, keep)
    g.check()


@pytest.mark.parametrize("tile,splits,fmt,M,N,K,r", int8_sizes.FWD)
def test_forward_tiles(q, tile, splits, fmt, M, N, K, r):
    say(f"[int8 fwd {tile} split {splits}] {fmt} M={M} N={N} K={K} r={r}")
    run_forward(q, fmt, M + N + K, M, N, K, r)


@pytest.mark.parametrize("own,turns,fmt,M,N,K,r", int8_sizes.DECODE)
def test_decode_row_tiles(q, own, turns, fmt, M, N, K, r):
    say(f"[int8 decode, {turns} row tiles] {fmt} M={M} N={N} K={K} r={r}")
    run_forward(q, fmt, M + N + K, M, N, K, r)


@pytest.mark.parametrize("per,fmt,M,K,r", int8_sizes.PREP)
def test_preparation_groups(q, per, fmt, M, K, r):
    say(f"[int8 prep, {per} tokens each] {fmt} M={M} K={K} r={r}")
    run_forward(q, fmt, M + K, M, 72, K, r)


@pytest.mark.parametrize("tile,splits,fmt,M,N,K,r", int8_sizes.DX)
def test_input_gradient_tiles(q, tile, splits, fmt, M, N, K, r):
    say(f"[int8 dx {tile} split {splits}] {fmt} M={M} N={N} K={K} r={r}")
    L, g = Layer(q, fmt, M + N + K, M, N, K, r), Guarded()
    u, dx = L.backward(g)
    if r:
        L.check_u(u)
    L.check_dx(dx, u)
    u2, dx2 = L.backward(g)                                                 # deterministic
    assert torch.equal(dx2, dx) and (u is None or torch.equal(u2, u))
    dx3 = g(L.dt, M, K)                                                     # for a given u, without a workspace
    q.int8_gemm_bwd_dx(L.w, L.dy, u, L.A, dx=dx3)
    L.check_dx(dx3, u)
    g.check()


@pytest.mark.parametrize("per,fmt,M,N,r", int8_sizes.U)
def test_u_of_few_tokens(q, per, fmt, M, N, r):
    say(f"[int8 u, {per} tokens each] {fmt} M={M} N={N} r={r}")
    L, g = Layer(q, fmt, M + N, M, N, 64, r), Guarded()
    u, dx = L.backward(g)
    L.check_u(u)
    L.check_dx(dx, u)
    g.check()


# ranks per lane 1, 2 and 4, whole or not; dy's columns in fours or not; split sums (M > 512) and not
GRADS = [(fmt, r, M, N, K) for fmt, M in (("f16", 2050), ("bf16", 1030), ("f16", 200))
         for r, N, K in ((5, 136, 256), (32, 137, 64), (33, 260, 128), (34, 134, 192), (63, 129, 320), (64, 72, 64),
                         (66, 301, 64), (100, 200, 192), (127, 128, 128), (128, 515, 64))]


@pytest.mark.parametrize("fmt,r,M,N,K", GRADS)
def test_gradient_ranks_and_splits(q, fmt, r, M, N, K):
    say(f"[int8 grads] {fmt} r={r} M={M} N={N} K={K}")
    dt = TYPES[fmt][0]
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(r + M + N)
    n = lambda std, *s: (torch.randn(s, generator=gen, device="cuda:0") * std).to(dt)
    x, t, u, dy = n(1.0, M, K), n(0.5, M, r), n(0.1, M, r), n(0.5, M, N)
    g = Guarded()
    dA, dB = g(F32, K, r), g(F32, r, N)
    ck = q.int8_quantize(x)
    q.lora_grads_batch_int8([(ck, t, u, dy)], dA=[dA], dB=[dB])
    c, s = codes_of(x)
    x16 = (c.to(F64) * s.to(F64)[:, None]).to(F32).to(dt).to(F64)
    for name, got, a, b in (("dA", dA, x16, u.to(F64)), ("dB", dB, t.to(F64), dy.to(F64))):
        close(got, mm(a.t(), b), (M + 8) * 2.0 ** -23 * mm(a.abs().t(), b.abs()) + 2.0 ** -149, name)
    g.check()


# ---- split products in graphs and on several streams: (fmt, forward M, N, K, r), (dx M, N, K, r)
SPLIT_FWD, SPLIT_DX = ("f16", 708, 1104, 6080, 24), ("f16", 440, 2864, 2624, 40)


def _split_step(q, F, D, ws, out, ck):
    q.int8_linear_fwd(F.w, F.x, F.A, F.B, F.alpha, y=out["y"], t=out["t"], keep=ck, ws=ws)
    q.int8_linear_bwd_dx(D.w, D.A, D.B, D.alpha, D.dy, u=out["u"], dx=out["dx"], ws=ws)
    q.lora_grads_batch_int8([(ck, out["t"], out["t"], F.dy)], dA=[out["dA"]], dB=[out["dB"]], ws=ws)


def _outputs(q, F, D):
    e = lambda dt, *s: torch.empty(s, dtype=dt, device="cuda:0")
    out = dict(y=e(F.dt, F.M, F.N), t=e(F.dt, F.M, F.r), u=e(D.dt, D.M, D.r), dx=e(D.dt, D.M, D.K), dA=e(F32, F.K, F.r),
               dB=e(F32, F.r, F.N))
    return out, q.Int8Tensor.empty(F.M, F.K, dtype=F.dt)


def test_split_products_in_graphs(q):
    """Two graphs of split products that share their workspace, replayed in turn with eager work between; what the
    workspace holds before a replay (tags of earlier launches, or anything else) does not matter."""
    say("[int8 graph] split products")
    F, D = Layer(q, SPLIT_FWD[0], 1, *SPLIT_FWD[1:]), Layer(q, SPLIT_DX[0], 2, *SPLIT_DX[1:])
    out, ck = _outputs(q, F, D)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda:0")
    assert q.lib.qlora_int8_fwd_workspace(*SPLIT_FWD[1:]) <= ws.numel()
    assert q.lib.qlora_int8_linear_bwd_dx_workspace(*SPLIT_DX[1:]) <= ws.numel()

    def snap():
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in out.items()}

    _split_step(q, F, D, ws, out, ck)
    eager = snap()
    F.check_y(out["y"], out["t"], ck)
    D.check_dx(out["dx"], out["u"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _split_step(q, F, D, ws, out, ck)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _split_step(q, F, D, ws, out, ck)
        graphs.append(g)
    for rep in range(6):
        for v in out.values():
            v.fill_(float("nan"))
        ck.codes.zero_()
        if rep % 3 == 0:
            ws.fill_(0xA5)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        got = snap()
        for k in out:
            assert torch.equal(got[k], eager[k]), f"replay {rep}: {k} differs"
        _split_step(q, F, D, ws, out, ck)


def test_split_products_on_two_streams(q):
    """The same layers on two streams at once, each with its own workspace: both are what they are alone."""
    say("[int8] split products on two streams")
    F, D = Layer(q, SPLIT_FWD[0], 3, *SPLIT_FWD[1:]), Layer(q, SPLIT_DX[0], 4, *SPLIT_DX[1:])
    sides = []
    for _ in range(2):
        out, ck = _outputs(q, F, D)
        sides.append((torch.cuda.Stream(), out, ck, torch.empty(1 << 25, dtype=torch.uint8, device="cuda:0")))
    out, ck = _outputs(q, F, D)
    _split_step(q, F, D, torch.empty(1 << 25, dtype=torch.uint8, device="cuda:0"), out, ck)
    torch.cuda.synchronize()
    for _ in range(4):
        for s, o, c, ws in sides:
            with torch.cuda.stream(s):
                _split_step(q, F, D, ws, o, c)
    torch.cuda.synchronize()
    for _, o, c, _ in sides:
        for k in out:
            assert torch.equal(o[k], out[k]), k
        assert torch.equal(c.codes, ck.codes)


# ---- infinities and NaN stay in their rows, in every kernel (the first size of each with a LoRA branch)
def _firsts(cases, key):
    seen = {}
    for c in cases:
        if c[-1]:
            seen.setdefault(key(c), c)
    return list(seen.values())


FWD_KINDS = [c[2:] for c in _firsts(int8_sizes.FWD, lambda c: (c[0], c[1] > 1, (c[4] | c[6]) % 8 == 0))]
FWD_KINDS += [c[2:] for c in _firsts(int8_sizes.DECODE, lambda c: c[0])]
DX_KINDS = [c[2:] for c in _firsts(int8_sizes.DX, lambda c: (c[0], c[1] > 1, c[4] % 8 == 0))]


@pytest.mark.parametrize("fmt,M,N,K,r", FWD_KINDS)
def test_forward_of_rows_that_are_not_finite(q, fmt, M, N, K, r):
    say(f"[int8 fwd, not finite] {fmt} M={M} N={N} K={K} r={r}")
    L, inf, nan = Layer(q, fmt, 50 + M, M, N, K, r), float("inf"), float("nan")
    y0, t0 = q.int8_linear_fwd(L.w, L.x, L.A, L.B, L.alpha)
    bad = sorted({0, M // 3, M - 1})
    rows = [m for m in range(M) if m not in bad]
    L.x[bad[0], 1], L.x[bad[len(bad) // 2], K - 1], L.x[bad[-1], K // 2] = inf, nan, -inf
    w = L.w16.clone()
    w[N // 2, 3] = nan                                             # and an output
    cols = [n for n in range(N) if n != N // 2]
    y, t = q.int8_linear_fwd(q.int8_quantize(w), L.x, L.A, L.B, L.alpha)
    assert torch.isnan(y[bad]).all() and torch.isnan(y[:, N // 2]).all()
    assert torch.equal(y[rows][:, cols], y0[rows][:, cols]) and torch.equal(t[rows], t0[rows])


@pytest.mark.parametrize("fmt,M,N,K,r", DX_KINDS)
def test_input_gradient_of_rows_that_are_not_finite(q, fmt, M, N, K, r):
    say(f"[int8 dx, not finite] {fmt} M={M} N={N} K={K} r={r}")
    L = Layer(q, fmt, 60 + M, M, N, K, r)
    u0, dx0 = q.int8_linear_bwd_dx(L.w, L.A, L.B, L.alpha, L.dy)
    bad = sorted({0, M // 3, M - 1})
    rows = [m for m in range(M) if m not in bad]
    for m, n, v in zip(bad, (0, N // 2, N - 1), (float("nan"), float("inf"), float("-inf"))):
        L.dy[m, n] = v
    u, dx = q.int8_linear_bwd_dx(L.w, L.A, L.B, L.alpha, L.dy)
    assert not torch.isfinite(dx[bad]).any() and not torch.isfinite(u[bad]).any()
    assert torch.equal(dx[rows], dx0[rows]) and torch.equal(u[rows], u0[rows])


@pytest.mark.parametrize("fmt,r,M,N,K", GRADS[::3])
def test_gradients_of_rows_that_are_not_finite(q, fmt, r, M, N, K):
    """A token that is not finite has a checkpoint row of scale NaN: it reaches every column of its layer's dA and
    none of dB.  A value of dy that is not finite stays in its column."""
    say(f"[int8 grads, not finite] {fmt} r={r} M={M} N={N} K={K}")
    dt = TYPES[fmt][0]
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(r + M)
    n = lambda std, *s: (torch.randn(s, generator=gen, device="cuda:0") * std).to(dt)
    x, t, u, dy = n(1.0, M, K), n(0.5, M, r), n(0.1, M, r), n(0.5, M, N)
    (dA0,), (dB0,) = q.lora_grads_batch_int8([(q.int8_quantize(x), t, u, dy)])
    x[M - 1, 5] = float("inf")
    dy[M // 2, N - 1] = float("nan")
    (dA,), (dB,) = q.lora_grads_batch_int8([(q.int8_quantize(x), t, u, dy)])
    assert torch.isnan(dA).all() and torch.isnan(dB[:, N - 1]).all()
    assert torch.equal(dB[:, :N - 1], dB0[:, :N - 1]) and torch.isfinite(dA0).all()
