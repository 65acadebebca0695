"""The int8 layer at the ends of its documented ranges: the largest sums of codes, and sizes whose tiles come
close to 31-bit offsets or change kernels because of them.  Bounds as in test_gpu_int8.py."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
H = 2.0 ** -8


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def randn(g, *s, std=1.0):
    return (torch.randn(s, generator=g, device="cuda:0") * std).to(BF)


def codes(q, g, rows, cols):
    """Random codes and scales."""
    c = torch.empty((rows, cols), dtype=torch.int8, device="cuda:0")
    c.random_(-127, 128, generator=g)
    return q.Int8Tensor(c, torch.rand(rows, generator=g, device="cuda:0") * 2.0 ** -8 + 2.0 ** -9)


def values(w, rows):
    return (w.codes[rows].to(F64) * w.scale[rows].to(F64)[:, None]).to(F32).to(BF).to(F64)


def mm(a, b):
    return torch.mm(a.contiguous(), b.contiguous())


def close(got, want, tol, what):
    bad = ~((got.to(F64) - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("M,N", [(1, 72), (16, 40), (20, 72), (300, 1000), (1100, 72), (1100, 4100)])
def test_largest_sums(q, M, N):
    """The longest rows with every code at its end: sums of 127^2 K, and of 128^2 K for codes that a caller made,
    just below 2^31 (the scales powers of two, so y is one rounding of an exact value)."""
    say(f"[int8 largest sums] M={M} N={N}")
    K = 131072 - 64
    x = torch.ones((M, K), dtype=BF, device="cuda:0")
    x[1::2] = -1.0
    w = q.int8_quantize(torch.ones((N, K), dtype=BF, device="cuda:0"))
    y, _ = q.int8_linear_fwd(w, x)
    want = torch.full((M, N), float(K), dtype=F64, device="cuda:0")
    want[1::2] *= -1.0
    close(y, want, want.abs() * (H + 2.0 ** -20), "127")
    full = lambda rows: q.Int8Tensor(torch.full((rows, K), -128, dtype=torch.int8, device="cuda:0"),
                                     torch.full((rows,), 2.0 ** -10, device="cuda:0"))
    y = q.int8_gemm_fwd(full(N), full(M))
    assert torch.equal(y, torch.full((M, N), 128.0 * 128.0 * K * 2.0 ** -20, device="cuda:0").to(BF))


@pytest.mark.parametrize("M,N,K,r", [(20, (1 << 22) - 8, 64, 8), (20, (1 << 22) + 8, 64, 0), (70, (1 << 22) + 3, 64, 8),
                                     (2063, (1 << 22) - 8, 4352, 0)])
def test_input_gradient_of_long_reductions(q, M, N, K, r):
    """dy's rows up to and past the length that direct loads address; all but some columns of dy are zero."""
    say(f"[int8 dx, long] M={M} N={N} K={K} r={r}")
    g = gen(N + M)
    w = codes(q, g, N, K)
    cols = torch.unique(torch.cat([torch.randint(0, N, (50,), generator=g, device="cuda:0"),
                                   torch.tensor([0, 63, 64, N // 2, N - 64, N - 9, N - 2, N - 1], device="cuda:0")]))
    dy = torch.zeros((M, N), dtype=BF, device="cuda:0")
    dy[:, cols] = randn(g, M, len(cols))
    A, B = (randn(g, K, r, std=r ** -0.5), randn(g, r, N, std=0.05)) if r else (None, None)
    u, dx = q.int8_linear_bwd_dx(w, A, B, 16.0, dy)
    d, wv = dy[:, cols].to(F64), values(w, cols)
    want, mag, n = mm(d, wv), mm(d.abs(), wv.abs()), len(cols) + r + 8   # (zeros add nothing to a sum's error)
    if r:
        b = B[:, cols].to(F64)
        wu = 16.0 / r * mm(d, b.t())
        close(u, wu, H * wu.abs() + n * 2.0 ** -23 * 16.0 / r * mm(d.abs(), b.abs().t()) * (1 + H), "u")
        want, mag = want + mm(u.to(F64), A.to(F64).t()), mag + mm(u.to(F64).abs(), A.to(F64).abs().t())
    close(dx, want, (n * 2.0 ** -23 * mag + H * want.abs()) * (1 + 2 * H), "dx")


@pytest.mark.parametrize("M,N,r", [(40, 72, 8), (300, 72, 0), (300, 73, 12)])
def test_input_gradient_of_wide_layers(q, M, N, r):
    say(f"[int8 dx, wide] M={M} N={N} r={r}")
    K = (1 << 22) - 64
    g = gen(M + N)
    w, dy = codes(q, g, N, K), randn(g, M, N, std=0.5)
    A, B = (randn(g, K, r, std=r ** -0.5), randn(g, r, N, std=0.05)) if r else (None, None)
    u, dx = q.int8_linear_bwd_dx(w, A, B, 16.0, dy)
    rows = torch.arange(N, device="cuda:0")
    wv = values(w, rows)
    for part in (slice(0, 4096), slice(K // 2, K // 2 + 4096), slice(K - 4096, K)):
        want, mag = mm(dy.to(F64), wv[:, part]), mm(dy.to(F64).abs(), wv[:, part].abs())
        if r:
            a = A[part].to(F64).t()
            want, mag = want + mm(u.to(F64), a), mag + mm(u.to(F64).abs(), a.abs())
        close(dx[:, part], want, ((N + r + 8) * 2.0 ** -23 * mag + H * want.abs()) * (1 + 2 * H), f"dx {part}")


@pytest.mark.parametrize("M", [5, 16, 20])
def test_forward_with_a_large_b(q, M):
    """B of over 2^31 bytes: decode sizes leave the one-launch kernel, and t, B and y go by the element."""
    say(f"[int8 fwd, large B] M={M}")
    N, K, r = (1 << 23) + 8, 64, 128
    g = gen(M)
    w, x, A = codes(q, g, N, K), randn(g, M, K), randn(g, K, r, std=r ** -0.5)
    B = torch.empty((r, N), dtype=BF, device="cuda:0")
    for j in range(r):
        B[j] = randn(g, N, std=0.05)
    keep = q.Int8Tensor.empty(M, K)
    y, t = q.int8_linear_fwd(w, x, A, B, 64.0, keep=keep)
    tf = t.to(F64)
    for part in (slice(0, 4096), slice(N // 2, N // 2 + 4096), slice(N - 4096, N)):
        base = mm(keep.codes.to(F64) * keep.scale.to(F64)[:, None], (w.codes[part].to(F64) * w.scale[part].to(F64)[:, None]).t())
        b = B[:, part].to(F64)
        want, mag = base + mm(tf, b), base.abs() + mm(tf.abs(), b.abs())
        close(y[:, part], want, ((r + 8) * 2.0 ** -23 * mag + H * want.abs()) * (1 + 2 * H), f"y {part}")


def test_gradients_at_the_widest(q):
    """K and N of 2^22: the fewest rows per workgroup."""
    say("[int8 grads, widest]")
    M, D, r = 600, 1 << 22, 8
    g = gen(3)
    ck, dy = codes(q, g, M, D), torch.empty((M, D), dtype=BF, device="cuda:0")
    for m in range(M):
        dy[m] = randn(g, D, std=0.5)
    t, u = randn(g, M, r), randn(g, M, r, std=0.1)
    (dA,), (dB,) = q.lora_grads_batch_int8([(ck, t, u, dy)])
    rows = torch.arange(M, device="cuda:0")
    for part in (slice(0, 4096), slice(D // 2, D // 2 + 4096), slice(D - 4096, D)):
        x16 = (ck.codes[:, part].to(F64) * ck.scale.to(F64)[rows, None]).to(F32).to(BF).to(F64)
        for got, a, b, what in ((dA[part], x16, u.to(F64), "dA"), (dB[:, part], t.to(F64), dy[:, part].to(F64), "dB")):
            close(got, mm(a.t(), b), (M + 8) * 2.0 ** -23 * mm(a.abs().t(), b.abs()), f"{what} {part}")
