"""Refusals of the entry points with dropout, without a GPU: argument errors are reported before anything is launched
(fake, never-dereferenced device pointers are used), and the binding refuses what it can see itself."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -4
FAKE, BIG = 0x10000, 1 << 40


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


BAD_P = [-0.1, 1.0, 1.5, float("nan"), float("inf"), 65535.6 / 65536]


def drop(q, p=0.1):
    return q.DropoutState(1, 2, p)


def calls(q):
    """Each entry point as f(drop, **changes), with good arguments that it would launch with."""
    w4 = q.NF4State(FAKE, FAKE, FAKE, 64, 128, 0, 0)
    w8 = q.Int8State(FAKE, FAKE, 64, 128, 0)
    R = ctypes.byref

    def dx4(d, w=w4, M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, dy=FAKE, u=FAKE, dx=FAKE, ws=FAKE, n=BIG):
        return q.lib.qlora_linear_bwd_dx_dropout(R(w), M, A, B, r, alpha, d, dy, u, dx, ws, n, None)

    def dx8(d, w=w8, M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, dy=FAKE, u=FAKE, dx=FAKE, ws=FAKE, n=BIG):
        return q.lib.qlora_int8_linear_bwd_dx_dropout(R(w), M, A, B, r, alpha, d, dy, u, dx, ws, n, None)

    def st4(d, w=w4, M=4, A=FAKE, r=8, dy=FAKE, u=FAKE, dx=FAKE):
        return q.lib.qlora_fused_gemm_bwd_dx_dropout(R(w), dy, M, u, A, r, d, dx, None)

    def st8(d, w=w8, M=4, A=FAKE, r=8, dy=FAKE, u=FAKE, dx=FAKE):
        return q.lib.qlora_int8_gemm_bwd_dx_dropout(R(w), dy, M, u, A, r, d, dx, None)
    return dx4, dx8, st4, st8


def test_input_gradient_arguments(q):
    R = ctypes.byref
    for f in calls(q):
        assert f(None) == INVALID
        for p in BAD_P:
            assert f(R(drop(q, p))) == INVALID, p
        for p in (0.0, 0.1):
            d = R(drop(q, p))
            assert f(d, M=0) == OK
            for kw in (dict(M=-1), dict(r=-1), dict(r=129), dict(dy=None), dict(dx=None), dict(A=None), dict(u=None), dict(r=0)):
                assert f(d, **kw) == INVALID, kw
            for kw in (dict(A=FAKE + 2), dict(dy=FAKE + 2), dict(u=FAKE + 2), dict(dx=FAKE + 2)):
                assert f(d, **kw) == MISALIGNED, kw
    for f in calls(q)[:2]:
        d = R(drop(q))
        assert f(d, B=None) == INVALID and f(d, alpha=float("nan")) == INVALID
        assert f(d, ws=None) == WORKSPACE and f(d, n=16) == WORKSPACE and f(d, ws=FAKE + 8) == MISALIGNED
    for f in (calls(q)[0], calls(q)[2]):
        assert f(R(drop(q)), w=q.NF4State(FAKE, FAKE, FAKE, 64, 128, 0, 2)) == INVALID      # fp32


def test_batch_arguments(q):
    D = lambda *ps: (q.DropoutState * len(ps))(*[drop(q, p) for p in ps])
    prods = (q.LoraProd * 2)(*[q.LoraProd(FAKE, FAKE, FAKE, 4, 128)] * 2)
    layers = (q.LoraGrads * 2)(*[q.LoraGrads(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128)] * 2)

    def down(d, items=prods, n=2, r=8, alpha=1.0, dtype=0, ws=FAKE, nb=BIG):
        return q.lib.qlora_lora_down_batch_dropout(items, d, n, r, alpha, dtype, ws, nb, None)

    def grads(d, items=layers, n=2, r=8, dtype=0, ws=FAKE, nb=BIG):
        return q.lib.qlora_lora_grads_batch_dropout(items, d, n, r, dtype, ws, nb, None)

    for f in (down, grads):
        good = D(0.1, 0.5)
        assert f(None) == INVALID and f(None, n=0) == OK and f(good, n=0) == OK
        for p in BAD_P:
            assert f(D(0.1, p)) == INVALID and f(D(p, 0.0)) == INVALID
        for kw in (dict(n=-1), dict(r=0), dict(r=129), dict(dtype=2), dict(dtype=9), dict(items=None)):
            assert f(good, **kw) == INVALID, kw
        assert f(good, ws=None) == WORKSPACE and f(good, nb=16) == WORKSPACE and f(good, ws=FAKE + 8) == MISALIGNED
    assert down(D(0.1, 0.1), alpha=float("inf")) == INVALID
    assert down(D(0.1, 0.1), items=(q.LoraProd * 2)(*[q.LoraProd(FAKE, FAKE, FAKE, 4, 100)] * 2)) == SHAPE
    for C in (2 ** 31 - 64, 2 ** 31 - 1024):       # columns that the kernel could not count in 32 bits
        wide = (q.LoraProd * 2)(q.LoraProd(FAKE, FAKE, FAKE, 4, 128), q.LoraProd(FAKE, FAKE, FAKE, 4, C))
        assert down(D(0.0, 0.1), items=wide) == SHAPE
    for N, K in ((64, 2 ** 22), (2 ** 22, 128)):
        wide = (q.LoraGrads * 2)(q.LoraGrads(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128),
                                 q.LoraGrads(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, N, K))
        assert grads(D(0.0, 0.1), items=wide) == SHAPE


def test_the_class(q):
    for p in BAD_P:
        with pytest.raises(ValueError):
            q.Dropout(p)
    for kw in (dict(seed=-1), dict(seed=2 ** 64), dict(offset=-1), dict(offset=2 ** 64)):
        with pytest.raises(ValueError):
            q.Dropout(0.1, **kw)
    d = q.Dropout(0.05, 2 ** 64 - 1, 3).state()
    assert (d.seed, d.offset, d.p) == (2 ** 64 - 1, 3, 0.05)
    q.Dropout(65535 / 65536), q.Dropout(0.0)


def test_struct_layout(q):
    """As the header's structs are laid out on this ABI."""
    assert ctypes.sizeof(q.DropoutState) == 24 and ctypes.sizeof(q.Fp8State) == 40


@pytest.mark.parametrize("call", ["down", "grads", "fwd"])
def test_lists_of_another_length_and_fp32(q, call):
    x = torch.zeros((4, 64))
    if call == "fwd":
        w = q.NF4Weight(x, None, x, 64, 64, dtype=torch.float32)
        for f in (lambda: q.linear_fwd(w, x, x, x, 1.0, dropout=q.Dropout(0.1)),
                  lambda: q.linear_bwd(w, x, x, x, 1.0, x, dropout=q.Dropout(0.1))):
            with pytest.raises(TypeError):
                f()
        return
    with pytest.raises(ValueError):
        q._drops([q.Dropout(0.1)] * 2, 3)
