"""Refusals and size queries of the fp8 entry points, without a GPU: every argument error is reported before anything
is launched (fake, never-dereferenced device pointers are used)."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -4
FAKE = 0x10000
BIG = 1 << 60


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


def _st(q, rows=64, cols=128, codes=FAKE, scale=FAKE, dtype=0, block_rows=128):
    return q.Fp8State(codes, scale, rows, cols, dtype, block_rows)


def _ref(s):
    return None if s is None else ctypes.byref(s)


# what is wrong with a state, and the status it gives
BAD_STATES = [(None, INVALID), (dict(codes=0), INVALID), (dict(scale=0), INVALID), (dict(dtype=2), INVALID),
              (dict(dtype=7), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(block_rows=0), INVALID),
              (dict(block_rows=64), INVALID), (dict(cols=100), SHAPE), (dict(rows=1 << 31), SHAPE),
              (dict(cols=1 << 22), SHAPE), (dict(codes=FAKE + 8), MISALIGNED), (dict(scale=FAKE + 4), MISALIGNED)]


@pytest.mark.parametrize("bad,status", BAD_STATES)
def test_states(q, bad, status):
    st = None if bad is None else _st(q, **bad)
    rows = None if bad is None else _st(q, **{"block_rows": 1, **bad})
    good, x = _st(q), _st(q, rows=4, block_rows=1)
    assert q.lib.qlora_fp8_quantize(FAKE, _ref(st), None) == status
    assert q.lib.qlora_fp8_dequantize(_ref(st), FAKE, None) == status
    assert q.lib.qlora_fp8_quantize(FAKE, _ref(rows), None) == status
    assert q.lib.qlora_fp8_linear_fwd(_ref(st), FAKE, 4, FAKE, FAKE, 8, 1.0, None, FAKE, None, FAKE, BIG, None) == status
    assert q.lib.qlora_fp8_gemm_fwd(_ref(st), _ref(x), None, None, 0, FAKE, None) == status
    assert q.lib.qlora_fp8_gemm_fwd(_ref(good), _ref(rows), None, None, 0, FAKE, None) == status
    assert q.lib.qlora_fp8_linear_bwd_dx(_ref(st), 4, FAKE, FAKE, 8, 1.0, None, FAKE, FAKE, FAKE, FAKE, BIG, None) == status


def test_quantize_arguments(q):
    for br in (1, 128):
        st = _st(q, block_rows=br)
        for f in (lambda p, s: q.lib.qlora_fp8_quantize(p, ctypes.byref(s), None),
                  lambda p, s: q.lib.qlora_fp8_dequantize(ctypes.byref(s), p, None)):
            assert f(None, st) == INVALID
            assert f(FAKE + 2, st) == MISALIGNED
            assert f(None, _st(q, rows=0, codes=0, scale=0, block_rows=br)) == OK             # nothing to do


def test_scale_bytes(q):
    f = q.lib.qlora_fp8_scale_bytes
    for rows, cols in ((1, 64), (128, 128), (129, 192), (11008, 4096), (7, 28672)):
        for br in (1, 128):
            a, b = q.Fp8Tensor.scale_shape(rows, cols, br)
            assert f(rows, cols, br) == a * b and b % 4 == 0
    assert f(300, 320, 128) == 3 * 4 and f(300, 320, 1) == 3 * 300 and f(301, 320, 1) == 3 * 304
    assert f(-1, 64, 1) == f(4, 0, 1) == f(4, 64, 2) == 0


def test_linear_fwd_arguments(q):
    f = q.lib.qlora_fp8_linear_fwd
    w = _st(q)
    need = int(q.lib.qlora_fp8_fwd_workspace(4, 64, 128, 8))
    assert need > 4 * 128
    d = lambda p=0.1: ctypes.byref(q.DropoutState(1, 2, p))

    def call(x=FAKE, M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, drop=None, y=FAKE, t=None, ws=FAKE, n=need, w=w):
        return f(ctypes.byref(w), x, M, A, B, r, alpha, drop, y, t, ws, n, None)

    assert call(M=0, x=None, y=None) == OK and call(M=0, drop=d()) == OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(r=-1), dict(r=129), dict(alpha=float("nan")), dict(x=None),
               dict(y=None), dict(A=None), dict(B=None), dict(r=0), dict(r=0, A=None), dict(r=0, A=None, B=None, t=FAKE),
               dict(r=0, A=None, B=None, drop=d()), dict(drop=d(1.0)), dict(drop=d(-0.5)), dict(drop=d(float("nan"))),
               dict(w=_st(q, block_rows=1))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(A=FAKE + 2), dict(B=FAKE + 2), dict(y=FAKE + 2), dict(t=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(**kw) == MISALIGNED, kw
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(w=_st(q, rows=1 << 22), n=BIG) == SHAPE and call(M=(1 << 31) - 1, n=BIG) == SHAPE


def test_gemm_fwd_arguments(q):
    f = q.lib.qlora_fp8_gemm_fwd

    def call(x=None, t=FAKE, B=FAKE, r=8, y=FAKE, w=None):
        w, x = w or _st(q), x or _st(q, rows=4, block_rows=1)
        return f(ctypes.byref(w), ctypes.byref(x), t, B, r, y, None)

    assert call(x=_st(q, rows=0, codes=0, scale=0, block_rows=1), y=None) == OK
    for kw in (dict(x=_st(q, rows=4, cols=64, block_rows=1)), dict(x=_st(q, rows=4, dtype=1, block_rows=1)),
               dict(x=_st(q, rows=4)), dict(w=_st(q, block_rows=1)), dict(r=-1), dict(r=129), dict(y=None), dict(t=None),
               dict(B=None), dict(r=0), dict(r=0, t=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(t=FAKE + 2), dict(B=FAKE + 2), dict(y=FAKE + 2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(w=_st(q, rows=1 << 22)) == SHAPE


def test_bwd_dx_arguments(q):
    f = q.lib.qlora_fp8_linear_bwd_dx
    w = _st(q)
    need = int(q.lib.qlora_fp8_linear_bwd_dx_workspace(4, 64, 128, 8))
    assert need > 0
    big = q.lib.qlora_fp8_linear_bwd_dx_workspace
    assert big(300, 4000, 128, 0) < big(300, 4000, 128, 8) < big(300, 4000, 128, 64)      # (sums of u's splits)
    d = lambda p=0.1: ctypes.byref(q.DropoutState(1, 2, p))

    def call(M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, drop=None, dy=FAKE, u=FAKE, dx=FAKE, ws=FAKE, n=need, w=w):
        return f(ctypes.byref(w), M, A, B, r, alpha, drop, dy, u, dx, ws, n, None)

    assert call(M=0, dy=None) == OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(r=-1), dict(r=129), dict(dy=None), dict(dx=None), dict(A=None), dict(B=None),
               dict(u=None), dict(r=0), dict(r=0, A=None), dict(alpha=float("inf")), dict(r=0, A=None, B=None, u=None, drop=d()),
               dict(drop=d(1.0)), dict(w=_st(q, block_rows=1))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(A=FAKE + 2), dict(B=FAKE + 2), dict(dy=FAKE + 2), dict(u=FAKE + 2), dict(dx=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(**kw) == MISALIGNED, kw
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(w=_st(q, rows=1 << 22), n=BIG) == SHAPE and call(M=(1 << 31) - 1, n=BIG) == SHAPE


def test_workspace_queries_of_bad_sizes(q):
    for f in (q.lib.qlora_fp8_fwd_workspace, q.lib.qlora_fp8_linear_bwd_dx_workspace):
        for a in ((0, 64, 64, 8), (-1, 64, 64, 8), (4, 0, 64, 8), (4, 64, 0, 8), (4, 64, 100, 8), (4, 64, 64, 129),
                  (4, 64, 64, -1), (4, 1 << 22, 64, 8), (4, 64, 1 << 22, 8), (1 << 31, 64, 64, 8)):
            assert f(*a) == 0, a
        assert f(100, 200, 320, 0) > 0


def test_the_binding_refuses(q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.Fp8Tensor.empty(4, 64, device="cpu")
    with pytest.raises(ValueError):
        q.fp8_quantize(x)
    with pytest.raises(ValueError):
        q.Fp8Tensor.empty(4, 64, block_rows=2)
    with pytest.raises(TypeError):
        q.Fp8Tensor.empty(4, 64, dtype=torch.float32)
    with pytest.raises(TypeError):
        q.Fp8Tensor(x, torch.zeros((1, 4), dtype=torch.uint8))
