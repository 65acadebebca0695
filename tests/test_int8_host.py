"""Refusals and size queries of the int8 entry points, without a GPU: every argument error is reported
before anything is launched (fake, never-dereferenced device pointers are used)."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -4
FAKE = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


def _st(q, rows=64, cols=128, codes=FAKE, scale=FAKE, dtype=0):
    return q.Int8State(codes, scale, rows, cols, dtype)


def _ref(s):
    return None if s is None else ctypes.byref(s)


# what is wrong with a state, and the status it gives
BAD_STATES = [(None, INVALID), (dict(codes=0), INVALID), (dict(scale=0), INVALID), (dict(dtype=2), INVALID),
              (dict(dtype=7), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=100), SHAPE),
              (dict(rows=1 << 31), SHAPE), (dict(cols=1 << 31), SHAPE), (dict(codes=FAKE + 8), MISALIGNED),
              (dict(scale=FAKE + 4), MISALIGNED)]


@pytest.mark.parametrize("bad,status", BAD_STATES)
def test_states(q, bad, status):
    st = None if bad is None else _st(q, **bad)
    good = _st(q)
    assert q.lib.qlora_int8_quantize(FAKE, _ref(st), None) == status
    assert q.lib.qlora_int8_dequantize(_ref(st), FAKE, None) == status
    assert q.lib.qlora_int8_linear_fwd(_ref(st), FAKE, 4, FAKE, FAKE, 8, 1.0, FAKE, None, None, FAKE, BIG, None) == status
    assert q.lib.qlora_int8_gemm_fwd(_ref(st), _ref(good), None, None, 0, FAKE, None) == status
    assert q.lib.qlora_int8_gemm_fwd(_ref(good), _ref(st), None, None, 0, FAKE, None) == status
    assert q.lib.qlora_int8_linear_bwd_dx(_ref(st), 4, FAKE, FAKE, 8, 1.0, FAKE, FAKE, FAKE, FAKE, BIG, None) == status
    assert q.lib.qlora_int8_gemm_bwd_dx(_ref(st), FAKE, 4, FAKE, FAKE, 8, FAKE, None) == status


def test_quantize_arguments(q):
    st = _st(q)
    for f in (lambda p, s: q.lib.qlora_int8_quantize(p, ctypes.byref(s), None),
              lambda p, s: q.lib.qlora_int8_dequantize(ctypes.byref(s), p, None)):
        assert f(None, st) == INVALID
        assert f(FAKE + 2, st) == MISALIGNED
        assert f(None, _st(q, rows=0, codes=0, scale=0)) == OK             # nothing to do


def test_linear_fwd_arguments(q):
    f = q.lib.qlora_int8_linear_fwd
    w = _st(q)
    need = int(q.lib.qlora_int8_fwd_workspace(4, 64, 128, 8))
    assert need > 4 * 128

    def call(x=FAKE, M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, y=FAKE, t=None, keep=None, ws=FAKE, n=need, w=w):
        return f(ctypes.byref(w), x, M, A, B, r, alpha, y, t, _ref(keep), ws, n, None)

    assert call(M=0, x=None, y=None) == OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(r=-1), dict(r=129), dict(alpha=float("nan")), dict(x=None),
               dict(y=None), dict(A=None), dict(B=None), dict(r=0), dict(r=0, A=None), dict(r=0, A=None, B=None, t=FAKE),
               dict(keep=_st(q, rows=5)), dict(keep=_st(q, rows=4, cols=64)), dict(keep=_st(q, rows=4, dtype=1)),
               dict(keep=_st(q, rows=4, codes=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(A=FAKE + 2), dict(B=FAKE + 2), dict(y=FAKE + 2), dict(t=FAKE + 2),
               dict(ws=FAKE + 8)):
        assert call(**kw) == MISALIGNED, kw
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(w=_st(q, cols=1 << 17), n=BIG) == SHAPE


def test_gemm_fwd_arguments(q):
    f = q.lib.qlora_int8_gemm_fwd

    def call(x=None, t=FAKE, B=FAKE, r=8, y=FAKE, w=None):
        w, x = w or _st(q), x or _st(q, rows=4)
        return f(ctypes.byref(w), ctypes.byref(x), t, B, r, y, None)

    assert call(x=_st(q, rows=0, codes=0, scale=0), y=None) == OK
    for kw in (dict(x=_st(q, rows=4, cols=64)), dict(x=_st(q, rows=4, dtype=1)), dict(r=-1), dict(r=129),
               dict(y=None), dict(t=None), dict(B=None), dict(r=0), dict(r=0, t=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(t=FAKE + 2), dict(B=FAKE + 2), dict(y=FAKE + 2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(w=_st(q, cols=1 << 17), x=_st(q, rows=4, cols=1 << 17)) == SHAPE


def test_bwd_dx_arguments(q):
    f, g = q.lib.qlora_int8_linear_bwd_dx, q.lib.qlora_int8_gemm_bwd_dx
    w = _st(q)
    need = int(q.lib.qlora_int8_linear_bwd_dx_workspace(4, 64, 128, 8))
    assert need > 0 and int(q.lib.qlora_int8_linear_bwd_dx_workspace(4, 64, 128, 0)) < need

    def layer(M=4, A=FAKE, B=FAKE, r=8, alpha=1.0, dy=FAKE, u=FAKE, dx=FAKE, ws=FAKE, n=need):
        return f(ctypes.byref(w), M, A, B, r, alpha, dy, u, dx, ws, n, None)

    def stage(M=4, dy=FAKE, u=FAKE, A=FAKE, r=8, dx=FAKE):
        return g(ctypes.byref(w), dy, M, u, A, r, dx, None)

    assert layer(M=0, dy=None) == OK and stage(M=0, dy=None) == OK
    for kw in (dict(M=-1), dict(r=-1), dict(r=129), dict(dy=None), dict(dx=None), dict(A=None), dict(u=None), dict(r=0),
               dict(r=0, A=None)):
        assert layer(**kw) == INVALID and stage(**kw) == INVALID, kw
    assert layer(B=None) == INVALID and layer(alpha=float("inf")) == INVALID
    for kw in (dict(A=FAKE + 2), dict(dy=FAKE + 2), dict(u=FAKE + 2), dict(dx=FAKE + 2)):
        assert layer(**kw) == MISALIGNED and stage(**kw) == MISALIGNED, kw
    assert layer(B=FAKE + 2) == MISALIGNED and layer(ws=FAKE + 8) == MISALIGNED
    assert layer(ws=None) == WORKSPACE and layer(n=need - 1) == WORKSPACE


def test_grads_arguments(q):
    f = q.lib.qlora_lora_grads_batch_int8

    def rec(x=FAKE, sc=FAKE, t=FAKE, u=FAKE, dy=FAKE, dA=FAKE, dB=FAKE, M=70, N=64, K=128):
        return q.LoraGradsInt8(x, sc, t, u, dy, dA, dB, M, N, K)

    def call(*recs, count=None, r=8, dtype=0, ws=FAKE, n=BIG):
        a = (q.LoraGradsInt8 * max(len(recs), 1))(*recs)
        return f(a, len(recs) if count is None else count, r, dtype, ws, n, None)

    assert call(count=0) == OK and f(None, 0, 8, 0, None, 0, None) == OK
    assert f(None, 1, 8, 0, FAKE, BIG, None) == INVALID
    for kw in (dict(count=-1), dict(r=0), dict(r=129), dict(dtype=2)):
        assert call(rec(), **kw) == INVALID, kw
    for kw in (dict(x=None), dict(sc=None), dict(t=None), dict(u=None), dict(dy=None), dict(dA=None), dict(dB=None),
               dict(M=-1), dict(N=0), dict(K=0)):
        assert call(rec(), rec(**kw)) == INVALID, kw                       # the second entry is checked too
    assert call(rec(), rec(K=100)) == SHAPE
    for k in ("x", "sc", "t", "u", "dy", "dA", "dB"):
        assert call(rec(), rec(**{k: FAKE + 8 if k not in ("dA", "dB") else FAKE + 4})) == MISALIGNED, k
    one = (q.LoraGradsInt8 * 1)(rec())
    need = int(q.lib.qlora_lora_grads_batch_int8_workspace(one, 1, 8))
    if need:
        assert call(rec(), ws=None) == WORKSPACE and call(rec(), n=need - 1) == WORKSPACE
        assert call(rec(), ws=FAKE + 8) == MISALIGNED


def test_sizes_past_the_offsets_of_a_tile(q):
    """Refused before anything is launched: rows whose tiles pass 31-bit offsets."""
    w = _st(q, cols=1 << 22)
    assert q.lib.qlora_int8_linear_bwd_dx(ctypes.byref(w), 4, FAKE, FAKE, 8, 1.0, FAKE, FAKE, FAKE, FAKE, BIG,
                                          None) == SHAPE
    assert q.lib.qlora_int8_gemm_bwd_dx(ctypes.byref(w), FAKE, 4, FAKE, FAKE, 8, FAKE, None) == SHAPE
    for K, N in (((1 << 22) + 64, 64), (128, (1 << 22) + 1)):
        one = (q.LoraGradsInt8 * 1)(q.LoraGradsInt8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 70, N, K))
        assert q.lib.qlora_lora_grads_batch_int8(one, 1, 8, 0, FAKE, BIG, None) == SHAPE


def test_workspace_queries_of_bad_sizes(q):
    for a in ((0, 64, 64, 8), (4, 64, 100, 8), (-1, 64, 64, 8), (4, 0, 64, 8), (4, 64, 64, 129), (4, 64, 64, -1)):
        assert int(q.lib.qlora_int8_fwd_workspace(*a)) == 0
    assert int(q.lib.qlora_lora_grads_batch_int8_workspace(None, 1, 8)) == 0


def test_python_refusals(q):
    """The binding's own checks, before any pointer is taken."""
    codes, scale = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(TypeError):
        q.Int8Tensor(codes, scale, torch.float32)
    with pytest.raises(TypeError):
        q.Int8Tensor(codes.float(), scale)
    with pytest.raises(ValueError):
        q.Int8Tensor(codes, scale)                                         # not on a device
    with pytest.raises(ValueError):
        q.Int8Tensor(codes.view(-1), scale)
