"""Sizes past what the int8 kernels' offsets hold are refused, without a GPU: before anything is launched
(fake, never-dereferenced device pointers are used)."""
import ctypes

import pytest

SHAPE = -2
FAKE = 0x10000
BIG = 1 << 60


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_15_amd import qlora
    return qlora


def _st(q, rows, cols=64, dtype=0):
    return ctypes.byref(q.Int8State(FAKE, FAKE, rows, cols, dtype))


def _fwd(q, w, M=4, r=8):
    ab = FAKE if r else None
    return q.lib.qlora_int8_linear_fwd(w, FAKE, M, ab, ab, r, 1.0, FAKE, None, None, FAKE, BIG, None)


def _dx(q, w, M=4, r=8):
    ab = FAKE if r else None
    return q.lib.qlora_int8_linear_bwd_dx(w, M, ab, ab, r, 1.0, FAKE, ab, FAKE, FAKE, BIG, None)


def _gemm_dx(q, w, M=4, r=8):
    ab = FAKE if r else None
    return q.lib.qlora_int8_gemm_bwd_dx(w, FAKE, M, ab, ab, r, FAKE, None)


@pytest.mark.parametrize("r", [0, 8])
@pytest.mark.parametrize("N", [1 << 29, (1 << 29) + 1, 1 << 30, (1 << 31) - 1])
def test_input_gradient_of_too_many_outputs(q, N, r):
    """The input gradient reads the weight's scales at 31-bit byte offsets: 2^29 of them do not fit (they would
    read as zero, or as another row's)."""
    assert _dx(q, _st(q, N), r=r) == SHAPE
    assert _gemm_dx(q, _st(q, N), r=r) == SHAPE


LAST = (1 << 31) - 16384          # the largest row count that is accepted


@pytest.mark.parametrize("rows", [LAST + 1, (1 << 31) - 1])
@pytest.mark.parametrize("r", [0, 8])
def test_row_counts_that_overflow_an_index(q, rows, r):
    """Tiles and chunks of rows are counted in 32 bits past their last row: the forward's output columns, the
    decode kernel's row tiles, and every kernel's tokens, up to some 8000 rows further."""
    small = _st(q, 64)
    ab = FAKE if r else None
    for M in (4, 40):                                        # decode and tiled
        assert _fwd(q, _st(q, rows), M, r) == SHAPE
        assert q.lib.qlora_int8_gemm_fwd(_st(q, rows), _st(q, M), ab, ab, r, FAKE, None) == SHAPE
    assert _fwd(q, small, rows, r) == SHAPE
    assert q.lib.qlora_int8_gemm_fwd(small, _st(q, rows), ab, ab, r, FAKE, None) == SHAPE
    assert _dx(q, small, rows, r) == SHAPE
    assert _gemm_dx(q, small, rows, r) == SHAPE


@pytest.mark.parametrize("M", [LAST + 1, (1 << 31) - 1])
def test_gradients_of_too_many_tokens(q, M):
    """The gradient kernel's last chunk of rows would end past 2^31."""
    one = (q.LoraGradsInt8 * 1)(q.LoraGradsInt8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, M, 64, 64))
    assert q.lib.qlora_lora_grads_batch_int8(one, 1, 8, 0, FAKE, BIG, None) == SHAPE


def test_the_largest_row_count_passes_the_checks(q):
    """LAST itself is not refused for its size: the next check, of the workspace, answers."""
    w = _st(q, LAST)
    assert q.lib.qlora_int8_linear_fwd(w, FAKE, 4, None, None, 0, 1.0, FAKE, None, None, FAKE, 16, None) == -4
    one = (q.LoraGradsInt8 * 1)(q.LoraGradsInt8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, LAST, 64, 64))
    assert q.lib.qlora_lora_grads_batch_int8(one, 1, 8, 0, FAKE, 16, None) == -4
