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
