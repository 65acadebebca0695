"""The documented limit of the fp8 codes: a tensor that could not be restored is not quantized either (no GPU: nothing
is launched, and the pointers are never dereferenced)."""
import ctypes

import pytest

SHAPE, FAKE = -2, 0x10000


@pytest.mark.parametrize("rows,cols", [(1 << 24, 1 << 12), (1 << 15, 1 << 21), ((1 << 30) + 128, 64), (1 << 30, 128)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_tensors_of_2_to_the_36_elements_are_refused(rows, cols, block_rows):
    from bit_nf4_quantized_15_amd import qlora as q
    st = q.Fp8State(FAKE, FAKE, rows, cols, 0, block_rows)
    assert rows * cols >= 1 << 36
    assert q.lib.qlora_fp8_quantize(FAKE, ctypes.byref(st), None) == SHAPE
    assert q.lib.qlora_fp8_dequantize(ctypes.byref(st), FAKE, None) == SHAPE
