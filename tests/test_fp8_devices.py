"""Every tensor of an fp8 call, and of a call with dropout, has to be on the current device: the binding's check, with
stand-ins for tensors and for the library, without a GPU."""
import pytest
import torch

from test_int8_devices import Fake, q  # noqa: F401  (a library that only counts its calls; current device cuda:0)

BF, F32, U8, F8 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn
M, N, K, R = 3, 40, 64, 8


def _fp8(q, rows, device, block_rows):
    t = q.Fp8Tensor.__new__(q.Fp8Tensor)
    t.codes, t.scale = Fake((rows, K), F8, device), Fake(q.Fp8Tensor.scale_shape(rows, K, block_rows), U8, device)
    t.dtype, t.rows, t.cols, t.block_rows = BF, rows, K, block_rows
    return t


def _nf4(q, device):
    return q.NF4Weight(Fake((N * K // 2,), U8, device), Fake((N * K // 64,), U8, device), Fake((1,), F32, device), N, K)


def _calls(q):
    """Each entry point: its tensor arguments (name -> maker on a device) and the call."""
    f = lambda *s, dtype=BF: (lambda d: Fake(s, dtype, d))
    w, x8, w4 = (lambda d: _fp8(q, N, d, 128)), (lambda d: _fp8(q, M, d, 1)), (lambda d: _nf4(q, d))
    ws, drop = f(1 << 20, dtype=U8), q.Dropout(0.1, 1, 2)
    grads = dict(x=f(M, K), t=f(M, R), u=f(M, R), dy=f(M, N), dA=f(K, R, dtype=F32), dB=f(R, N, dtype=F32), ws=ws)
    return {
        "quantize": (dict(x=f(N, K), out=w), lambda a: q.fp8_quantize(a["x"], out=a["out"])),
        "quantize_rows": (dict(x=f(M, K), out=x8), lambda a: q.fp8_quantize_rows(a["x"], out=a["out"])),
        "dequantize": (dict(q=x8, out=f(M, K)), lambda a: q.fp8_dequantize(a["q"], out=a["out"])),
        "linear_fwd": (dict(w=w, x=f(M, K), A=f(K, R), B=f(R, N), y=f(M, N), t=f(M, R), ws=ws),
                       lambda a: q.fp8_linear_fwd(a["w"], a["x"], a["A"], a["B"], 1.0, y=a["y"], t=a["t"], ws=a["ws"],
                                                  dropout=drop)),
        "gemm_fwd": (dict(w=w, x=x8, t=f(M, R), B=f(R, N), y=f(M, N)),
                     lambda a: q.fp8_gemm_fwd(a["w"], a["x"], a["t"], a["B"], y=a["y"])),
        "linear_bwd_dx": (dict(w=w, A=f(K, R), B=f(R, N), dy=f(M, N), u=f(M, R), dx=f(M, K), ws=ws),
                          lambda a: q.fp8_linear_bwd_dx(a["w"], a["A"], a["B"], 1.0, a["dy"], u=a["u"], dx=a["dx"],
                                                        ws=a["ws"], dropout=drop)),
        "dropped down": (dict(x=f(M, K), A=f(K, R), t=f(M, R), ws=ws),
                         lambda a: q.lora_down_batch([(a["x"], a["A"])], 1.0, t=[a["t"]], ws=a["ws"], dropout=[drop])),
        "dropped grads": (grads, lambda a: q.lora_grads_batch([(a["x"], a["t"], a["u"], a["dy"])], dA=[a["dA"]],
                                                              dB=[a["dB"]], ws=a["ws"], dropout=[drop])),
        "dropped dx": (dict(w=w4, A=f(K, R), B=f(R, N), dy=f(M, N), u=f(M, R), dx=f(M, K), ws=ws),
                       lambda a: q.linear_bwd_dx(a["w"], a["A"], a["B"], 1.0, a["dy"], u=a["u"], dx=a["dx"], ws=a["ws"],
                                                 dropout=drop)),
        "dropped dx stage": (dict(w=w4, dy=f(M, N), u=f(M, R), A=f(K, R), dx=f(M, K)),
                             lambda a: q.fused_gemm_bwd_dx(a["w"], a["dy"], a["u"], a["A"], dx=a["dx"], dropout=drop)),
    }


NAMES = ["quantize", "quantize_rows", "dequantize", "linear_fwd", "gemm_fwd", "linear_bwd_dx", "dropped down",
         "dropped grads", "dropped dx", "dropped dx stage"]


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_elsewhere_is_refused(q, name):  # noqa: F811
    makers, call = _calls(q.q)[name]
    call({k: m(0) for k, m in makers.items()})
    assert len(q.calls) == 1                                    # all on the current device: one call
    for other in (1, -1):                                       # another GPU, the host
        for k in makers:
            with pytest.raises(ValueError):
                call({n: m(other if n == k else 0) for n, m in makers.items()})
            assert len(q.calls) == 1, f"{k} on device {other} reached the library"


@pytest.mark.parametrize("base", ["int8", "fp8"])
def test_a_layer_without_a_branch_has_no_dropout(q, base):  # noqa: F811
    lib, drop = q.q, q.q.Dropout(0.1)
    if base == "fp8":
        for f in (lambda: lib.fp8_linear_fwd(_fp8(lib, N, 0, 128), Fake((M, K), BF), dropout=drop),
                  lambda: lib.fp8_linear_bwd_dx(_fp8(lib, N, 0, 128), None, None, 0.0, Fake((M, N), BF), dropout=drop)):
            with pytest.raises(ValueError):
                f()
    elif base == "int8":
        w = lib.Int8Tensor.__new__(lib.Int8Tensor)
        w.codes, w.scale, w.dtype, w.rows, w.cols = Fake((N, K), torch.int8), Fake((N,), F32), BF, N, K
        for f in (lambda: lib.int8_linear_fwd(w, Fake((M, K), BF), dropout=drop),
                  lambda: lib.int8_linear_bwd_dx(w, None, None, 0.0, Fake((M, N), BF), dropout=drop),
                  lambda: lib.int8_gemm_bwd_dx(w, Fake((M, N), BF), dropout=drop)):
            with pytest.raises(ValueError):
                f()
    assert not q.calls
