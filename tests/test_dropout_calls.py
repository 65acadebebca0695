"""The binding's calls with dropout that are made of several library calls, with stand-ins for tensors and for the
library, without a GPU: which library calls they make, and what they refuse before the first of them."""
import types

import pytest
import torch

from test_int8_devices import Fake

BF, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8
M, N, K, R = 3, 40, 64, 8


@pytest.fixture
def q(monkeypatch):
    """The binding with a library that notes its calls and launches nothing; the current device is cuda:0.  `refuse` names
    an entry point that reports an unsupported shape."""
    from bit_nf4_quantized_15_amd import qlora
    seen = types.SimpleNamespace(q=qlora, calls=[], refuse=None)

    class Lib:
        def __getattr__(self, name):
            def f(*a):
                if name == "qlora_status_string":
                    return b"refused"
                if name.endswith("_workspace"):
                    return 4096
                seen.calls.append(name)
                return -2 if name == seen.refuse else 0
            return f

    monkeypatch.setattr(qlora, "lib", Lib())
    monkeypatch.setattr(qlora, "empty_hook", lambda *s, dtype, device: Fake(s[0] if isinstance(s[0], tuple) else s, dtype))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return seen


def int8(q, rows, cols=K):
    t = q.Int8Tensor.__new__(q.Int8Tensor)
    t.codes, t.scale, t.dtype, t.rows, t.cols = Fake((rows, cols), I8), Fake((rows,), F32), BF, rows, cols
    return t


def test_a_checkpoint_is_not_kept_of_a_layer_that_drops(q):
    """The gradients from an 8-bit checkpoint know no mask: dA would be that of x, not of drop(x)."""
    lib = q.q
    w, x, A, B = int8(lib, N), Fake((M, K), BF), Fake((K, R), BF), Fake((R, N), BF)
    with pytest.raises(ValueError, match="keep"):
        lib.int8_linear_fwd(w, x, A, B, 1.0, keep=int8(lib, M), dropout=lib.Dropout(0.1))
    assert not q.calls
    for drop in (None, lib.Dropout(0.0), lib.Dropout(0.4 / 65536)):     # nothing is dropped: x is the branch's
        lib.int8_linear_fwd(w, x, A, B, 1.0, keep=int8(lib, M), dropout=drop)
    lib.int8_linear_fwd(w, x, A, B, 1.0, dropout=lib.Dropout(0.1))


def nf4(lib, dtype=BF):
    return lib.NF4Weight(Fake((N * K // 2,), U8), Fake((N * K // 64,), U8), Fake((1,), F32), N, K, dtype=dtype)


@pytest.mark.parametrize("p", [0.0, 0.4 / 65536])
def test_a_dropout_that_drops_nothing_is_the_call_without(q, p):
    lib = q.q
    w4, w8 = nf4(lib), int8(lib, N)
    x, A, B, dy, t = Fake((M, K), BF), Fake((K, R), BF), Fake((R, N), BF), Fake((M, N), BF), Fake((M, R), BF)
    for f in (lambda d: lib.linear_fwd(w4, x, A, B, 1.0, dropout=d),
              lambda d: lib.linear_fwd(w4, x, A, B, 1.0, t=t, want_t=False, dropout=d),
              lambda d: lib.linear_bwd(w4, x, A, B, 1.0, dy, dropout=d),
              lambda d: lib.linear_bwd(w4, x, A, B, 1.0, dy, t=t, need_dx=False, dropout=d),
              lambda d: lib.int8_linear_fwd(w8, x, A, B, 1.0, dropout=d),
              lambda d: lib.int8_linear_fwd(w8, x, A, B, 1.0, want_t=False, dropout=d)):
        f(None)
        plain = list(q.calls)
        q.calls.clear()
        got, want = f(lib.Dropout(p, 1, 2)), f(None)
        assert q.calls == plain * 2
        assert [v is None for v in got] == [v is None for v in want]
        q.calls.clear()
    for f in (lib.linear_fwd, lambda *a, **kw: lib.linear_bwd(*a, dy, **kw)):    # offered for the 16-bit dtypes all the same
        with pytest.raises(TypeError):
            f(nf4(lib, F32), x, A, B, 1.0, dropout=lib.Dropout(p))


class Off(Fake):
    """A tensor whose first element is not on 16 bytes."""

    def data_ptr(self):
        return 0x10008


def _steps(lib):
    """Calls of several launches: their tensors, and the call."""
    t = dict(x=((M, K), BF), A=((K, R), BF), B=((R, N), BF), t=((M, R), BF))
    fwd = dict(t, y=((M, N), BF))
    bwd = dict(t, dy=((M, N), BF), dA=((K, R), F32), dB=((R, N), F32))
    w4, w8, d = nf4(lib), int8(lib, N), lib.Dropout(0.1)
    return {
        "linear_fwd": (fwd, lambda a: lib.linear_fwd(w4, a["x"], a["A"], a["B"], 1.0, y=a["y"], t=a["t"], dropout=d)),
        "int8_linear_fwd": (fwd, lambda a: lib.int8_linear_fwd(w8, a["x"], a["A"], a["B"], 1.0, y=a["y"], t=a["t"],
                                                               dropout=d)),
        "linear_bwd": (dict(bwd, dx=((M, K), BF)),
                       lambda a: lib.linear_bwd(w4, a["x"], a["A"], a["B"], 1.0, a["dy"], t=a["t"], dx=a["dx"], dA=a["dA"],
                                                dB=a["dB"], dropout=d)),
        "linear_bwd without dx": (bwd, lambda a: lib.linear_bwd(w4, a["x"], a["A"], a["B"], 1.0, a["dy"], t=a["t"],
                                                                need_dx=False, dA=a["dA"], dB=a["dB"], dropout=d)),
    }


@pytest.mark.parametrize("name", ["linear_fwd", "int8_linear_fwd", "linear_bwd", "linear_bwd without dx"])
def test_a_call_of_several_launches_is_refused_before_the_first(q, name):
    lib = q.q
    tensors, call = _steps(lib)[name]
    make = lambda other=None, cls=Fake, cut=0: {k: (cls if k == other else Fake)((s[0] + (cut if k == other else 0), s[1]), dt)
                                                for k, (s, dt) in tensors.items()}
    call(make())
    launches = [c for c in q.calls if c not in ("qlora_fused_gemm_fwd", "qlora_int8_gemm_fwd")]   # (asked with no rows, too)
    assert launches
    for k in tensors:
        for kw in (dict(cls=Off), dict(cut=1)):
            q.calls.clear()
            with pytest.raises((ValueError, lib.QLoraError)):
                call(make(k, **kw))
            assert not [c for c in q.calls if c in launches], f"{k} {kw}: {q.calls}"


@pytest.mark.parametrize("name,stage", [("linear_fwd", "qlora_fused_gemm_fwd"), ("int8_linear_fwd", "qlora_int8_gemm_fwd")])
def test_a_weight_that_the_product_refuses_leaves_t_alone(q, name, stage):
    tensors, call = _steps(q.q)[name]
    q.refuse = stage
    with pytest.raises(q.q.QLoraError):
        call({k: Fake(s, dt) for k, (s, dt) in tensors.items()})
    assert q.calls == [stage]


def test_widths_that_the_gradients_refuse_leave_dx_alone(q):
    lib, d = q.q, q.q.Dropout(0.1)
    for n, k in ((N, 1 << 22), (1 << 22, K)):
        w = lib.NF4Weight(Fake((n * k // 2,), U8), Fake((n * k // 64,), U8), Fake((1,), F32), n, k)
        with pytest.raises(lib.QLoraError):
            lib.linear_bwd(w, Fake((M, k), BF), Fake((k, R), BF), Fake((R, n), BF), 1.0, Fake((M, n), BF), dropout=d)
        assert not q.calls
    w = nf4(lib)                                # no rows: nothing to count, nothing to align
    lib.linear_bwd(w, Off((0, K), BF), Fake((K, R), BF), Fake((R, N), BF), 1.0, Off((0, N), BF), dropout=d)
    lib.linear_fwd(w, Off((0, K), BF), Fake((K, R), BF), Fake((R, N), BF), 1.0, dropout=d)
