"""Thin ctypes binding over libqlora.so (include/qlora.h).

Argument marshalling only: torch supplies device memory and the current HIP
stream; every step of the computation runs in the library's HIP kernels.
Importing this module loads the library and raises ImportError when it has not
been built (python -m bit_nf4_quantized_15_amd.build); there is no fallback.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "qlora.h")

BLOCK = 64
SUPER = 256

c_i64 = ctypes.c_int64
c_vp = ctypes.c_void_p
c_sz = ctypes.c_size_t


class NF4State(ctypes.Structure):
    """Mirror of struct qlora_nf4."""
    _fields_ = [("codes", c_vp), ("q8", c_vp), ("a2", c_vp), ("n", c_i64), ("k", c_i64), ("quant_type", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class LoraGrads(ctypes.Structure):
    """Mirror of struct qlora_lora_grads."""
    _fields_ = [("x", c_vp), ("t", c_vp), ("u", c_vp), ("dy", c_vp), ("dA", c_vp), ("dB", c_vp), ("M", c_i64),
                ("N", c_i64), ("K", c_i64)]


class LoraProd(ctypes.Structure):
    """Mirror of struct qlora_lora_prod."""
    _fields_ = [("x", c_vp), ("w", c_vp), ("out", c_vp), ("M", c_i64), ("C", c_i64)]


class Int8State(ctypes.Structure):
    """Mirror of struct qlora_int8."""
    _fields_ = [("codes", c_vp), ("scale", c_vp), ("rows", c_i64), ("cols", c_i64), ("dtype", ctypes.c_int32)]


class LoraGradsInt8(ctypes.Structure):
    """Mirror of struct qlora_lora_grads_int8."""
    _fields_ = [("x", c_vp), ("x_scale", c_vp), ("t", c_vp), ("u", c_vp), ("dy", c_vp), ("dA", c_vp), ("dB", c_vp),
                ("M", c_i64), ("N", c_i64), ("K", c_i64)]


class DropoutState(ctypes.Structure):
    """Mirror of struct qlora_dropout."""
    _fields_ = [("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("p", ctypes.c_double)]


class Fp8State(ctypes.Structure):
    """Mirror of struct qlora_fp8."""
    _fields_ = [("codes", c_vp), ("scale", c_vp), ("rows", c_i64), ("cols", c_i64), ("dtype", ctypes.c_int32),
                ("block_rows", ctypes.c_int32)]


QUANT_TYPES = {"nf4": 0, "fp4": 1}                        # qlora_quant_type: the 4-bit codebook
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # qlora_dtype: the compute dtype


def _dtype_code(dtype):
    if dtype not in DTYPES:
        raise TypeError(f"compute dtype must be torch.bfloat16, torch.float16 or torch.float32, got {dtype}")
    return DTYPES[dtype]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m bit_nf4_quantized_15_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(NF4State)
    I8 = ctypes.POINTER(Int8State)
    F8 = ctypes.POINTER(Fp8State)
    DR = ctypes.POINTER(DropoutState)
    sig = {
        "qlora_version": (ctypes.c_int, []),
        "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "qlora_nf4_sizes": (ctypes.c_int, [c_i64, c_i64, ctypes.POINTER(c_sz), ctypes.POINTER(c_sz),
                                           ctypes.POINTER(c_sz)]),
        "qlora_nf4_sizes_nodq": (ctypes.c_int, [c_i64, c_i64, ctypes.POINTER(c_sz), ctypes.POINTER(c_sz)]),
        "qlora_quantize": (ctypes.c_int, [c_vp, c_i64, c_i64, P, c_vp]),
        "qlora_quantize_batch": (ctypes.c_int, [ctypes.POINTER(c_vp), P, ctypes.c_int, c_vp]),
        "qlora_dequantize": (ctypes.c_int, [P, c_vp, c_vp]),
        "qlora_dequantize_f32": (ctypes.c_int, [P, c_vp, c_vp]),
        "qlora_merge": (ctypes.c_int, [P, c_vp, c_vp, ctypes.c_int, ctypes.c_float, c_vp, c_vp]),
        "qlora_fwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_linear_fwd": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float,
                                            c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_linear_fwd_noalloc": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float,
                                                    c_vp, c_vp, c_vp]),
        "qlora_read_probe": (ctypes.c_int, [c_vp, c_sz, c_vp, ctypes.c_int, c_vp]),
        "qlora_lora_down_workspace": (c_sz, [c_i64, c_i64, ctypes.c_int]),
        "qlora_lora_down": (ctypes.c_int, [c_vp, c_i64, c_i64, c_vp, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                                           c_vp, c_vp, c_sz, c_vp]),
        "qlora_fused_gemm_fwd": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, c_vp, c_vp]),
        "qlora_fused_gemm_bwd_dx": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, c_vp, c_vp]),
        "qlora_pooled_fwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int]),
        "qlora_pooled_fwd": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                            c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_pooled_bwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int]),
        "qlora_pooled_bwd": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                            c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_bwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_linear_bwd": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float,
                                            c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_linear_bwd_dx_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_linear_bwd_dx": (ctypes.c_int, [P, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, c_vp, c_vp, c_vp,
                                               c_vp, c_sz, c_vp]),
        "qlora_lora_grads_batch_workspace": (c_sz, [ctypes.POINTER(LoraGrads), ctypes.c_int, ctypes.c_int]),
        "qlora_lora_grads_batch": (ctypes.c_int, [ctypes.POINTER(LoraGrads), ctypes.c_int, ctypes.c_int,
                                                  ctypes.c_int, c_vp, c_sz, c_vp]),
        "qlora_lora_prod_batch_workspace": (c_sz, [ctypes.POINTER(LoraProd), ctypes.c_int, ctypes.c_int]),
        "qlora_lora_down_batch": (ctypes.c_int, [ctypes.POINTER(LoraProd), ctypes.c_int, ctypes.c_int,
                                                 ctypes.c_float, ctypes.c_int, c_vp, c_sz, c_vp]),
        "qlora_lora_u_batch": (ctypes.c_int, [ctypes.POINTER(LoraProd), ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                              ctypes.c_int, c_vp, c_sz, c_vp]),
        "qlora_quantize_f32": (ctypes.c_int, [c_vp, c_i64, c_i64, P, c_vp]),
        "qlora_fwd_workspace_f32": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_linear_fwd_f32": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float,
                                                c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_bwd_workspace_f32": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_linear_bwd_f32": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float,
                                                c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_int8_quantize": (ctypes.c_int, [c_vp, I8, c_vp]),
        "qlora_int8_dequantize": (ctypes.c_int, [I8, c_vp, c_vp]),
        "qlora_int8_fwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_int8_linear_fwd": (ctypes.c_int, [I8, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, c_vp,
                                                 c_vp, I8, c_vp, c_sz, c_vp]),
        "qlora_int8_gemm_fwd": (ctypes.c_int, [I8, I8, c_vp, c_vp, ctypes.c_int, c_vp, c_vp]),
        "qlora_int8_linear_bwd_dx_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_int8_linear_bwd_dx": (ctypes.c_int, [I8, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, c_vp, c_vp,
                                                    c_vp, c_vp, c_sz, c_vp]),
        "qlora_int8_gemm_bwd_dx": (ctypes.c_int, [I8, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, c_vp, c_vp]),
        "qlora_lora_grads_batch_int8_workspace": (c_sz, [ctypes.POINTER(LoraGradsInt8), ctypes.c_int, ctypes.c_int]),
        "qlora_lora_grads_batch_int8": (ctypes.c_int, [ctypes.POINTER(LoraGradsInt8), ctypes.c_int, ctypes.c_int,
                                                       ctypes.c_int, c_vp, c_sz, c_vp]),
    }
    sig.update({
        "qlora_lora_down_batch_dropout": (ctypes.c_int, [ctypes.POINTER(LoraProd), DR, ctypes.c_int, ctypes.c_int,
                                                         ctypes.c_float, ctypes.c_int, c_vp, c_sz, c_vp]),
        "qlora_lora_grads_batch_dropout": (ctypes.c_int, [ctypes.POINTER(LoraGrads), DR, ctypes.c_int, ctypes.c_int,
                                                          ctypes.c_int, c_vp, c_sz, c_vp]),
        "qlora_linear_bwd_dx_dropout": (ctypes.c_int, [P, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, DR, c_vp,
                                                       c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_fused_gemm_bwd_dx_dropout": (ctypes.c_int, [P, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, DR, c_vp, c_vp]),
        "qlora_int8_linear_bwd_dx_dropout": (ctypes.c_int, [I8, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, DR,
                                                            c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "qlora_int8_gemm_bwd_dx_dropout": (ctypes.c_int, [I8, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, DR, c_vp, c_vp]),
        "qlora_fp8_scale_bytes": (c_sz, [c_i64, c_i64, ctypes.c_int]),
        "qlora_fp8_quantize": (ctypes.c_int, [c_vp, F8, c_vp]),
        "qlora_fp8_dequantize": (ctypes.c_int, [F8, c_vp, c_vp]),
        "qlora_fp8_fwd_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_fp8_linear_fwd": (ctypes.c_int, [F8, c_vp, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, DR, c_vp,
                                                c_vp, c_vp, c_sz, c_vp]),
        "qlora_fp8_gemm_fwd": (ctypes.c_int, [F8, F8, c_vp, c_vp, ctypes.c_int, c_vp, c_vp]),
        "qlora_fp8_linear_bwd_dx_workspace": (c_sz, [c_i64, c_i64, c_i64, ctypes.c_int]),
        "qlora_fp8_linear_bwd_dx": (ctypes.c_int, [F8, c_i64, c_vp, c_vp, ctypes.c_int, ctypes.c_float, DR, c_vp, c_vp,
                                                   c_vp, c_vp, c_sz, c_vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(lib, name, None)
        if fn is None:
            continue
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class QLoraError(RuntimeError):
    def __init__(self, status, where):
        msg = lib.qlora_status_string(status).decode()
        super().__init__(f"{where}: status {status} ({msg})")
        self.status = status


def _empty(*shape, dtype, device):
    """Every buffer this module hands to the library is allocated here (outputs, weight state and workspace).
    Uninitialised, like torch.empty; the GPU tests replace `empty_hook` to fill new buffers with a poison
    pattern, so that an element a kernel never writes cannot pass for a correct one."""
    return empty_hook(*shape, dtype=dtype, device=device)


empty_hook = torch.empty


def _check(status, where):
    if status != 0:
        raise QLoraError(status, where)


def _stream():
    """The current stream's handle.  Read directly: building torch's stream object takes longer (2.9 us) than
    checking the arguments of a call."""
    return c_vp(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _ptr(t):
    return None if t is None else c_vp(t.data_ptr())


def _dev(t, dtype, name, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: must be a contiguous device tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


class Dropout:
    """Dropout of a LoRA branch's input (struct qlora_dropout): probability p, and the counter-based generator's seed
    and offset, 64 bits each.  The forward and the backward of a layer are given the same one; layers and steps whose
    masks are to differ take other offsets or seeds.  Seed and offset are read when a call is made: one captured into
    a graph has the same mask at every replay.  p acts as round(65536 p) / 65536."""

    def __init__(self, p, seed=0, offset=0):
        if not 0.0 <= p < 1.0 or round(p * 65536) > 65535:
            raise ValueError(f"p: expected 0 <= p < 1 and at most 65535/65536 when rounded, got {p}")
        for name, v in (("seed", seed), ("offset", offset)):
            if not 0 <= v < 2 ** 64:
                raise ValueError(f"{name}: expected 0 <= {name} < 2**64, got {v}")
        self.p, self.seed, self.offset = float(p), int(seed), int(offset)

    @property
    def drops(self):
        """Whether it drops anything: round(65536 p) > 0."""
        return round(self.p * 65536) > 0

    def state(self):
        return DropoutState(self.seed, self.offset, self.p)


def _drops(dropout, n):
    """The array of n drops of a list whose None entries drop nothing."""
    if len(dropout) != n:
        raise ValueError("dropout: one entry per layer (None: no dropout)")
    return (DropoutState * n)(*[DropoutState(0, 0, 0.0) if d is None else d.state() for d in dropout])


def _no_f32(w, what):
    if w.dtype == torch.float32:
        raise TypeError(f"{what}: dropout is offered for the 16-bit dtypes")


def _here(*tensors):
    """A call with dropout runs on the current device's stream: its tensors (None: not given) have to be there."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"a tensor on {t.device}, but the current device is cuda:{cur}")


def _aligned(where, *tensors):
    """Of a call that makes several: their tensors' alignment, before the first of them is made, so that one that is
    refused leaves every output as it was."""
    if any(t is not None and t.data_ptr() % 16 for t in tensors):
        raise QLoraError(-3, where)


GRADS_DROPOUT_WIDTH = 1 << 22      # N and K of qlora_lora_grads_batch_dropout lie below


def sizes(N, K):
    """(codes bytes, q8 bytes, a2 bytes) of an [N, K] quantized weight."""
    cb, qb, ab = c_sz(), c_sz(), c_sz()
    _check(lib.qlora_nf4_sizes(N, K, ctypes.byref(cb), ctypes.byref(qb), ctypes.byref(ab)), "qlora_nf4_sizes")
    return cb.value, qb.value, ab.value


def sizes_nodq(N, K):
    """(codes bytes, fp32 block-absmax bytes) of an [N, K] weight quantized without double quantization."""
    cb, ab = c_sz(), c_sz()
    _check(lib.qlora_nf4_sizes_nodq(N, K, ctypes.byref(cb), ctypes.byref(ab)), "qlora_nf4_sizes_nodq")
    return cb.value, ab.value


class NF4Weight:
    """Device-resident quantized weight: codes (uint8), q8 (uint8) and a2 (float32) tensors; without
    double quantization q8 is None and a2 holds one fp32 absmax per 64-block.  quant_type names the
    4-bit codebook ("nf4" or "fp4"); dtype is the compute dtype of every float tensor used with it
    (torch.bfloat16, torch.float16, or torch.float32: then the layer calls take the _f32 entry points and the
    dequantized weight is the fp32 product itself)."""

    def __init__(self, codes, q8, a2, N, K, quant_type="nf4", dtype=torch.bfloat16):
        if quant_type not in QUANT_TYPES:
            raise ValueError(f"quant_type must be one of {sorted(QUANT_TYPES)}, got {quant_type!r}")
        _dtype_code(dtype)
        self.codes, self.q8, self.a2, self.N, self.K = codes, q8, a2, int(N), int(K)
        self.quant_type, self.dtype = quant_type, dtype

    @property
    def double_quant(self):
        return self.q8 is not None

    @classmethod
    def empty(cls, N, K, device="cuda", double_quant=True, quant_type="nf4", dtype=torch.bfloat16):
        if not double_quant:
            cb, ab = sizes_nodq(N, K)
            return cls(_empty(cb, dtype=torch.uint8, device=device), None,
                       _empty(ab // 4, dtype=torch.float32, device=device), N, K, quant_type, dtype)
        cb, qb, ab = sizes(N, K)
        return cls(_empty(cb, dtype=torch.uint8, device=device),
                   _empty(qb, dtype=torch.uint8, device=device),
                   _empty(ab // 4, dtype=torch.float32, device=device), N, K, quant_type, dtype)

    def state(self):
        q8 = None if self.q8 is None else self.q8.data_ptr()
        return NF4State(self.codes.data_ptr(), q8, self.a2.data_ptr(), self.N, self.K, QUANT_TYPES[self.quant_type],
                        _dtype_code(self.dtype))


def quantize(W, out=None, double_quant=True, quant_type="nf4"):
    """4-bit blockwise quantization of a bf16, fp16 or fp32 [N, K] device weight (qlora_quantize, or
    qlora_quantize_f32 for fp32) with the NF4 or the FP4 codebook, with or without double quantization of
    the block scales (both ignored when `out` is given: its layout and quant_type decide).  W's dtype
    becomes the weight's compute dtype."""
    N, K = W.shape
    _dtype_code(W.dtype)
    _dev(W, W.dtype, "W")
    w = NF4Weight.empty(N, K, W.device, double_quant, quant_type, W.dtype) if out is None else out
    if w.dtype != W.dtype:
        raise TypeError(f"out has compute dtype {w.dtype}, W is {W.dtype}")
    st = w.state()
    if W.dtype == torch.float32:
        _check(lib.qlora_quantize_f32(_ptr(W), N, K, ctypes.byref(st), _stream()), "qlora_quantize_f32")
    else:
        _check(lib.qlora_quantize(_ptr(W), N, K, ctypes.byref(st), _stream()), "qlora_quantize")
    return w


def quantize_batch(Ws, outs):
    """Quantize bf16/fp16 device weights Ws[i] into the existing NF4Weight outs[i] (qlora_quantize_batch:
    the results of one qlora_quantize per weight, in one launch per run of up to 16 weights that share
    their configuration)."""
    if len(Ws) != len(outs):
        raise ValueError("Ws and outs differ in length")
    for W, w in zip(Ws, outs):
        _dtype_code(W.dtype)
        _dev(W, w.dtype, "W", (w.N, w.K))
    n = len(Ws)
    ptrs = (c_vp * max(n, 1))(*[_ptr(W) for W in Ws])
    states = (NF4State * max(n, 1))(*[w.state() for w in outs])
    _check(lib.qlora_quantize_batch(ptrs, states, n, _stream()), "qlora_quantize_batch")
    return outs


def dequantize(w, out=None, fp32=False):
    """[N, K] reconstruction in the weight's compute dtype (qlora_dequantize), or with fp32=True the fp32
    products themselves (qlora_dequantize_f32, also the reconstruction of an fp32 weight); tests and export
    only."""
    fp32 = fp32 or w.dtype == torch.float32
    dt = torch.float32 if fp32 else w.dtype
    o = _empty((w.N, w.K), dtype=dt, device=w.codes.device) if out is None else out
    _dev(o, dt, "out", (w.N, w.K))
    st = w.state()
    if fp32:
        _check(lib.qlora_dequantize_f32(ctypes.byref(st), _ptr(o), _stream()), "qlora_dequantize_f32")
    else:
        _check(lib.qlora_dequantize(ctypes.byref(st), _ptr(o), _stream()), "qlora_dequantize")
    return o


def merge(w, A, B, alpha, out=None):
    """LoRA merge for deployment (qlora_merge): bf16 [N, K] = w_hat + (alpha/r) (A B)^T.
    Re-quantize with quantize(out)."""
    K, r = A.shape
    _dev(A, w.dtype, "A", (w.K, r))
    _dev(B, w.dtype, "B", (r, w.N))
    o = _empty((w.N, w.K), dtype=w.dtype, device=A.device) if out is None else out
    _dev(o, w.dtype, "out", (w.N, w.K))
    st = w.state()
    _check(lib.qlora_merge(ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(o), _stream()), "qlora_merge")
    return o


def fwd_workspace(M, N, K, r, dtype=torch.bfloat16):
    if dtype == torch.float32:
        return int(lib.qlora_fwd_workspace_f32(M, N, K, r))
    return int(lib.qlora_fwd_workspace(M, N, K, r))


def bwd_workspace(M, N, K, r, dtype=torch.bfloat16):
    if dtype == torch.float32:
        return int(lib.qlora_bwd_workspace_f32(M, N, K, r))
    return int(lib.qlora_bwd_workspace(M, N, K, r))


def _ws(nbytes, device, ws):
    if nbytes == 0:
        return None, 0
    if ws is not None and ws.numel() >= nbytes:
        return ws, ws.numel()
    return _empty(nbytes, dtype=torch.uint8, device=device), nbytes


def linear_fwd(w, x, A, B, alpha, y=None, t=None, want_t=True, ws=None, dropout=None):
    """y = x W_hat + (alpha/r)(x A) B (qlora_linear_fwd).  Returns (y, t or None).  With a Dropout the branch takes
    drop(x) for x (qlora_lora_down_batch_dropout, then qlora_fused_gemm_fwd); one that drops nothing is None."""
    if dropout is not None:
        _no_f32(w, "linear_fwd")
        _here(x, A, B, w.codes, w.q8, w.a2, y, t, ws)
    if dropout is not None and dropout.drops:
        M, r = x.shape[0], A.shape[1]
        _dev(B, w.dtype, "B", (r, w.N))
        _dev(x, w.dtype, "x", (M, w.K))
        _dev(A, w.dtype, "A", (w.K, r))
        if y is not None:
            _dev(y, w.dtype, "y", (M, w.N))
        if t is not None:
            _dev(t, w.dtype, "t", (M, r))
        if M:
            _aligned("linear_fwd", x, A, B, y, t)
        # (the product of no rows: its checks of the weight, before t is written)
        _check(lib.qlora_fused_gemm_fwd(ctypes.byref(w.state()), None, 0, None, None, r, None, _stream()),
               "qlora_fused_gemm_fwd")
        t = lora_down(x, A, alpha, t=t, ws=ws, dropout=dropout)
        return fused_gemm_fwd(w, x, t, B, y=y), (t if want_t else None)
    M, K = x.shape
    r = A.shape[1]
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(A, w.dtype, "A", (w.K, r))
    _dev(B, w.dtype, "B", (r, w.N))
    dev = x.device
    y = _empty((M, w.N), dtype=w.dtype, device=dev) if y is None else _dev(y, w.dtype, "y", (M, w.N))
    if want_t and t is None:
        t = _empty((M, r), dtype=w.dtype, device=dev)
    if t is not None:
        _dev(t, w.dtype, "t", (M, r))
    wsb, wsn = _ws(fwd_workspace(M, w.N, w.K, r, w.dtype), dev, ws)
    st = w.state()
    fn, name = ((lib.qlora_linear_fwd_f32, "qlora_linear_fwd_f32") if w.dtype == torch.float32
                else (lib.qlora_linear_fwd, "qlora_linear_fwd"))
    _check(fn(ctypes.byref(st), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(y), _ptr(t), _ptr(wsb), wsn,
              _stream()), name)
    return y, t


def linear_fwd_noalloc(w, x, A, B, alpha, y=None, t=None, want_t=True):
    """linear_fwd without a workspace argument (qlora_linear_fwd_noalloc): the library's fixed per-GPU
    array serves as workspace, so the call itself allocates nothing.  Returns (y, t or None)."""
    M, K = x.shape
    r = A.shape[1]
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(A, w.dtype, "A", (w.K, r))
    _dev(B, w.dtype, "B", (r, w.N))
    dev = x.device
    y = _empty((M, w.N), dtype=w.dtype, device=dev) if y is None else _dev(y, w.dtype, "y", (M, w.N))
    if want_t and t is None:
        t = _empty((M, r), dtype=w.dtype, device=dev)
    if t is not None:
        _dev(t, w.dtype, "t", (M, r))
    st = w.state()
    _check(lib.qlora_linear_fwd_noalloc(ctypes.byref(st), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(y),
                                        _ptr(t), _stream()), "qlora_linear_fwd_noalloc")
    return y, t


def read_probe(buf, sink, variant=0):
    """Plain read of a device buffer (qlora_read_probe): the same-size bandwidth ceiling of the bench."""
    _check(lib.qlora_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), variant, _stream()),
           "qlora_read_probe")


def lora_down(x, A, alpha, t=None, ws=None, dropout=None):
    """t = (alpha/r) x A [M, r] in x's dtype, bf16 or fp16 (qlora_lora_down); with a Dropout, of drop(x)
    (qlora_lora_down_batch_dropout)."""
    if dropout is not None:
        return lora_down_batch([(x, A)], alpha, t=[t], ws=ws, dropout=[dropout])[0]
    M, K = x.shape
    r = A.shape[1]
    dt = x.dtype
    code = _dtype_code(dt)
    _dev(x, dt, "x")
    _dev(A, dt, "A", (K, r))
    t = _empty((M, r), dtype=dt, device=x.device) if t is None else _dev(t, dt, "t", (M, r))
    wsb, wsn = _ws(int(lib.qlora_lora_down_workspace(M, K, r)), x.device, ws)
    _check(lib.qlora_lora_down(_ptr(x), M, K, _ptr(A), r, float(alpha), code, _ptr(t), _ptr(wsb), wsn, _stream()),
           "qlora_lora_down")
    return t


def fused_gemm_fwd(w, x, t, B, y=None):
    """y = x W_hat + t B (qlora_fused_gemm_fwd): one kernel launch."""
    M = x.shape[0]
    r = t.shape[1]
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(t, w.dtype, "t", (M, r))
    _dev(B, w.dtype, "B", (r, w.N))
    y = _empty((M, w.N), dtype=w.dtype, device=x.device) if y is None else _dev(y, w.dtype, "y", (M, w.N))
    st = w.state()
    _check(lib.qlora_fused_gemm_fwd(ctypes.byref(st), _ptr(x), M, _ptr(t), _ptr(B), r, _ptr(y), _stream()),
           "qlora_fused_gemm_fwd")
    return y


def fused_gemm_bwd_dx(w, dy, u, A, dx=None, dropout=None):
    """dx = dy W_hat^T + u A^T (qlora_fused_gemm_bwd_dx), u = (alpha/r) dy B^T given: one kernel launch.  With a
    Dropout, dy W_hat^T + drop(u A^T) (qlora_fused_gemm_bwd_dx_dropout)."""
    M = dy.shape[0]
    r = u.shape[1]
    _dev(dy, w.dtype, "dy", (M, w.N))
    _dev(u, w.dtype, "u", (M, r))
    _dev(A, w.dtype, "A", (w.K, r))
    dx = _empty((M, w.K), dtype=w.dtype, device=dy.device) if dx is None else _dev(dx, w.dtype, "dx", (M, w.K))
    st = w.state()
    if dropout is not None:
        _no_f32(w, "fused_gemm_bwd_dx")
        _here(dy, u, A, w.codes, w.q8, w.a2, dx)
        _check(lib.qlora_fused_gemm_bwd_dx_dropout(ctypes.byref(st), _ptr(dy), M, _ptr(u), _ptr(A), r,
                                                   ctypes.byref(dropout.state()), _ptr(dx), _stream()),
               "qlora_fused_gemm_bwd_dx_dropout")
        return dx
    _check(lib.qlora_fused_gemm_bwd_dx(ctypes.byref(st), _ptr(dy), M, _ptr(u), _ptr(A), r, _ptr(dx), _stream()),
           "qlora_fused_gemm_bwd_dx")
    return dx


def linear_bwd(w, x, A, B, alpha, dy, t=None, need_dx=True, dx=None, dA=None, dB=None, ws=None, dropout=None):
    """(dx, dA, dB) of the layer for upstream dy (qlora_linear_bwd); dx is None when not needed.  With the forward's
    Dropout: its three stages (u and dx, then the gradients of drop(x); a t not given is computed again); one that
    drops nothing is None."""
    if dropout is not None:
        _no_f32(w, "linear_bwd")
        _here(x, A, B, dy, t, w.codes, w.q8, w.a2, dx, dA, dB, ws)
    if dropout is not None and dropout.drops:
        M, r = x.shape[0], A.shape[1]
        for v, dt, name, shape in ((x, w.dtype, "x", (M, w.K)), (A, w.dtype, "A", (w.K, r)), (B, w.dtype, "B", (r, w.N)),
                                   (dy, w.dtype, "dy", (M, w.N)), (t, w.dtype, "t", (M, r)),
                                   (dx if need_dx else None, w.dtype, "dx", (M, w.K)),
                                   (dA, torch.float32, "dA", (w.K, r)), (dB, torch.float32, "dB", (r, w.N))):
            if v is not None:
                _dev(v, dt, name, shape)
        if M:
            _aligned("linear_bwd", x, A, B, dy, t, dx if need_dx else None, dA, dB, ws)
            if max(w.N, w.K) >= GRADS_DROPOUT_WIDTH:
                raise QLoraError(-2, "linear_bwd")
        if need_dx:
            u, dx = linear_bwd_dx(w, A, B, alpha, dy, dx=dx, ws=ws, dropout=dropout)
        else:
            u = lora_u_batch([(dy, B)], alpha, ws=ws)[0]
        if t is None:
            t = lora_down(x, A, alpha, ws=ws, dropout=dropout)
        (dA,), (dB,) = lora_grads_batch([(x, t, u, dy)], dA=[dA], dB=[dB], ws=ws, dropout=[dropout])
        return (dx if need_dx else None), dA, dB
    M, K = x.shape
    r = A.shape[1]
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(A, w.dtype, "A", (w.K, r))
    _dev(B, w.dtype, "B", (r, w.N))
    _dev(dy, w.dtype, "dy", (M, w.N))
    if t is not None:
        _dev(t, w.dtype, "t", (M, r))
    dev = x.device
    if need_dx:
        dx = _empty((M, w.K), dtype=w.dtype, device=dev) if dx is None else _dev(dx, w.dtype, "dx", (M, w.K))
    dA = _empty((w.K, r), dtype=torch.float32, device=dev) if dA is None else _dev(dA, torch.float32, "dA", (w.K, r))
    dB = _empty((r, w.N), dtype=torch.float32, device=dev) if dB is None else _dev(dB, torch.float32, "dB", (r, w.N))
    wsb, wsn = _ws(bwd_workspace(M, w.N, w.K, r, w.dtype), dev, ws)
    st = w.state()
    fn, name = ((lib.qlora_linear_bwd_f32, "qlora_linear_bwd_f32") if w.dtype == torch.float32
                else (lib.qlora_linear_bwd, "qlora_linear_bwd"))
    _check(fn(ctypes.byref(st), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(t), _ptr(dy),
              _ptr(dx) if need_dx else None, _ptr(dA), _ptr(dB), _ptr(wsb), wsn, _stream()), name)
    return (dx if need_dx else None), dA, dB


def linear_bwd_dx(w, A, B, alpha, dy, u=None, dx=None, ws=None, dropout=None):
    """(u, dx) of the layer for upstream dy (qlora_linear_bwd_dx): u = (alpha/r) dy B^T, kept for
    lora_grads_batch, and dx = dy W_hat^T + u A^T.  With the forward's Dropout, dy W_hat^T + drop(u A^T)
    (qlora_linear_bwd_dx_dropout)."""
    M = dy.shape[0]
    r = A.shape[1]
    _dev(A, w.dtype, "A", (w.K, r))
    _dev(B, w.dtype, "B", (r, w.N))
    _dev(dy, w.dtype, "dy", (M, w.N))
    dev = dy.device
    u = _empty((M, r), dtype=w.dtype, device=dev) if u is None else _dev(u, w.dtype, "u", (M, r))
    dx = _empty((M, w.K), dtype=w.dtype, device=dev) if dx is None else _dev(dx, w.dtype, "dx", (M, w.K))
    wsb, wsn = _ws(int(lib.qlora_linear_bwd_dx_workspace(M, w.N, w.K, r)), dev, ws)
    st = w.state()
    if dropout is not None:
        _no_f32(w, "linear_bwd_dx")
        _here(A, B, dy, w.codes, w.q8, w.a2, u, dx, ws)
        _check(lib.qlora_linear_bwd_dx_dropout(ctypes.byref(st), M, _ptr(A), _ptr(B), r, float(alpha),
                                               ctypes.byref(dropout.state()), _ptr(dy), _ptr(u), _ptr(dx), _ptr(wsb),
                                               wsn, _stream()), "qlora_linear_bwd_dx_dropout")
        return u, dx
    _check(lib.qlora_linear_bwd_dx(ctypes.byref(st), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(dy), _ptr(u),
                                   _ptr(dx), _ptr(wsb), wsn, _stream()), "qlora_linear_bwd_dx")
    return u, dx


def lora_grads_batch(layers, dA=None, dB=None, ws=None, dropout=None):
    """dA = x^T u and dB = t^T dy (fp32) of several layers in one launch per 8 layers
    (qlora_lora_grads_batch).  layers: a list of (x, t, u, dy), all of one rank r and one dtype (bf16 or
    fp16); dA, dB: optional lists of output tensors.  dropout: optional list of the layers' Dropouts (None entries
    drop nothing), then dA = drop(x)^T u (qlora_lora_grads_batch_dropout).  Returns the lists (dA, dB)."""
    n = len(layers)
    if n == 0:
        return [], []
    dt = layers[0][0].dtype
    code = _dtype_code(dt)
    r = layers[0][1].shape[1]
    dA = [None] * n if dA is None else list(dA)
    dB = [None] * n if dB is None else list(dB)
    descs = (LoraGrads * n)()
    for i, (x, t, u, dy) in enumerate(layers):
        M, K = x.shape
        N = dy.shape[1]
        _dev(x, dt, "x")
        _dev(t, dt, "t", (M, r))
        _dev(u, dt, "u", (M, r))
        _dev(dy, dt, "dy", (M, N))
        dev = x.device
        dA[i] = _empty((K, r), dtype=torch.float32, device=dev) if dA[i] is None else _dev(dA[i], torch.float32,
                                                                                          "dA", (K, r))
        dB[i] = _empty((r, N), dtype=torch.float32, device=dev) if dB[i] is None else _dev(dB[i], torch.float32,
                                                                                          "dB", (r, N))
        descs[i] = LoraGrads(x.data_ptr(), t.data_ptr(), u.data_ptr(), dy.data_ptr(), dA[i].data_ptr(),
                             dB[i].data_ptr(), M, N, K)
    wsb, wsn = _ws(int(lib.qlora_lora_grads_batch_workspace(descs, n, r)), layers[0][0].device, ws)
    if dropout is not None:
        _here(ws, *dA, *dB, *(v for layer in layers for v in layer))
        _check(lib.qlora_lora_grads_batch_dropout(descs, _drops(dropout, n), n, r, code, _ptr(wsb), wsn, _stream()),
               "qlora_lora_grads_batch_dropout")
        return dA, dB
    _check(lib.qlora_lora_grads_batch(descs, n, r, code, _ptr(wsb), wsn, _stream()), "qlora_lora_grads_batch")
    return dA, dB


def _lora_prod_batch(fn, name, items, alpha, natural, outs, ws, dropout=None):
    n = len(items)
    if n == 0:
        return []
    dt = items[0][0].dtype
    code = _dtype_code(dt)
    r = items[0][1].shape[1] if natural else items[0][1].shape[0]
    outs = [None] * n if outs is None else list(outs)
    descs = (LoraProd * n)()
    for i, (X, Y) in enumerate(items):
        M, C = X.shape
        _dev(X, dt, "x" if natural else "dy")
        _dev(Y, dt, "A" if natural else "B", (C, r) if natural else (r, C))
        outs[i] = _empty((M, r), dtype=dt, device=X.device) if outs[i] is None else _dev(outs[i], dt, "out", (M, r))
        descs[i] = LoraProd(X.data_ptr(), Y.data_ptr(), outs[i].data_ptr(), M, C)
    wsb, wsn = _ws(int(lib.qlora_lora_prod_batch_workspace(descs, n, r)), items[0][0].device, ws)
    if dropout is not None:
        _here(ws, *outs, *(v for item in items for v in item))
        _check(fn(descs, _drops(dropout, n), n, r, float(alpha), code, _ptr(wsb), wsn, _stream()), name)
        return outs
    _check(fn(descs, n, r, float(alpha), code, _ptr(wsb), wsn, _stream()), name)
    return outs


def lora_down_batch(items, alpha, t=None, ws=None, dropout=None):
    """t_i = (alpha/r) x_i A_i for items [(x_i, A_i)] in one launch per 8 (qlora_lora_down_batch); each t_i is
    that of lora_down.  t: optional list of outputs.  dropout: optional list of Dropouts (None entries drop nothing),
    then t_i = (alpha/r) drop_i(x_i) A_i (qlora_lora_down_batch_dropout; the last bit may depend on how many of the
    items drop something).  Returns the list of t_i."""
    if dropout is not None:
        return _lora_prod_batch(lib.qlora_lora_down_batch_dropout, "qlora_lora_down_batch_dropout", items, alpha, True, t,
                                ws, dropout)
    return _lora_prod_batch(lib.qlora_lora_down_batch, "qlora_lora_down_batch", items, alpha, True, t, ws)


def lora_u_batch(items, alpha, u=None, ws=None):
    """u_i = (alpha/r) dy_i B_i^T for items [(dy_i, B_i)], B_i [r, N_i], in one launch per 8
    (qlora_lora_u_batch); each u_i is that of linear_bwd_dx.  u: optional list of outputs."""
    return _lora_prod_batch(lib.qlora_lora_u_batch, "qlora_lora_u_batch", items, alpha, False, u, ws)


def pooled_fwd(w, x, A, B, alpha, g, y=None, t=None, ws=None):
    """QA-LoRA pooled forward (qlora_pooled_fwd): y = x W_hat + s pool(x) A B, A [K/g, r]. Returns (y, t)."""
    M, K = x.shape
    _, r = A.shape
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(A, w.dtype, "A", (w.K // g, r))
    _dev(B, w.dtype, "B", (r, w.N))
    y = _empty((M, w.N), dtype=w.dtype, device=x.device) if y is None else _dev(y, w.dtype, "y", (M, w.N))
    t = _empty((M, r), dtype=w.dtype, device=x.device) if t is None else _dev(t, w.dtype, "t", (M, r))
    wsb, wsn = _ws(int(lib.qlora_pooled_fwd_workspace(M, w.N, w.K, r, g)), x.device, ws)
    st = w.state()
    _check(lib.qlora_pooled_fwd(ctypes.byref(st), _ptr(x), M, _ptr(A), _ptr(B), r, g, float(alpha), _ptr(y), _ptr(t),
                                _ptr(wsb), wsn, _stream()), "qlora_pooled_fwd")
    return y, t


def pooled_bwd(w, x, A, B, alpha, g, dy, t=None, need_dx=True, dx=None, dA=None, dB=None, ws=None):
    """QA-LoRA pooled backward (qlora_pooled_bwd). Returns (dx or None, dA [K/g, r] fp32, dB [r, N] fp32)."""
    M, K = x.shape
    _, r = A.shape
    _dev(x, w.dtype, "x", (M, w.K))
    _dev(A, w.dtype, "A", (w.K // g, r))
    _dev(B, w.dtype, "B", (r, w.N))
    _dev(dy, w.dtype, "dy", (M, w.N))
    if t is not None:
        _dev(t, w.dtype, "t", (M, r))
    if need_dx:
        dx = _empty((M, w.K), dtype=w.dtype, device=x.device) if dx is None else \
            _dev(dx, w.dtype, "dx", (M, w.K))
    else:
        dx = None
    dA = _empty((w.K // g, r), dtype=torch.float32, device=x.device) if dA is None else \
        _dev(dA, torch.float32, "dA", (w.K // g, r))
    dB = _empty((r, w.N), dtype=torch.float32, device=x.device) if dB is None else \
        _dev(dB, torch.float32, "dB", (r, w.N))
    wsb, wsn = _ws(int(lib.qlora_pooled_bwd_workspace(M, w.N, w.K, r, g)), x.device, ws)
    st = w.state()
    _check(lib.qlora_pooled_bwd(ctypes.byref(st), _ptr(x), M, _ptr(A), _ptr(B), r, g, float(alpha), _ptr(t), _ptr(dy),
                                _ptr(dx), _ptr(dA), _ptr(dB), _ptr(wsb), wsn, _stream()), "qlora_pooled_bwd")
    return dx, dA, dB


def _dev8(t, dtype, name, shape, cur):
    """_dev, for tensors that have to be on the current device `cur`: all of an int8 call's, which runs on its
    current stream."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != cur or not t.is_contiguous():
        _dev(t, dtype, name)
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{cur}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    return t


def _int8_here(q, name, cur):
    """The state of an Int8Tensor on the current device (its codes and scale are on one device)."""
    if q.codes.get_device() != cur:
        raise ValueError(f"{name}: on {q.codes.device}, but the current device is cuda:{cur}")
    return ctypes.byref(q.state())


def _ws8(nbytes, device, ws, cur):
    """_ws on the current device."""
    if ws is None:
        return (None, 0) if nbytes == 0 else (_empty(nbytes, dtype=torch.uint8, device=device), nbytes)
    if ws.get_device() != cur or not ws.is_contiguous():
        raise ValueError(f"ws: must be a contiguous tensor on cuda:{cur}")
    return _ws(nbytes, device, ws)


def _stream8(cur):
    return c_vp(torch._C._cuda_getCurrentRawStream(cur))


class Int8Tensor:
    """Device-resident int8 codes [rows, cols] with one fp32 scale per row (struct qlora_int8): an 8-bit frozen
    weight [N, K], or activations [M, K] kept in 8 bits for the backward.  dtype (torch.bfloat16 or
    torch.float16) is the 16-bit format of the tensors it is used with."""

    def __init__(self, codes, scale, dtype=torch.bfloat16):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        if codes.dim() != 2:
            raise ValueError("codes: expected two dimensions")
        _dev(codes, torch.int8, "codes")
        _dev(scale, torch.float32, "scale", (codes.shape[0],))
        if scale.device != codes.device:
            raise ValueError("codes and scale are on different devices")
        self.codes, self.scale, self.dtype = codes, scale, dtype
        self.rows, self.cols = codes.shape

    @classmethod
    def empty(cls, rows, cols, device="cuda", dtype=torch.bfloat16):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        q = cls.__new__(cls)      # (made here: nothing to check but the device)
        q.codes = _empty((rows, cols), dtype=torch.int8, device=device)
        q.scale = _empty((rows,), dtype=torch.float32, device=device)
        if not q.codes.is_cuda:
            raise ValueError(f"device: must be a GPU, got {device}")
        q.dtype, q.rows, q.cols = dtype, rows, cols
        return q

    def state(self):
        return Int8State(self.codes.data_ptr(), self.scale.data_ptr(), self.rows, self.cols, DTYPES[self.dtype])


def int8_quantize(x, out=None):
    """int8 codes and a scale per row of a bf16 or fp16 [rows, cols] device tensor (qlora_int8_quantize): an
    8-bit weight, or an activation checkpoint.  Returns an Int8Tensor."""
    rows, cols = x.shape
    q = Int8Tensor.empty(rows, cols, x.device, x.dtype) if out is None else out
    cur = torch.cuda.current_device()
    _dev8(x, q.dtype, "x", (q.rows, q.cols), cur)
    _check(lib.qlora_int8_quantize(_ptr(x), _int8_here(q, "out", cur), _stream8(cur)), "qlora_int8_quantize")
    return q


def int8_dequantize(q, out=None):
    """The 16-bit [rows, cols] tensor that the codes stand for (qlora_int8_dequantize)."""
    cur = torch.cuda.current_device()
    st = _int8_here(q, "q", cur)
    o = _empty((q.rows, q.cols), dtype=q.dtype, device=q.codes.device) if out is None else out
    _dev8(o, q.dtype, "out", (q.rows, q.cols), cur)
    _check(lib.qlora_int8_dequantize(st, _ptr(o), _stream8(cur)), "qlora_int8_dequantize")
    return o


def _int8_branch(w, A, B, cur):
    """Rank of the LoRA branch of an int8 layer, 0 when there is none (A and B None)."""
    if A is None and B is None:
        return 0
    if A is None or B is None:
        raise ValueError("A and B: both or neither")
    r = A.shape[1]
    if r == 0:
        raise ValueError("A and B of rank 0: pass None for a layer without a LoRA branch")
    _dev8(A, w.dtype, "A", (w.cols, r), cur)
    _dev8(B, w.dtype, "B", (r, w.rows), cur)
    return r


def int8_linear_fwd(w, x, A=None, B=None, alpha=0.0, y=None, t=None, want_t=True, keep=None, ws=None, dropout=None):
    """y = sx sw (xq wq^T) + (alpha/r)(x A) B of an int8 weight (qlora_int8_linear_fwd); A = B = None: the int8
    product alone.  keep: an Int8Tensor [M, K] that receives x in 8 bits for the backward.  Returns (y, t or
    None).  With a Dropout the branch takes drop(x) for x (qlora_lora_down_batch_dropout, qlora_int8_quantize,
    qlora_int8_gemm_fwd), and the backward needs the 16-bit x (lora_grads_batch): the gradients from an 8-bit
    checkpoint apply no mask, so keep is refused.  A Dropout that drops nothing is None."""
    if dropout is not None and (A is None or B is None):
        raise ValueError("dropout: a layer without a LoRA branch has none")
    if dropout is not None and dropout.drops:
        if keep is not None:
            raise ValueError("keep: lora_grads_batch_int8 has no dropout; keep the 16-bit x of a layer that drops")
        M, cur = x.shape[0], torch.cuda.current_device()
        st, r = _int8_here(w, "w", cur), _int8_branch(w, A, B, cur)
        _dev8(x, w.dtype, "x", (M, w.cols), cur)
        if y is not None:
            _dev8(y, w.dtype, "y", (M, w.rows), cur)
        if t is not None:
            _dev8(t, w.dtype, "t", (M, r), cur)
        _here(ws)
        if M:
            _aligned("int8_linear_fwd", x, A, B, y, t)
        # (the product of no rows: its checks of the weight, before t is written)
        none = Int8State(None, None, 0, w.cols, DTYPES[w.dtype])
        _check(lib.qlora_int8_gemm_fwd(st, ctypes.byref(none), None, None, r, None, _stream8(cur)),
               "qlora_int8_gemm_fwd")
        t = lora_down(x, A, alpha, t=t, ws=ws, dropout=dropout)
        return int8_gemm_fwd(w, int8_quantize(x), t, B, y=y), (t if want_t else None)
    M = x.shape[0]
    cur = torch.cuda.current_device()
    st = _int8_here(w, "w", cur)
    r = _int8_branch(w, A, B, cur)
    dev = x.device
    _dev8(x, w.dtype, "x", (M, w.cols), cur)
    y = _empty((M, w.rows), dtype=w.dtype, device=dev) if y is None else _dev8(y, w.dtype, "y", (M, w.rows), cur)
    if r == 0:
        if t is not None:
            raise ValueError("t: a layer without a LoRA branch has none")
    elif t is not None:
        _dev8(t, w.dtype, "t", (M, r), cur)
    elif want_t:
        t = _empty((M, r), dtype=w.dtype, device=dev)
    if keep is not None and (keep.rows, keep.cols, keep.dtype) != (M, w.cols, w.dtype):
        raise ValueError(f"keep: expected [{M}, {w.cols}] of {w.dtype}")
    wsb, wsn = _ws8(int(lib.qlora_int8_fwd_workspace(M, w.rows, w.cols, r)), dev, ws, cur)
    _check(lib.qlora_int8_linear_fwd(st, _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(y), _ptr(t),
                                     None if keep is None else _int8_here(keep, "keep", cur), _ptr(wsb), wsn,
                                     _stream8(cur)), "qlora_int8_linear_fwd")
    return y, t


def int8_gemm_fwd(w, x, t=None, B=None, y=None):
    """y = sx sw (xq wq^T) + t B for x given as an Int8Tensor (qlora_int8_gemm_fwd); t = B = None: the product
    alone."""
    if (t is None) != (B is None):
        raise ValueError("t and B: both or neither")
    if (x.cols, x.dtype) != (w.cols, w.dtype):
        raise ValueError(f"x: expected [M, {w.cols}] of {w.dtype}")
    cur = torch.cuda.current_device()
    sw, sx = _int8_here(w, "w", cur), _int8_here(x, "x", cur)
    r = 0 if t is None else t.shape[1]
    if t is not None:
        _dev8(t, w.dtype, "t", (x.rows, r), cur)
        _dev8(B, w.dtype, "B", (r, w.rows), cur)
    y = _empty((x.rows, w.rows), dtype=w.dtype, device=x.codes.device) if y is None else \
        _dev8(y, w.dtype, "y", (x.rows, w.rows), cur)
    _check(lib.qlora_int8_gemm_fwd(sw, sx, _ptr(t), _ptr(B), r, _ptr(y), _stream8(cur)), "qlora_int8_gemm_fwd")
    return y


def int8_linear_bwd_dx(w, A, B, alpha, dy, u=None, dx=None, ws=None, dropout=None):
    """(u, dx) of the int8 layer for upstream dy (qlora_int8_linear_bwd_dx): u = (alpha/r) dy B^T, kept for
    lora_grads_batch_int8, and dx = dy W + u A^T; A = B = None: (None, dy W).  With the forward's Dropout,
    dy W + drop(u A^T) (qlora_int8_linear_bwd_dx_dropout); u is then for lora_grads_batch with that Dropout."""
    M = dy.shape[0]
    cur = torch.cuda.current_device()
    st = _int8_here(w, "w", cur)
    r = _int8_branch(w, A, B, cur)
    dev = dy.device
    _dev8(dy, w.dtype, "dy", (M, w.rows), cur)
    if r:
        u = _empty((M, r), dtype=w.dtype, device=dev) if u is None else _dev8(u, w.dtype, "u", (M, r), cur)
    elif u is not None:
        raise ValueError("u: a layer without a LoRA branch has none")
    dx = _empty((M, w.cols), dtype=w.dtype, device=dev) if dx is None else _dev8(dx, w.dtype, "dx", (M, w.cols), cur)
    wsb, wsn = _ws8(int(lib.qlora_int8_linear_bwd_dx_workspace(M, w.rows, w.cols, r)), dev, ws, cur)
    if dropout is not None:
        if r == 0:
            raise ValueError("dropout: a layer without a LoRA branch has none")
        _check(lib.qlora_int8_linear_bwd_dx_dropout(st, M, _ptr(A), _ptr(B), r, float(alpha),
                                                    ctypes.byref(dropout.state()), _ptr(dy), _ptr(u), _ptr(dx),
                                                    _ptr(wsb), wsn, _stream8(cur)), "qlora_int8_linear_bwd_dx_dropout")
        return u, dx
    _check(lib.qlora_int8_linear_bwd_dx(st, M, _ptr(A), _ptr(B), r, float(alpha), _ptr(dy), _ptr(u), _ptr(dx),
                                        _ptr(wsb), wsn, _stream8(cur)), "qlora_int8_linear_bwd_dx")
    return u, dx


def int8_gemm_bwd_dx(w, dy, u=None, A=None, dx=None, dropout=None):
    """dx = dy W + u A^T of an int8 weight, u given (qlora_int8_gemm_bwd_dx); u = A = None: dy W alone.  With a
    Dropout, dy W + drop(u A^T) (qlora_int8_gemm_bwd_dx_dropout)."""
    if (u is None) != (A is None):
        raise ValueError("u and A: both or neither")
    M = dy.shape[0]
    r = 0 if u is None else u.shape[1]
    cur = torch.cuda.current_device()
    st = _int8_here(w, "w", cur)
    _dev8(dy, w.dtype, "dy", (M, w.rows), cur)
    if u is not None:
        _dev8(u, w.dtype, "u", (M, r), cur)
        _dev8(A, w.dtype, "A", (w.cols, r), cur)
    dx = _empty((M, w.cols), dtype=w.dtype, device=dy.device) if dx is None else \
        _dev8(dx, w.dtype, "dx", (M, w.cols), cur)
    if dropout is not None:
        if r == 0:
            raise ValueError("dropout: a layer without a LoRA branch has none")
        _check(lib.qlora_int8_gemm_bwd_dx_dropout(st, _ptr(dy), M, _ptr(u), _ptr(A), r, ctypes.byref(dropout.state()),
                                                  _ptr(dx), _stream8(cur)), "qlora_int8_gemm_bwd_dx_dropout")
        return dx
    _check(lib.qlora_int8_gemm_bwd_dx(st, _ptr(dy), M, _ptr(u), _ptr(A), r, _ptr(dx), _stream8(cur)),
           "qlora_int8_gemm_bwd_dx")
    return dx


def lora_grads_batch_int8(layers, dA=None, dB=None, ws=None):
    """lora_grads_batch with each layer's x as its 8-bit checkpoint (qlora_lora_grads_batch_int8).  layers: a list
    of (x, t, u, dy), x an Int8Tensor, all of one rank and one dtype; dA, dB: optional lists of output tensors.
    No layer among them drops anything: lora_grads_batch takes those, with their 16-bit x.  Returns the lists
    (dA, dB), fp32."""
    n = len(layers)
    if n == 0:
        return [], []
    dt = layers[0][0].dtype
    r = layers[0][1].shape[1]
    dA = [None] * n if dA is None else list(dA)
    dB = [None] * n if dB is None else list(dB)
    if len(dA) != n or len(dB) != n:
        raise ValueError("dA and dB: one tensor per layer")
    cur = torch.cuda.current_device()
    descs = (LoraGradsInt8 * n)()
    for i, (x, t, u, dy) in enumerate(layers):
        if x.dtype != dt:
            raise TypeError(f"x: expected {dt}, got {x.dtype}")
        M, K = x.rows, x.cols
        N = dy.shape[1]
        if x.codes.get_device() != cur:
            _int8_here(x, "x", cur)      # (raises)
        _dev8(t, dt, "t", (M, r), cur)
        _dev8(u, dt, "u", (M, r), cur)
        _dev8(dy, dt, "dy", (M, N), cur)
        dev = dy.device
        dA[i] = _empty((K, r), dtype=torch.float32, device=dev) if dA[i] is None else \
            _dev8(dA[i], torch.float32, "dA", (K, r), cur)
        dB[i] = _empty((r, N), dtype=torch.float32, device=dev) if dB[i] is None else \
            _dev8(dB[i], torch.float32, "dB", (r, N), cur)
        descs[i] = LoraGradsInt8(x.codes.data_ptr(), x.scale.data_ptr(), t.data_ptr(), u.data_ptr(), dy.data_ptr(),
                                 dA[i].data_ptr(), dB[i].data_ptr(), M, N, K)
    wsb, wsn = _ws8(int(lib.qlora_lora_grads_batch_int8_workspace(descs, n, r)), dev, ws, cur)
    _check(lib.qlora_lora_grads_batch_int8(descs, n, r, DTYPES[dt], _ptr(wsb), wsn, _stream8(cur)),
           "qlora_lora_grads_batch_int8")
    return dA, dB


FP8_BLOCK = 128


class Fp8Tensor:
    """Device-resident e4m3 codes [rows, cols] with a power-of-two scale byte for each block (struct qlora_fp8): an
    8-bit frozen weight [N, K] (block_rows 128), or activations (block_rows 1).  codes is torch.float8_e4m3fn, scale
    torch.uint8 (E8M0) of scale_shape(rows, cols, block_rows).  dtype (torch.bfloat16 or torch.float16) is the 16-bit
    format of the tensors it is used with."""

    def __init__(self, codes, scale, dtype=torch.bfloat16, block_rows=FP8_BLOCK):
        if codes.dim() != 2:
            raise ValueError("codes: expected two dimensions")
        _fp8_args(dtype, block_rows)
        _dev(codes, torch.float8_e4m3fn, "codes")
        _dev(scale, torch.uint8, "scale", self.scale_shape(*codes.shape, block_rows))
        if scale.device != codes.device:
            raise ValueError("codes and scale are on different devices")
        self.codes, self.scale, self.dtype, self.block_rows = codes, scale, dtype, block_rows
        self.rows, self.cols = codes.shape

    @staticmethod
    def scale_shape(rows, cols, block_rows=FP8_BLOCK):
        """Shape of the scale bytes: [row of blocks, block] of a weight, [block, row] of activations, the last
        dimension rounded up to a multiple of 4."""
        blocks = -(-cols // FP8_BLOCK)
        if block_rows == 1:
            return blocks, -(-rows // 4) * 4
        return -(-rows // FP8_BLOCK), -(-blocks // 4) * 4

    @classmethod
    def empty(cls, rows, cols, device="cuda", dtype=torch.bfloat16, block_rows=FP8_BLOCK):
        _fp8_args(dtype, block_rows)
        q = cls.__new__(cls)      # (made here: nothing to check but the device)
        q.codes = _empty((rows, cols), dtype=torch.float8_e4m3fn, device=device)
        q.scale = _empty(cls.scale_shape(rows, cols, block_rows), dtype=torch.uint8, device=device)
        if not q.codes.is_cuda:
            raise ValueError(f"device: must be a GPU, got {device}")
        q.dtype, q.block_rows, q.rows, q.cols = dtype, block_rows, rows, cols
        return q

    def state(self):
        return Fp8State(self.codes.data_ptr(), self.scale.data_ptr(), self.rows, self.cols, DTYPES[self.dtype],
                        self.block_rows)


def _fp8_args(dtype, block_rows):
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK}, got {block_rows}")


def _fp8_quantize(x, out, block_rows):
    rows, cols = x.shape
    q = Fp8Tensor.empty(rows, cols, x.device, x.dtype, block_rows) if out is None else out
    if q.block_rows != block_rows:
        raise ValueError(f"out: expected block_rows {block_rows}, got {q.block_rows}")
    cur = torch.cuda.current_device()
    _dev8(x, q.dtype, "x", (q.rows, q.cols), cur)
    _check(lib.qlora_fp8_quantize(_ptr(x), _int8_here(q, "out", cur), _stream8(cur)), "qlora_fp8_quantize")
    return q


def fp8_quantize(W, out=None):
    """e4m3 codes and a power-of-two scale for each 128 x 128 block of a bf16 or fp16 [N, K] device weight
    (qlora_fp8_quantize).  Returns an Fp8Tensor."""
    return _fp8_quantize(W, out, FP8_BLOCK)


def fp8_quantize_rows(x, out=None):
    """The same for activations [M, K], in blocks of 128 along each row: the x of fp8_gemm_fwd."""
    return _fp8_quantize(x, out, 1)


def fp8_dequantize(q, out=None):
    """The 16-bit [rows, cols] tensor that the codes stand for (qlora_fp8_dequantize)."""
    cur = torch.cuda.current_device()
    st = _int8_here(q, "q", cur)
    o = _empty((q.rows, q.cols), dtype=q.dtype, device=q.codes.device) if out is None else out
    _dev8(o, q.dtype, "out", (q.rows, q.cols), cur)
    _check(lib.qlora_fp8_dequantize(st, _ptr(o), _stream8(cur)), "qlora_fp8_dequantize")
    return o


def _fp8_weight(w, cur):
    if w.block_rows != FP8_BLOCK:
        raise ValueError(f"w: expected a weight (block_rows {FP8_BLOCK})")
    return _int8_here(w, "w", cur)


def _drop_ref(dropout, r):
    if dropout is None:
        return None
    if r == 0:
        raise ValueError("dropout: a layer without a LoRA branch has none")
    return ctypes.byref(dropout.state())


def fp8_linear_fwd(w, x, A=None, B=None, alpha=0.0, y=None, t=None, want_t=True, ws=None, dropout=None):
    """y = xq Wq^T + (alpha/r)(x A) B of an fp8 weight, xq the 8-bit x (qlora_fp8_linear_fwd); A = B = None: the fp8
    product alone.  With a Dropout the branch takes drop(x) for x.  Returns (y, t or None)."""
    M = x.shape[0]
    cur = torch.cuda.current_device()
    st = _fp8_weight(w, cur)
    r = _int8_branch(w, A, B, cur)
    drop = _drop_ref(dropout, r)
    dev = x.device
    _dev8(x, w.dtype, "x", (M, w.cols), cur)
    y = _empty((M, w.rows), dtype=w.dtype, device=dev) if y is None else _dev8(y, w.dtype, "y", (M, w.rows), cur)
    if r == 0:
        if t is not None:
            raise ValueError("t: a layer without a LoRA branch has none")
    elif t is not None:
        _dev8(t, w.dtype, "t", (M, r), cur)
    elif want_t:
        t = _empty((M, r), dtype=w.dtype, device=dev)
    wsb, wsn = _ws8(int(lib.qlora_fp8_fwd_workspace(M, w.rows, w.cols, r)), dev, ws, cur)
    _check(lib.qlora_fp8_linear_fwd(st, _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), drop, _ptr(y), _ptr(t), _ptr(wsb),
                                    wsn, _stream8(cur)), "qlora_fp8_linear_fwd")
    return y, t


def fp8_gemm_fwd(w, x, t=None, B=None, y=None):
    """y = xq Wq^T + t B for x given as an Fp8Tensor of block_rows 1 (qlora_fp8_gemm_fwd), for layers that share it;
    t = B = None: the product alone."""
    if (t is None) != (B is None):
        raise ValueError("t and B: both or neither")
    if (x.cols, x.dtype, x.block_rows) != (w.cols, w.dtype, 1):
        raise ValueError(f"x: expected [M, {w.cols}] of {w.dtype} in blocks of one row")
    cur = torch.cuda.current_device()
    sw, sx = _fp8_weight(w, cur), _int8_here(x, "x", cur)
    r = 0 if t is None else t.shape[1]
    if t is not None:
        if r == 0:
            raise ValueError("t and B of rank 0: pass None for a layer without a LoRA branch")
        _dev8(t, w.dtype, "t", (x.rows, r), cur)
        _dev8(B, w.dtype, "B", (r, w.rows), cur)
    y = _empty((x.rows, w.rows), dtype=w.dtype, device=x.codes.device) if y is None else \
        _dev8(y, w.dtype, "y", (x.rows, w.rows), cur)
    _check(lib.qlora_fp8_gemm_fwd(sw, sx, _ptr(t), _ptr(B), r, _ptr(y), _stream8(cur)), "qlora_fp8_gemm_fwd")
    return y


def fp8_linear_bwd_dx(w, A, B, alpha, dy, u=None, dx=None, ws=None, dropout=None):
    """(u, dx) of the fp8 layer for upstream dy (qlora_fp8_linear_bwd_dx): u = (alpha/r) dy B^T, kept for
    lora_grads_batch, and dx = dyq Wq + u A^T, dyq the 8-bit dy; with the forward's Dropout dyq Wq + drop(u A^T).
    A = B = None: (None, dyq Wq)."""
    M = dy.shape[0]
    cur = torch.cuda.current_device()
    st = _fp8_weight(w, cur)
    r = _int8_branch(w, A, B, cur)
    drop = _drop_ref(dropout, r)
    dev = dy.device
    _dev8(dy, w.dtype, "dy", (M, w.rows), cur)
    if r:
        u = _empty((M, r), dtype=w.dtype, device=dev) if u is None else _dev8(u, w.dtype, "u", (M, r), cur)
    elif u is not None:
        raise ValueError("u: a layer without a LoRA branch has none")
    dx = _empty((M, w.cols), dtype=w.dtype, device=dev) if dx is None else _dev8(dx, w.dtype, "dx", (M, w.cols), cur)
    wsb, wsn = _ws8(int(lib.qlora_fp8_linear_bwd_dx_workspace(M, w.rows, w.cols, r)), dev, ws, cur)
    _check(lib.qlora_fp8_linear_bwd_dx(st, M, _ptr(A), _ptr(B), r, float(alpha), drop, _ptr(dy), _ptr(u), _ptr(dx),
                                       _ptr(wsb), wsn, _stream8(cur)), "qlora_fp8_linear_bwd_dx")
    return u, dx


def declared_symbols():
    """Function names declared in include/qlora.h (for the export check)."""
    import re
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(qlora_[a-z0-9_]+)\s*\(", text)))
