"""Cases for the int8 operators: 8-bit activation checkpoints, the linear layer on an int8 base with its
LoRA branch, its input gradient, and the LoRA weight gradients taken from 8-bit checkpoints.

The format they share: int8 codes [rows, cols] and one fp32 scale per row.  With a = max|x| over the row,
scale = fl32(a / 127) and code = the integer nearest to 127 x / a, ties toward zero (a = 0: both 0).  In a
16-bit compute type a code stands for RNE_16(fl32(scale * code)).

  checkpoint  x [m, k] is stored in 8 bits and restored
  linear      y = sx sw (qx qw^T) + t B,  t = (alpha / r) x A   (r = 0: the product alone)
  dx          u = (alpha / r) dy B^T,  dx = dy W + u A^T,  W the 16-bit values of the int8 weight
  grads       dA = X^T u,  dB = t^T dy  for each layer, X the 16-bit values of the layer's checkpoint
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ALPHA = 16.0


def listed():
    return [
        # a short prompt's activations kept for the backward pass: latency counts
        {"name": "checkpoint short", "kind": "checkpoint", "dtype": "fp16", "m": 77, "k": 4096},
        # the widest activations of the 70B-size MLP, 8192 tokens
        {"name": "checkpoint 70B mlp", "kind": "checkpoint", "dtype": "bf16", "m": 8192, "k": 28672},
        # one token through q_proj of a 7B-size block
        {"name": "linear decode 1", "kind": "linear", "dtype": "bf16", "m": 1, "n": 4096, "k": 4096, "r": 16},
        # a ragged batch of sequences, one token each, through gate or up
        {"name": "linear decode 13", "kind": "linear", "dtype": "fp16", "m": 13, "n": 11008, "k": 4096, "r": 64},
        # one ragged prompt through down_proj
        {"name": "linear ragged", "kind": "linear", "dtype": "bf16", "m": 333, "n": 4096, "k": 11008, "r": 8},
        # a base with its adapter merged: the int8 product alone
        {"name": "linear merged", "kind": "linear", "dtype": "fp16", "m": 1024, "n": 4096, "k": 4096, "r": 0},
        # up_proj over 2048 tokens, rank 64
        {"name": "linear up_proj", "kind": "linear", "dtype": "bf16", "m": 2048, "n": 11008, "k": 4096, "r": 64},
        # gate or up of the 70B-size MLP over 8192 tokens
        {"name": "linear 70B mlp", "kind": "linear", "dtype": "bf16", "m": 8192, "n": 28672, "k": 8192, "r": 64},
        # a short ragged batch's gradient into a layer whose outputs are no whole number of blocks
        {"name": "dx ragged", "kind": "dx", "dtype": "fp16", "m": 777, "n": 11000, "k": 4096, "r": 24},
        # a training step of the 7B-size block, up_proj
        {"name": "dx up_proj", "kind": "dx", "dtype": "bf16", "m": 4096, "n": 11008, "k": 4096, "r": 64},
        # one layer's gradients on a small ragged batch
        {"name": "grads one layer", "kind": "grads", "dtype": "fp16", "m": 500, "n": 11008, "k": 4096, "r": 16,
         "layers": 1},
        # every linear of the 7B-size block at the end of a backward pass
        {"name": "grads 7B block", "kind": "grads", "dtype": "bf16", "m": 4096, "n": 11008, "k": 4096, "r": 64,
         "layers": 7},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    def width(lo, hi):                    # a reduction width: whole blocks of 64
        return 64 * log(max(1, lo // 64), hi // 64)

    def outputs(lo, hi):                  # output widths: most are whole blocks, some are not
        n = log(lo, hi)
        return n if rng.random() < 0.25 else (n + 7) // 8 * 8 if rng.random() < 0.5 else (n + 63) // 64 * 64

    kind = rng.choice(["checkpoint", "linear", "linear", "linear", "dx", "grads"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "checkpoint":
        return {"kind": kind, "dtype": dtype, "m": log(1, 8192), "k": width(64, 28672)}
    if kind == "linear":
        r = rng.choice([0, rng.randint(1, 128), 8, 16, 64])
        m = log(1, 16) if rng.random() < 0.4 else log(17, 8192)
        return {"kind": kind, "dtype": dtype, "m": m, "n": outputs(64, 28672), "k": width(64, 8192), "r": r}
    if kind == "dx":
        return {"kind": kind, "dtype": dtype, "m": log(16, 4096), "n": outputs(64, 11008), "k": width(64, 4096),
                "r": rng.choice([0, rng.randint(1, 128), 16, 64])}
    return {"kind": kind, "dtype": dtype, "m": log(16, 4096), "n": outputs(64, 11008), "k": width(64, 4096),
            "r": rng.choice([rng.randint(1, 64), 8, 16, 64]), "layers": rng.choice([1, 2, 4, 7])}


def layer_shapes(case):
    """(outputs, inputs) of each layer: the attention projections first, then the MLP of a decoder block."""
    n, k = case["n"], case["k"]
    block = [(k, k), (k, k), (k, k), (k, k), (n, k), (n, k)]
    if case["layers"] == 7 and n % 64 == 0:
        return block + [(k, n)]
    return (block + [(n, k)])[-case["layers"]:]


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, sigma, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sigma).to(dtype)

    def activations(m, k):
        """Unit normal, some channels 8 times as large, and in a batch the padding's rows zero."""
        x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float32)
        loud = torch.rand((k,), generator=g, device="cuda") < 0.005
        x = x * torch.where(loud, 8.0, 1.0)
        if m >= 64:
            x[m - m // 32:] = 0.0
        return x.to(dt)

    def int8(m, k, sigma):
        """Codes and scales of a normal matrix, as quantizing it gives."""
        v = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float32).mul_(sigma).to(dt).float()
        return encode(v)

    m, k = case["m"], case["k"]
    state = {"kind": case["kind"], "dtype": dt}
    if case["kind"] == "checkpoint":
        state["x"] = activations(m, k)
        return state
    n, r = case["n"], case["r"]
    state["scale"] = ALPHA / r if r else 0.0
    if case["kind"] == "grads":
        state["layers"] = []
        for no, ni in layer_shapes(case):
            codes, scale = encode(activations(m, ni).float())
            state["layers"].append({"codes": codes, "scale": scale, "t": normal((m, r), 0.5, dt),
                                    "u": normal((m, r), 0.05, dt), "dy": normal((m, no), 0.1, dt)})
        return state
    state["w"], state["ws"] = int8(n, k, 0.02)
    state["A"] = normal((k, r), r ** -0.5, dt) if r else None
    state["B"] = normal((r, n), 0.01, dt) if r else None
    if case["kind"] == "linear":
        state["x"] = activations(m, k)
    else:
        state["dy"] = normal((m, n), 0.1, dt)
    return state


def encode(v):
    """Codes and scales of fp32 rows that hold 16-bit values.  127 v is exact, the quotient is rounded once, and
    it is a half only where the real quotient is one (a 16-bit v and a leave every other quotient further away)."""
    a = v.abs().amax(dim=1, keepdim=True)
    z = 127.0 * v / torch.where(a > 0, a, 1.0)
    return (torch.ceil(z.abs() - 0.5) * torch.sign(z)).to(torch.int8), (a / 127.0).squeeze(1)


def decode(codes, scale, dt):
    """The 16-bit values that codes stand for, as fp32."""
    return (codes.float() * scale[:, None]).to(dt).float()


def run(state):
    return run_own(state) if own else run_plain(state)


def run_plain(state):
    kind, dt = state["kind"], state["dtype"]
    if kind == "checkpoint":
        codes, scale = encode(state["x"].float())
        return {"scale": scale, "x": decode(codes, scale, dt).to(dt)}
    if kind == "grads":
        dA = [decode(e["codes"], e["scale"], dt).t() @ e["u"].float() for e in state["layers"]]
        dB = [e["t"].float().t() @ e["dy"].float() for e in state["layers"]]
        return {"dA": dA, "dB": dB}
    A, B, s = state["A"], state["B"], state["scale"]
    if kind == "linear":
        x = state["x"].float()
        codes, scale = encode(x)
        y = (codes.float() @ state["w"].float().t()) * scale[:, None] * state["ws"][None, :]
        if A is not None:
            y = y + (s * (x @ A.float())) @ B.float()
        return {"y": y.to(dt)}
    dy = state["dy"].float()
    dx = dy @ decode(state["w"], state["ws"], dt)
    if A is None:
        return {"dx": dx.to(dt)}
    u = s * (dy @ B.float().t())
    return {"u": u.to(dt), "dx": (dx + u @ A.float().t()).to(dt)}


def run_own(state):
    from bit_nf4_quantized_15_amd import qlora
    kind, dt = state["kind"], state["dtype"]
    if kind == "checkpoint":
        q = qlora.int8_quantize(state["x"])
        return {"scale": q.scale, "x": qlora.int8_dequantize(q)}
    if kind == "grads":
        dA, dB = qlora.lora_grads_batch_int8(
            [(qlora.Int8Tensor(e["codes"], e["scale"], dt), e["t"], e["u"], e["dy"]) for e in state["layers"]])
        return {"dA": dA, "dB": dB}
    w = qlora.Int8Tensor(state["w"], state["ws"], dt)
    if kind == "linear":
        y, _ = qlora.int8_linear_fwd(w, state["x"], state["A"], state["B"], ALPHA, want_t=False)
        return {"y": y}
    u, dx = qlora.int8_linear_bwd_dx(w, state["A"], state["B"], ALPHA, state["dy"])
    return {"dx": dx} if u is None else {"u": u, "dx": dx}


def work(case):
    m, k = case["m"], case["k"]
    if case["kind"] == "checkpoint":      # x in, codes out and in again, x out, the scales out and in
        return {"bytes": 6 * m * k + 8 * m, "flops": 0}
    n, r = case["n"], case["r"]
    if case["kind"] == "grads":
        b = f = 0
        for no, ni in layer_shapes(case):
            b += m * ni + 4 * m + 2 * m * no + 4 * m * r + 4 * r * (ni + no)
            f += 2 * m * r * (ni + no)
        return {"bytes": b, "flops": f}
    extra = 2 * m * r if case["kind"] == "dx" else 0
    return {"bytes": n * k + 4 * n + 2 * m * (n + k) + 2 * r * (n + k) + extra,
            "flops": 2 * m * n * k + 2 * m * r * (n + k)}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    state = prepare(case, seed)
    dt, f64 = state["dtype"], torch.float64

    def stored(x):
        """Codes and real scales: the nearest integer to 127 |x| / a is the number of halves below it."""
        mag = x.to(f64).abs()
        top = mag.max(dim=1).values
        ratio = mag * 127 / torch.where(top == 0, torch.ones_like(top), top).unsqueeze(1)
        whole = ratio.floor()
        q = torch.where(ratio - whole > 0.5, whole + 1, whole)
        return torch.where(x < 0, -q, q), top / 127

    def values(q, scale):
        """What codes stand for in the 16-bit type: the scale is an fp32 value, the product is rounded to fp32."""
        return (q.to(f64) * scale.to(torch.float32).to(f64).unsqueeze(1)).to(torch.float32).to(dt).to(f64)

    if state["kind"] == "checkpoint":
        q, scale = stored(state["x"])
        return {"scale": scale, "x": values(q, scale)}
    if state["kind"] == "grads":
        out = {"dA": [], "dB": []}
        for e in state["layers"]:
            out["dA"].append(torch.mm(values(e["codes"], e["scale"]).t().contiguous(), e["u"].to(f64)))
            out["dB"].append(torch.mm(e["t"].to(f64).t().contiguous(), e["dy"].to(f64)))
        return out
    A, B, s = state["A"], state["B"], state["scale"]
    if state["kind"] == "linear":
        q, scale = stored(state["x"])
        y = torch.mm(q * scale.unsqueeze(1), (state["w"].to(f64) * state["ws"].to(f64).unsqueeze(1)).t())
        if A is not None:
            y += torch.mm(torch.mm(state["x"].to(f64), A.to(f64)) * s, B.to(f64))
        return {"y": y}
    dy = state["dy"].to(f64)
    dx = torch.mm(dy, values(state["w"], state["ws"]))
    if A is None:
        return {"dx": dx}
    u = torch.mm(dy, B.to(f64).t()) * s
    return {"u": u, "dx": dx + torch.mm(u, A.to(f64).t())}
