"""The products on FP4 weights: what is measured, over which sizes, and their plain forms.

Four calls, all y = act(S * x W^T + bias) * mul + residual with W[n][k] held
as NVFP4 (E2M1 codes, one E4M3 scale per 16, one float S) or MXFP4 (E2M1
codes, one E8M0 scale per 32):

  linear         x bf16 [m][k]
  linear_group   x bf16, its rows sorted by expert, one weight per expert
  matmul         x FP4 in the same format as the weight (codes + block scales)
  matmul_group   x FP4, sorted by expert

A weight's scales are kept in the 128 x 4 tiled layout, laid out once when the
weight is quantized; an activation's scales are row-major, as its quantizer
writes them at every call.
"""
import math

import numpy as np
import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _case(op, fmt, m, n, k, experts=1, act="none", bias=False, mul=False, residual=False, out="bf16"):
    return {"op": op, "fmt": fmt, "m": m, "n": n, "k": k, "experts": experts, "act": act, "bias": bias,
            "mul": mul, "residual": residual, "out": out}


def listed():
    named = {
        # one token through an attention projection: latency
        "linear 1 token nvfp4": _case("linear", "nvfp4", 1, 4096, 4096),
        # a few concurrent requests through the gate projection, gated by the up projection's output
        "linear 5 tokens mxfp4 gate": _case("linear", "mxfp4", 5, 14336, 4096, act="silu", mul=True),
        # odd sizes, a bias, fp32 out
        "linear 100 tokens odd": _case("linear", "nvfp4", 100, 1001, 1056, act="gelu_tanh", bias=True, out="f32"),
        # a prompt through the gate projection
        "linear 2048 tokens nvfp4 gate": _case("linear", "nvfp4", 2048, 14336, 4096, act="silu", mul=True),
        # decoding with a mixture of experts: most experts see one or two tokens, some none
        "linear_group 48 rows mxfp4": _case("linear_group", "mxfp4", 48, 2048, 4096, experts=32),
        # a prompt's rows over the experts, ragged
        "linear_group 4099 rows nvfp4": _case("linear_group", "nvfp4", 4099, 4096, 2048, experts=16, act="silu", mul=True),
        # a small batch through the down projection, added to the residual stream
        "matmul 16 tokens nvfp4 down": _case("matmul", "nvfp4", 16, 4096, 14336, residual=True),
        # odd sizes
        "matmul 777 tokens odd": _case("matmul", "nvfp4", 777, 1111, 4128, act="gelu", bias=True),
        # a long prompt through the up projection
        "matmul 4096 tokens mxfp4 up": _case("matmul", "mxfp4", 4096, 14336, 4096),
        "matmul_group 33 rows nvfp4": _case("matmul_group", "nvfp4", 33, 1024, 2048, experts=64, bias=True),
        "matmul_group 8192 rows mxfp4": _case("matmul_group", "mxfp4", 8192, 2048, 4096, experts=16, act="relu"),
    }
    return [dict(c, name=name) for name, c in named.items()]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("linear", "linear_group", "matmul", "matmul_group"))
    group = op.endswith("group")
    while True:
        m = _log(rng, 1, 8192)
        n = _log(rng, 64, 16384)
        k = 32 * _log(rng, 1, 512)
        experts = _log(rng, 2, 64) if group else 1
        # at most the work of the largest listed case, and weights that leave room for three states
        if m * n * k <= 4096 * 14336 * 4096 and experts * n * k <= 1 << 29:
            break
    return _case(op, rng.choice(("nvfp4", "mxfp4")), m, n, k, experts, rng.choice(ACTS), rng.random() < 0.5,
                 rng.random() < 0.3, rng.random() < 0.3, rng.choice(("bf16", "bf16", "f32")))


def _counts(case):
    """Rows per expert: skewed, ragged, a quarter of the experts without any; known from the case alone."""
    e, m = case["experts"], case["m"]
    if e == 1:
        return np.array([m])
    share = 1.0 / (1.0 + np.arange(e))**0.5
    share[e - e // 4:] = 0.0
    ends = np.floor(np.cumsum(share) / share.sum() * m + 1e-9).astype(np.int64)
    ends[e - e // 4 - 1:] = m
    return np.diff(np.concatenate([[0], ends]))


def _spare(case):
    """Rows behind the last expert's that the grouped calls leave as they are."""
    return 3 if case["op"].endswith("group") else 0


def _quantized(g, rows, cols, fmt, scale):
    """Codes, block scales and the global scale of heavy-tailed values (Student-t, 4 degrees of freedom)."""
    dev = "cuda"
    z = torch.randn(rows, cols, generator=g, device=dev)
    chi = torch.zeros(rows, cols, device=dev)
    for _ in range(4):
        chi += torch.randn(rows, cols, generator=g, device=dev).square()
    z.mul_(scale).mul_(torch.rsqrt(chi / 4))
    del chi
    block = 16 if fmt == "nvfp4" else 32
    peak = z.abs().view(rows, cols // block, block).amax(2)
    if fmt == "nvfp4":
        s = peak.max() / 1536
        scales = (peak / (6 * s)).clamp(2.0**-9, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        step = scales.view(torch.float8_e4m3fn).float() * s
    else:
        s = torch.ones((), device=dev)
        e = torch.ceil(torch.log2(peak.clamp_min(1e-30) / 6)).clamp(-127, 127)
        scales = (e + 127).to(torch.uint8)
        step = torch.exp2(e)
    z = (z.view(rows, -1, block) / step.unsqueeze(2)).view(rows, cols)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    nib = torch.bucketize(z.abs(), edges).to(torch.uint8) | (z < 0).to(torch.uint8) << 3
    codes = nib[:, 0::2] | nib[:, 1::2] << 4
    return codes.contiguous(), scales.contiguous(), s.reshape(1).float()


def _tiled(scales):
    """Row-major block scales in the 128 x 4 tiled layout (zero-padded), flat."""
    rows, cols = scales.shape
    rt, ct = -(-rows // 128), -(-cols // 4)
    full = torch.zeros(rt * 128, ct * 4, dtype=torch.uint8, device=scales.device)
    full[:rows, :cols] = scales
    return full.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, fmt, m, n, k, e = (case[f] for f in ("op", "fmt", "m", "n", "k", "experts"))
    group, packed = op.endswith("group"), op.startswith("matmul")
    rows = m + _spare(case)
    block = 16 if fmt == "nvfp4" else 32
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s = {"case": dict(case), "dt": dt}
    s["codes"] = torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(e, n, k // block, dtype=torch.uint8, device="cuda")
    s["S"] = torch.empty(e, device="cuda")
    tiled = []
    for i in range(e):
        s["codes"][i], s["scales"][i], s["S"][i:i + 1] = _quantized(g, n, k, fmt, 0.02)
        tiled.append(_tiled(s["scales"][i]))
    s["tiled"] = torch.stack(tiled)
    if packed:
        s["x_codes"], s["x_scales"], s["x_S"] = _quantized(g, rows, k, fmt, 1.0)
    else:
        x = torch.randn(rows, k, generator=g, device="cuda")
        x *= 1 + 9 * (torch.rand(k, generator=g, device="cuda") < 0.01)     # a few loud channels
        s["x"] = x.bfloat16()

    def more(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    s["bias"] = more(e, n) if case["bias"] else None
    s["mul"] = more(rows, n) if case["mul"] else None
    s["residual"] = more(rows, n) if case["residual"] else None
    s["y"] = torch.zeros(rows, n, dtype=dt, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if group:
        counts = np.roll(_counts(case), seed % e)
        ends = np.concatenate([[0], np.cumsum(counts)])
        s["most"] = int(counts.max())
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["expert"] = torch.tensor(np.repeat(np.arange(e), counts), device="cuda")
        s["place"] = torch.tensor(np.arange(m) - ends[:-1].repeat(counts), device="cuda")
    return s


def _values(codes, scales, S, fmt):
    """The values that FP4 codes stand for, in 32 bits."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    if fmt == "nvfp4":
        step = scales.view(torch.float8_e4m3fn).float() * S
    else:
        step = torch.exp2(scales.float() - 127)
    return (grid[nib].unflatten(-1, (scales.shape[-1], -1)) * step.unsqueeze(-1)).flatten(-2)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * 0.5**0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi)**0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain(s):
    case = s["case"]
    fmt, m, group = case["fmt"], case["m"], case["op"].endswith("group")
    w = _values(s["codes"], s["scales"], s["S"].view(-1, 1, 1), fmt)
    x = _values(s["x_codes"], s["x_scales"], s["x_S"], fmt) if "x_codes" in s else s["x"].float()
    if group:
        # every expert's rows padded to the fullest expert's, one batched product, the rows taken back
        at = (s["offsets"][:-1, None] + torch.arange(s["most"], device=x.device)).clamp_max(x.shape[0] - 1)
        z = torch.bmm(x[at], w.transpose(1, 2))[s["expert"], s["place"]]
    else:
        z = x @ w[0].t()
    if s["bias"] is not None:
        z = z + (s["bias"].float()[s["expert"]] if group else s["bias"].float())
    z = _act(z, case["act"])
    if s["mul"] is not None:
        z = z * s["mul"][:m].float()
    if s["residual"] is not None:
        z = z + s["residual"][:m].float()
    y = torch.zeros(s["y"].shape, dtype=s["dt"], device=x.device)
    y[:m] = z.to(s["dt"])
    return y


def _own(s):
    import fp4_post_weight_grid_b200 as fq
    case = s["case"]
    fmt = fq.NVFP4 if case["fmt"] == "nvfp4" else fq.MXFP4
    act = getattr(fq, "ACT_" + case["act"].upper())
    nv = case["fmt"] == "nvfp4"
    extra = {"bias": s["bias"], "act": act, "mul": s["mul"], "residual": s["residual"]}
    S, x_S = (s["S"] if nv else None), (s.get("x_S") if nv else None)
    y, status, op = s["y"], s["status"], case["op"]
    if op == "linear":
        fq.fp4q_linear(fmt, s["x"], s["codes"][0], s["tiled"], S, y, status, **extra)
    elif op == "linear_group":
        fq.fp4q_linear_group(fmt, s["x"], s["offsets"], s["codes"], s["tiled"], S, y, status, **extra)
    elif op == "matmul":
        fq.fp4q_matmul(fmt, s["x_codes"], s["x_scales"], x_S, s["codes"][0], s["tiled"], S, y, status, **extra)
    else:
        fq.fp4q_matmul_group(fmt, s["x_codes"], s["x_scales"], x_S, s["offsets"], s["codes"], s["tiled"], S, y, status,
                             **extra)
    return y


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    m, n, k = case["m"], case["n"], case["k"]
    per = 0.5 + (1 / 16 if case["fmt"] == "nvfp4" else 1 / 32)
    size = 2 if case["out"] == "bf16" else 4
    busy = int((_counts(case) > 0).sum())
    total = busy * n * k * per + m * k * (per if case["op"].startswith("matmul") else 2)
    total += m * n * size * (1 + case["mul"] + case["residual"]) + (busy * n * size if case["bias"] else 0)
    return {"bytes": total, "flops": 2.0 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)

    def decode(codes, scales, S):
        out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device="cuda")
        for half in (0, 1):
            nib = (codes.int() >> (4 * half)) & 15
            e, f = (nib >> 1) & 3, (nib & 1).double()
            mag = torch.where(e == 0, f / 2, torch.ldexp(1 + f / 2, e - 1))
            out[..., half::2] = torch.where(nib > 7, -mag, mag)
        b = scales.int()
        if case["fmt"] == "nvfp4":
            e, f = (b >> 3) & 15, (b & 7).double()
            d = torch.where(e == 0, f / 512, torch.ldexp(1 + f / 8, e - 7)) * S.double()
            return out * d.repeat_interleave(16, -1)
        return torch.ldexp(out, (b - 127).repeat_interleave(32, -1))

    m = case["m"]
    x = decode(s["x_codes"], s["x_scales"], s["x_S"]) if "x_codes" in s else s["x"].double()
    ends = s["offsets"].tolist() if "offsets" in s else [0, m]
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        r = slice(ends[e], ends[e + 1])
        if r.start == r.stop:
            continue
        z = x[r] @ decode(s["codes"][e], s["scales"][e], s["S"][e]).T
        if s["bias"] is not None:
            z += s["bias"][e].double()
        if case["act"] == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "gelu_tanh":
            z = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z**3))
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        if s["mul"] is not None:
            z *= s["mul"][r].double()
        if s["residual"] is not None:
            z += s["residual"][r].double()
        y[r] = z
    return y
