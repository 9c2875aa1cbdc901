"""Measured cases of the expert (grouped) QLoRA linear and the 8-bit integer linear.

Four operators:

grouped_fwd    y_i = x_i W'_e^T + s (x_i A_e^T) B_e^T (+ bias_e) for the rows i of expert e, the rows sorted by expert and
               cut by `offsets`; W' the NF4 base of a stack of experts; T = s x A^T is returned too
grouped_bwd    its adapter backward for L = sum(dy * y): dA_e, dB_e (zero for an expert without rows) and dx
int8_quantize  one scale a row, scale = max|x| / 127, codes = x / scale rounded to the nearest integer, ties to even
int8_linear    y = (codes_x codes_w^T) * scale_x (per token) * scale_w (per channel) (+ bias), x quantized in the call

`run` gives each in its plain form (elementary torch operations) or, with `own` set, through this library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# The sixteen NF4 levels (normal quantiles with an exact zero), as fp32 bit patterns.
LEVEL_BITS = (0xbf800000, 0xbf3239b1, 0xbf066b2e, 0xbeca329e, 0xbe91a24b, 0xbe3d353d, 0xbdba7869, 0x00000000,
              0x3da2fb01, 0x3e24cadf, 0x3e7c04da, 0x3ead0336, 0x3ee1a4b5, 0x3f1007a9, 0x3f3913b0, 0x3f800000)


def _levels(device):
    bits = [b - (1 << 32) if b >= 1 << 31 else b for b in LEVEL_BITS]
    return torch.tensor(bits, dtype=torch.int32, device=device).view(torch.float32)


# ------------------------------------------------------------------ cases


def listed():
    grouped = dict(block=64, double_quant=True, bias=False, pad=0, skew=0.5)
    return [
        # one token routed to two of eight experts: the serving step where latency counts
        dict(name="experts fwd 1 token", op="grouped_fwd", dtype="bf16", m=2, e=8, n=4096, k=4096, r=16, **grouped),
        # a serving batch: sixteen tokens to two experts each, the 4-bit weights of every expert streamed once
        dict(name="experts fwd 16 tokens", op="grouped_fwd", dtype="bf16", m=32, e=8, n=11008, k=4096, r=16, **grouped),
        # a short prompt over odd-sized experts in f16, with bias, unused rows behind the last expert, plain fp32 scales
        dict(name="experts fwd ragged f16", op="grouped_fwd", dtype="f16", m=1499, e=16, n=1032, k=1088, r=24, block=64,
             double_quant=False, bias=True, pad=37, skew=1.0),
        # a training or prefill batch: 4096 tokens to two of eight gate_proj-like experts
        dict(name="experts fwd 4096 tokens", op="grouped_fwd", dtype="bf16", m=8192, e=8, n=11008, k=4096, r=64, **grouped),
        # the backward of a training batch: 2048 tokens to two of eight down_proj-like experts
        dict(name="experts bwd 2048 tokens", op="grouped_bwd", dtype="bf16", m=4096, e=8, n=4096, k=11008, r=64, **grouped),
        # many small experts, unevenly filled, some of them empty
        dict(name="experts bwd 64 small f16", op="grouped_bwd", dtype="f16", m=4001, e=64, n=1024, k=2048, r=16, block=128,
             double_quant=False, bias=False, pad=0, skew=1.5),
        # the fp32 reference mode on a small stack
        dict(name="experts bwd f32", op="grouped_bwd", dtype="f32", m=301, e=4, n=512, k=512, r=8, **grouped),
        # activations of a serving step
        dict(name="int8 quantize 16 tokens", op="int8_quantize", dtype="bf16", m=16, k=4096),
        # a merged weight brought to 8 bits, one scale an output channel
        dict(name="int8 quantize weight f32", op="int8_quantize", dtype="f32", m=11008, k=4096),
        # single-token serving
        dict(name="int8 linear 1 token", op="int8_linear", dtype="bf16", m=1, n=4096, k=4096, bias=False),
        # a short prompt on odd sizes
        dict(name="int8 linear odd f16", op="int8_linear", dtype="f16", m=333, n=1000, k=2064, bias=True),
        # a long prompt on the gate_proj-like layer
        dict(name="int8 linear 4096 tokens", op="int8_linear", dtype="bf16", m=4096, n=11008, k=4096, bias=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step or step))


def draw(rng):
    op = rng.choice(("grouped_fwd", "grouped_bwd", "int8_quantize", "int8_linear"))
    if op == "int8_quantize":
        return dict(op=op, dtype=rng.choice(("bf16", "f16", "f32")), m=_log(rng, 1, 8192), k=_log(rng, 16, 8192, 1))
    if op == "int8_linear":
        c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), m=_log(rng, 1, 4096), n=_log(rng, 64, 8192, 8),
                 k=_log(rng, 64, 8192, 16), bias=rng.random() < 0.3)
        return c
    dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
    small = dtype == "f32"
    n = _log(rng, 128, 1024 if small else 8192, 8)
    k = _log(rng, 64, 1024 if small else 8192, 64)
    e = _log(rng, 1, max(1, min(64, 300_000_000 // (n * k))))
    m = _log(rng, 1, 512 if small else min(6000, max(1, 150_000_000_000 // (n * k))))
    return dict(op=op, dtype=dtype, m=m, e=e, n=n, k=k, r=8 * rng.randint(1, 16), block=rng.choice((64, 64, 128, 256)),
                double_quant=rng.random() < 0.5, bias=op == "grouped_fwd" and rng.random() < 0.3,
                pad=rng.choice((0, 0, rng.randint(1, 40))), skew=rng.choice((0.0, 0.5, 1.0)))


# ------------------------------------------------------------------ inputs


def _nf4(n_rows, k, block, double_quant, gen, device):
    """codes, absmax, absmax_q, absmax_scale of a random N(0, 0.02^2) weight, quantized in plain torch."""
    lv = _levels(device)
    mid = (lv[1:] + lv[:-1]) * 0.5
    numel = n_rows * k
    blocks = -(-numel // block)
    codes = torch.empty(blocks * block, dtype=torch.uint8, device=device)
    absmax = torch.empty(blocks, dtype=torch.float32, device=device)
    step = max(1, (1 << 26) // block)
    for b in range(0, blocks, step):
        w = torch.randn(min(step, blocks - b) * block, generator=gen, device=device) * 0.02
        at = b * block + torch.arange(w.numel(), device=device)
        w = torch.where(at < numel, w, torch.zeros_like(w)).view(-1, block)
        am = w.abs().amax(1)
        absmax[b:b + am.numel()] = am
        codes[b * block:b * block + w.numel()] = torch.bucketize((w / am[:, None]).reshape(-1), mid, out_int32=True).to(torch.uint8)
    codes = codes[:numel].view(-1, 2)
    codes = (codes[:, 0] << 4) | codes[:, 1]
    if not double_quant:
        return codes.contiguous(), absmax, None, None
    scale = absmax.amax().reshape(1) / 255.0
    return codes.contiguous(), None, torch.round(absmax / scale).clamp(0, 255).to(torch.uint8), scale


def _counts(case, seed):
    """Rows of each expert: `m` rows routed by uneven probabilities."""
    rng = random.Random("counts %d" % seed)
    p = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(case["e"])]
    counts = [0] * case["e"]
    for i in rng.choices(range(case["e"]), weights=p, k=case["m"]):
        counts[i] += 1
    return counts


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, sigma=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * sigma).to(dt)

    m, k = case["m"], case["k"]
    s = dict(case=case, dt=dt)
    if case["op"] == "int8_quantize":
        # weights are near normal, activations have a few large channels
        s["x"] = randn(m, k, sigma=0.02) if case["dtype"] == "f32" else randn(m, k) * (1 + 9 * (torch.rand(k, generator=gen, device=dev) < 0.01)).to(dt)
        return s
    if case["op"] == "int8_linear":
        n = case["n"]
        s["x"] = randn(m, k)
        s["w_scale"] = (torch.rand(n, generator=gen, device=dev) + 0.5) * (0.08 / 127)
        s["w_codes"] = (torch.randn((n, k), generator=gen, device=dev) * 32).round().clamp(-127, 127).to(torch.int8)
        s["bias"] = randn(n, sigma=0.1) if case["bias"] else None
        return s
    e, n, r = case["e"], case["n"], case["r"]
    counts = _counts(case, seed)
    rows = m + case["pad"]
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    s["cap"] = max(counts)
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    s["alpha"] = 2.0 * r
    s["w"] = _nf4(e * n, k, case["block"], case["double_quant"], gen, dev)
    s["x"] = randn(rows, k)
    s["A"] = randn(e, r, k, sigma=1 / math.sqrt(k))
    s["B"] = randn(e, n, r, sigma=0.01)
    s["bias"] = randn(e, n, sigma=0.1) if case["bias"] else None
    if case["op"] == "grouped_fwd":
        s["y"] = torch.zeros((rows, n), dtype=dt, device=dev)
        s["t"] = torch.zeros((rows, r), dtype=dt, device=dev)
    else:
        s["dy"] = randn(rows, n)
        s["t"] = randn(rows, r, sigma=2.0)  # the forward's saved T = s x A^T, of this size
        s["dx"] = torch.zeros((rows, k), dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------ the plain forms


def _base(s):
    """The dequantized stack [E, N, K], rounded to the compute type, in fp32."""
    c = s["case"]
    codes, absmax, absmax_q, absmax_scale = s["w"]
    scale = absmax if absmax is not None else absmax_q.float() * absmax_scale
    idx = torch.stack((codes >> 4, codes & 15), 1).reshape(-1).to(torch.int32)
    w = _levels(codes.device)[idx]
    if w.numel() % c["block"] == 0:
        w = (w.view(-1, c["block"]) * scale[:, None]).view(-1)
    else:
        w = w * scale[torch.arange(w.numel(), device=w.device) // c["block"]]
    return w.to(s["dt"]).float().view(c["e"], c["n"], c["k"])


def _by_expert(s):
    """Row numbers [E, cap] of every expert's rows, with a mask; and for every row its expert, place and validity."""
    off = s["offsets"].long()
    rows = s["x"].shape[0]
    at = off[:-1, None] + torch.arange(s["cap"], device=off.device)
    there = at < off[1:, None]
    row = torch.arange(rows, device=off.device)
    expert = torch.searchsorted(off[1:], row, right=True).clamp(max=off.numel() - 2)
    return at.clamp(max=rows - 1), there, expert, row - off[expert], (row >= off[0]) & (row < off[-1])


def _gather(v, at, there):
    return torch.where(there[..., None], v[at].float(), torch.zeros((), device=v.device))


def _back(v, into, expert, place, used):
    """v [E, cap, :] to rows; rows of no expert stay as they were."""
    got = v[expert, place.clamp(0, v.shape[1] - 1)].to(into.dtype)
    return torch.where(used[:, None], got, into)


def _plain_fwd(s):
    scale = s["alpha"] / s["case"]["r"]
    at, there, expert, place, used = _by_expert(s)
    x = _gather(s["x"], at, there)
    t = scale * torch.bmm(x, s["A"].float().transpose(1, 2))
    y = torch.bmm(x, _base(s).transpose(1, 2)) + torch.bmm(t, s["B"].float().transpose(1, 2))
    if s["bias"] is not None:
        y = y + s["bias"].float()[:, None]
    return {"y": _back(y, s["y"], expert, place, used), "t": _back(t, s["t"], expert, place, used)}


def _plain_bwd(s):
    scale = s["alpha"] / s["case"]["r"]
    at, there, expert, place, used = _by_expert(s)
    x, dy, t = (_gather(s[v], at, there) for v in ("x", "dy", "t"))
    u = scale * torch.bmm(dy, s["B"].float())
    dx = torch.bmm(dy, _base(s)) + torch.bmm(u, s["A"].float())
    return {"dA": torch.bmm(u.transpose(1, 2), x), "dB": torch.bmm(dy.transpose(1, 2), t),
            "dx": _back(dx, s["dx"], expert, place, used)}


def _plain_quantize(x):
    """(codes, scale): both quotients in 64 bits (half of the largest value lies next to 63.5 steps)."""
    x = x.float()
    scale = (x.abs().amax(1).double() / 127.0).float()
    q = torch.where(scale[:, None] > 0, x.double() / scale.double()[:, None], torch.zeros((), dtype=torch.float64, device=x.device))
    return q.round().clamp(-127, 127).to(torch.int8), scale


def _plain_int8(s):
    codes, scale = _plain_quantize(s["x"])
    y = codes.float() @ s["w_codes"].float().t()
    y = y * scale[:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dt"])


# ------------------------------------------------------------------ run


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from qlora_linear_layers_nf4_b200 import nf4qlora as Q
        if op == "int8_quantize":
            q = Q.int8_quantize(s["x"])
            return {"values": q.codes * q.scale[:, None], "scale": q.scale}
        if op == "int8_linear":
            return Q.int8_linear_fwd(Q.Int8Matrix(s["w_codes"], s["w_scale"]), s["x"], bias=s["bias"])
        codes, absmax, absmax_q, absmax_scale = s["w"]
        q = Q.QuantizedWeight(codes, absmax, absmax_q, absmax_scale, c["e"] * c["n"], c["k"], c["block"], c["double_quant"])
        if op == "grouped_fwd":
            y, t = Q.grouped_fwd(q, s["x"], s["offsets"], s["A"], s["B"], s["alpha"], bias=s["bias"], out=s["y"], t_out=s["t"])
            return {"y": y, "t": t}
        d_a, d_b, dx = Q.grouped_bwd(q, s["x"], s["offsets"], s["A"], s["B"], s["alpha"], s["dy"], t=s["t"], dx=s["dx"])
        return {"dA": d_a, "dB": d_b, "dx": dx}
    if op == "int8_quantize":
        codes, scale = _plain_quantize(s["x"])
        return {"values": codes * scale[:, None], "scale": scale}
    if op == "int8_linear":
        return _plain_int8(s)
    return _plain_fwd(s) if op == "grouped_fwd" else _plain_bwd(s)


# ------------------------------------------------------------------ the work of one pass


def work(case):
    m, k = case["m"], case["k"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "int8_quantize":
        return {"bytes": m * k * (size + 1) + 4 * m, "flops": 2 * m * k}
    n = case["n"]
    if case["op"] == "int8_linear":
        return {"bytes": m * k * size + n * k + 4 * n + m * n * size, "flops": 2 * m * n * k}
    e, r = case["e"], case["r"]
    live = min(e, m)  # experts that have a row, at most
    weight = live * n * k // 2 + live * n * k // case["block"] * (1 if case["double_quant"] else 4)
    adapters = live * r * (n + k) * size
    if case["op"] == "grouped_fwd":
        return {"bytes": weight + adapters + m * (k + n + r) * size, "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    return {"bytes": weight + adapters + m * (2 * k + n + r) * size + e * r * (n + k) * 4,
            "flops": 2 * m * n * k + 6 * m * r * (n + k) - 2 * m * r * k}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("int8_quantize", "int8_linear"):
        x = s["x"].to(f64)
        top = x.abs().max(dim=1).values
        scale = (top / 127).to(torch.float32).to(f64)  # the scale is kept in fp32, and the codes go by it
        live = scale > 0
        codes = torch.zeros_like(x)
        codes[live] = torch.round(x[live] / scale[live].unsqueeze(1)).clamp(-127, 127)
        if case["op"] == "int8_quantize":
            return {"values": codes * scale.unsqueeze(1), "scale": scale}
        y = (codes * scale.unsqueeze(1)) @ (s["w_codes"].to(f64) * s["w_scale"].to(f64).unsqueeze(1)).T
        return y + s["bias"].to(f64) if s["bias"] is not None else y
    e, n, k, r = (case[v] for v in ("e", "n", "k", "r"))
    codes, absmax, absmax_q, absmax_scale = s["w"]
    two = torch.empty((codes.numel(), 2), dtype=torch.uint8, device=codes.device)
    two[:, 0], two[:, 1] = codes // 16, codes % 16
    two = two.view(e, n * k)
    scale = absmax if absmax is not None else (absmax_q.to(torch.float32) * absmax_scale)
    levels = _levels(codes.device)
    off = s["offsets"].tolist()
    alpha = s["alpha"] / r
    forward = case["op"] == "grouped_fwd"
    out = ({"y": s["y"].to(f64), "t": s["t"].to(f64)} if forward else
           {"dA": torch.zeros((e, r, k), dtype=f64, device=codes.device), "dB": torch.zeros((e, n, r), dtype=f64, device=codes.device), "dx": s["dx"].to(f64)})
    for i in range(e):
        a, b = off[i], off[i + 1]
        if a == b:
            continue
        first = i * n * k
        element = torch.arange(first, first + n * k, device=codes.device)
        w = levels[two[i].long()] * scale[element.div(case["block"], rounding_mode="floor")]  # one fp32 product,
        w = w.to(s["dt"]).to(f64).view(n, k)  # rounded to the compute type
        A, B, x = s["A"][i].to(f64), s["B"][i].to(f64), s["x"][a:b].to(f64)
        if forward:
            t = alpha * (x @ A.T)
            out["t"][a:b] = t
            out["y"][a:b] = x @ w.T + t @ B.T + (s["bias"][i].to(f64) if s["bias"] is not None else 0)
        else:
            dy = s["dy"][a:b].to(f64)
            u = alpha * (dy @ B)
            out["dA"][i], out["dB"][i] = u.T @ x, dy.T @ s["t"][a:b].to(f64)
            out["dx"][a:b] = dy @ w + u @ A
    return out
