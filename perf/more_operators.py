"""Measured cases of the gated feed-forward layer on NF4 weights and of the 8-bit floating point linear.

Five operators:

gated_fwd       g = x W'_g^T + s (x A_g^T) B_g^T (+ bias_g), u = x W'_u^T + s (x A_u^T) B_u^T (+ bias_u), h = act(g) * u;
                W' the NF4 bases, s = alpha / r; what a training step keeps, g and u (`pre`) and T = s x A^T, is returned too
gated_bwd       its adapter backward for L = sum(dh * h) from the saved g, u and T: dg = dh * u * act'(g), du = dh * act(g),
                dA, dB of both projections, and dx
fp8_quantize    e4m3 codes with one scale for each block of 128 columns of a row (tokens) or of 128 x 128 (weights):
                scale = max|x| / 448, codes = the e4m3 value nearest to x / scale, ties to even
fp8_dequantize  codes * scale
fp8_linear      y = sum over blocks of 128 of (codes_x codes_w^T) * scale_x * scale_w (+ bias), x quantized in the call

`run` gives each in its plain form (elementary torch operations) or, with `own` set, through this library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# The sixteen NF4 levels (normal quantiles with an exact zero), as fp32 bit patterns.
LEVEL_BITS = (0xbf800000, 0xbf3239b1, 0xbf066b2e, 0xbeca329e, 0xbe91a24b, 0xbe3d353d, 0xbdba7869, 0x00000000,
              0x3da2fb01, 0x3e24cadf, 0x3e7c04da, 0x3ead0336, 0x3ee1a4b5, 0x3f1007a9, 0x3f3913b0, 0x3f800000)

GELU_C = math.sqrt(2.0 / math.pi)


def _levels(device):
    bits = [b - (1 << 32) if b >= 1 << 31 else b for b in LEVEL_BITS]
    return torch.tensor(bits, dtype=torch.int32, device=device).view(torch.float32)


# ------------------------------------------------------------------ cases


def listed():
    gated = dict(block=64, double_quant=True, bias=False, act="silu")
    return [
        # one token through the gate and up projections of a decoder block: the serving step where latency counts
        dict(name="gated fwd 1 token", op="gated_fwd", dtype="bf16", m=1, n=11008, k=4096, r=16, save=False, **gated),
        # a serving batch of sixteen tokens: both 4-bit weights streamed once
        dict(name="gated fwd 16 tokens", op="gated_fwd", dtype="bf16", m=16, n=11008, k=4096, r=64, save=False, **gated),
        # a short prompt on odd sizes in f16, with biases, plain fp32 scales and the tanh form of GELU
        dict(name="gated fwd odd f16", op="gated_fwd", dtype="f16", m=333, n=1032, k=1088, r=24, save=True, block=64,
             double_quant=False, bias=True, act="gelu_tanh"),
        # the forward of a training batch, which keeps g, u and T
        dict(name="gated fwd 4096 tokens", op="gated_fwd", dtype="bf16", m=4096, n=11008, k=4096, r=64, save=True, **gated),
        # its backward
        dict(name="gated bwd 4096 tokens", op="gated_bwd", dtype="bf16", m=4096, n=11008, k=4096, r=64, **gated),
        # a small layer with a ragged batch in f16
        dict(name="gated bwd odd f16", op="gated_bwd", dtype="f16", m=777, n=2056, k=1088, r=24, block=128,
             double_quant=False, bias=False, act="gelu_tanh"),
        # the fp32 reference mode on a small layer
        dict(name="gated bwd f32", op="gated_bwd", dtype="f32", m=301, n=512, k=512, r=8, **gated),
        # activations of a serving step, and back
        dict(name="fp8 quantize 16 tokens", op="fp8_quantize", dtype="bf16", m=16, k=4096, block_rows=1),
        # a merged weight brought to 8 bits, one scale for 128 x 128, and back
        dict(name="fp8 quantize weight f32", op="fp8_quantize", dtype="f32", m=11008, k=4096, block_rows=128),
        # single-token serving
        dict(name="fp8 linear 1 token", op="fp8_linear", dtype="bf16", m=1, n=4096, k=4096, bias=False),
        # a short prompt on odd sizes: short last blocks on both axes
        dict(name="fp8 linear odd f16", op="fp8_linear", dtype="f16", m=333, n=1000, k=2064, bias=True),
        # a long prompt on the gate_proj-like layer
        dict(name="fp8 linear 4096 tokens", op="fp8_linear", dtype="bf16", m=4096, n=11008, k=4096, bias=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step or step))


def draw(rng):
    op = rng.choice(("gated_fwd", "gated_bwd", "gated_fwd", "gated_bwd", "fp8_quantize", "fp8_linear", "fp8_linear"))
    if op == "fp8_quantize":
        return dict(op=op, dtype=rng.choice(("bf16", "f16", "f32")), m=_log(rng, 1, 8192), k=_log(rng, 16, 5120, 1),
                    block_rows=rng.choice((1, 128)))
    if op == "fp8_linear":
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), m=_log(rng, 1, 4096), n=_log(rng, 64, 8192, 8),
                    k=_log(rng, 64, 8192, 16), bias=rng.random() < 0.3)
    dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
    small = dtype == "f32"
    n = _log(rng, 128, 1024 if small else 9216, 8)
    k = _log(rng, 64, 1024 if small else 4096, 64)
    m = _log(rng, 1, 512 if small else 4096)
    c = dict(op=op, dtype=dtype, m=m, n=n, k=k, r=8 * rng.randint(1, 16), block=rng.choice((64, 64, 128, 256)),
             double_quant=rng.random() < 0.5, bias=op == "gated_fwd" and rng.random() < 0.3,
             act=rng.choice(("silu", "gelu_tanh")))
    if op == "gated_fwd":
        c["save"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs


def _nf4(rows, k, block, double_quant, gen, device):
    """codes, absmax, absmax_q, absmax_scale of a random N(0, 0.02^2) weight, quantized in plain torch."""
    lv = _levels(device)
    mid = (lv[1:] + lv[:-1]) * 0.5
    numel = rows * k
    blocks = -(-numel // block)
    w = torch.randn(blocks * block, generator=gen, device=device) * 0.02
    w[numel:] = 0
    w = w.view(-1, block)
    absmax = w.abs().amax(1)
    codes = torch.bucketize((w / absmax[:, None]).reshape(-1), mid, out_int32=True).to(torch.uint8)[:numel].view(-1, 2)
    codes = ((codes[:, 0] << 4) | codes[:, 1]).contiguous()
    if not double_quant:
        return codes, absmax, None, None
    scale = absmax.amax().reshape(1) / 255.0
    return codes, None, torch.round(absmax / scale).clamp(0, 255).to(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, sigma=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * sigma).to(dt)

    m, k = case["m"], case["k"]
    s = dict(case=case, dt=dt)
    if case["op"] == "fp8_quantize":
        # weights are near normal, activations have a few large channels
        s["x"] = randn(m, k, sigma=0.02) if case["block_rows"] > 1 else randn(m, k) * (1 + 9 * (torch.rand(k, generator=gen, device=dev) < 0.01)).to(dt)
        return s
    n = case["n"]
    if case["op"] == "fp8_linear":
        s["x"] = randn(m, k) * (1 + 9 * (torch.rand(k, generator=gen, device=dev) < 0.01)).to(dt)
        s["w_codes"], s["w_scale"] = _plain_fp8(torch.randn((n, k), generator=gen, device=dev) * 0.02, 128)
        s["bias"] = randn(n, sigma=0.1) if case["bias"] else None
        return s
    r = case["r"]
    s["alpha"] = 2.0 * r
    s["gate"] = _nf4(n, k, case["block"], case["double_quant"], gen, dev)
    s["up"] = _nf4(n, k, case["block"], case["double_quant"], gen, dev)
    s["x"] = randn(m, k)
    s["A"] = randn(2, r, k, sigma=1 / math.sqrt(k))
    s["B"] = randn(2, n, r, sigma=0.01)
    s["bias"] = randn(2, n, sigma=0.1) if case["bias"] else None
    if case["op"] == "gated_bwd":
        s["dh"] = randn(m, n)
        s["pre"] = randn(2, m, n, sigma=0.02 * math.sqrt(k))  # g and u, of the size that such weights give
        s["t"] = randn(2, m, r, sigma=2.0)  # the forward's saved T = s x A^T
    return s


# ------------------------------------------------------------------ the plain forms


def _base(w, case, dt):
    """The dequantized weight [N, K], rounded to the compute type, in fp32."""
    codes, absmax, absmax_q, absmax_scale = w
    scale = absmax if absmax is not None else absmax_q.float() * absmax_scale
    idx = torch.stack((codes >> 4, codes & 15), 1).reshape(-1).to(torch.int32)
    v = _levels(codes.device)[idx]
    if v.numel() % case["block"] == 0:
        v = (v.view(-1, case["block"]) * scale[:, None]).view(-1)
    else:
        v = v * scale[torch.arange(v.numel(), device=v.device) // case["block"]]
    return v.to(dt).float().view(case["n"], case["k"])


def _act(g, act):
    """act(g) and its derivative, in fp32."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    t = torch.tanh(GELU_C * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * g * g)


def _plain_gated_fwd(s):
    c, x = s["case"], s["x"].float()
    A, B = s["A"].float(), s["B"].float()
    scale = s["alpha"] / c["r"]
    t = torch.stack((scale * (x @ A[0].t()), scale * (x @ A[1].t())))
    g = x @ _base(s["gate"], c, s["dt"]).t() + t[0] @ B[0].t()
    u = x @ _base(s["up"], c, s["dt"]).t() + t[1] @ B[1].t()
    if s["bias"] is not None:
        g, u = g + s["bias"][0].float(), u + s["bias"][1].float()
    h = (_act(g, c["act"])[0] * u).to(s["dt"])
    return {"h": h, "pre": torch.stack((g, u)).to(s["dt"]), "t": t.to(s["dt"])} if c["save"] else {"h": h}


def _plain_gated_bwd(s):
    c, x, dh = s["case"], s["x"].float(), s["dh"].float()
    A, B, t = s["A"].float(), s["B"].float(), s["t"].float()
    g, u = s["pre"][0].float(), s["pre"][1].float()
    scale = s["alpha"] / c["r"]
    a, d = _act(g, c["act"])
    dg, du = dh * u * d, dh * a
    v = torch.stack((scale * (dg @ B[0]), scale * (du @ B[1])))
    return {"dA": torch.stack((v[0].t() @ x, v[1].t() @ x)),
            "dB": torch.stack((dg.t() @ t[0], du.t() @ t[1])),
            "dx": (dg @ _base(s["gate"], c, s["dt"]) + du @ _base(s["up"], c, s["dt"]) + v[0] @ A[0] + v[1] @ A[1]).to(s["dt"])}


def _spread(scale, block_rows, rows, cols):
    """The scale of every element."""
    if block_rows > 1:
        scale = scale.repeat_interleave(block_rows, 0)[:rows]
    return scale.repeat_interleave(128, 1)[:, :cols]


def _plain_fp8(x, block_rows):
    """(codes, scale) of x [rows, cols]: both quotients in 64 bits, then in fp32 (halves of a step lie next to them)."""
    x = x.float()
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    pad = torch.nn.functional.pad(x, (0, bc * 128 - cols, 0, br * block_rows - rows))
    scale = (pad.view(br, block_rows, bc, 128).abs().amax((1, 3)).double() / 448.0).float()
    every = _spread(scale, block_rows, rows, cols)
    q = torch.where(every > 0, (x.double() / every.double()).float(), torch.zeros((), device=x.device))
    return q.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _plain_fp8_linear(s):
    codes, scale = _plain_fp8(s["x"], 1)
    m, k = codes.shape
    n = s["w_codes"].shape[0]
    x = codes.float() * _spread(scale, 1, m, k)
    y = x @ (s["w_codes"].float() * _spread(s["w_scale"], 128, n, k)).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dt"])


# ------------------------------------------------------------------ run


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from qlora_linear_layers_nf4_b200 import nf4qlora as Q
        if op == "fp8_quantize":
            q = Q.fp8_quantize(s["x"], block_rows=c["block_rows"])
            return {"values": Q.fp8_dequantize(q), "scale": q.scale}
        if op == "fp8_linear":
            return Q.fp8_linear_fwd(Q.Fp8Matrix(s["w_codes"], s["w_scale"], 128), s["x"], bias=s["bias"])
        gate, up = (Q.QuantizedWeight(*s[w], c["n"], c["k"], c["block"], c["double_quant"]) for w in ("gate", "up"))
        if op == "gated_fwd":
            h, saved = Q.gated_fwd(gate, up, s["x"], s["A"], s["B"], s["alpha"], activation=c["act"], bias=s["bias"],
                                   want_saved=c["save"])
            return {"h": h, "pre": saved.pre, "t": saved.t} if c["save"] else {"h": h}
        d_a, d_b, dx = Q.gated_bwd(gate, up, s["x"], s["A"], s["B"], s["alpha"], s["dh"], Q.GatedSaved(s["pre"], s["t"]),
                                   activation=c["act"])
        return {"dA": d_a, "dB": d_b, "dx": dx}
    if op == "fp8_quantize":
        codes, scale = _plain_fp8(s["x"], c["block_rows"])
        return {"values": codes.float() * _spread(scale, c["block_rows"], c["m"], c["k"]), "scale": scale}
    if op == "fp8_linear":
        return _plain_fp8_linear(s)
    return _plain_gated_fwd(s) if op == "gated_fwd" else _plain_gated_bwd(s)


# ------------------------------------------------------------------ the work of one pass


def work(case):
    m, k = case["m"], case["k"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "fp8_quantize":
        scales = -(-m // case["block_rows"]) * -(-k // 128) * 4
        return {"bytes": m * k * (size + 4) + scales, "flops": 3 * m * k}  # x in, the values and scales out
    n = case["n"]
    if case["op"] == "fp8_linear":
        return {"bytes": m * k * size + n * k + -(-n // 128) * -(-k // 128) * 4 + m * n * size, "flops": 2 * m * n * k}
    r = case["r"]
    weights = 2 * (n * k // 2 + n * k // case["block"] * (1 if case["double_quant"] else 4))
    adapters = 2 * r * (n + k) * size
    if case["op"] == "gated_fwd":
        return {"bytes": weights + adapters + m * (k + n) * size + (2 * m * (n + r) * size if case["save"] else 0),
                "flops": 4 * m * n * k + 4 * m * r * (n + k)}
    return {"bytes": weights + adapters + m * (2 * k + 3 * n + 2 * r) * size + 2 * r * (n + k) * 4,
            "flops": 4 * m * n * k + 8 * m * r * (n + k)}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_act(g, act):
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * (1 - sig)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    th = torch.tanh(inner)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th ** 2) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)


def _exact_fp8(x):
    """(values of the codes, scale of every element's block, block scales) with one scale for 128 columns."""
    f64 = torch.float64
    m, k = x.shape
    bc = (k + 127) // 128
    values, every = torch.zeros((m, k), dtype=f64, device=x.device), torch.zeros((m, k), dtype=f64, device=x.device)
    scales = torch.zeros((m, bc), dtype=f64, device=x.device)
    for b in range(bc):
        block = x[:, b * 128:(b + 1) * 128].to(f64)
        scale = (block.abs().max(dim=1).values / 448).to(torch.float32).to(f64)  # the scale is kept in fp32
        scales[:, b] = scale
        every[:, b * 128:(b + 1) * 128] = scale.unsqueeze(1)
        values[:, b * 128:(b + 1) * 128] = _e4m3(block, scale.unsqueeze(1))
    return values, every, scales


def _e4m3(x, scale):
    """The e4m3 value nearest to the fp32 quotient x / scale, ties to even: three bits after the leading one, from 2^-6 on."""
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x)).to(torch.float32).to(torch.float64)
    exponent = torch.frexp(q)[1].to(torch.float64) - 1
    step = torch.exp2(exponent.clamp(min=-6) - 3)
    return (torch.round(q / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    x = s["x"].to(f64)
    dev = x.device
    if case["op"] == "fp8_quantize":
        if case["block_rows"] == 1:
            values, every, scales = _exact_fp8(s["x"])
            return {"values": values * every, "scale": scales}
        m, k = x.shape
        values = torch.zeros((m, k), dtype=f64, device=dev)
        scales = torch.zeros(((m + 127) // 128, (k + 127) // 128), dtype=f64, device=dev)
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                block = x[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
                scale = (block.abs().max() / 448).to(torch.float32).to(f64)
                scales[i, j] = scale
                values[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = _e4m3(block, scale) * scale
        return {"values": values, "scale": scales}
    n, k = case["n"], case["k"]
    if case["op"] == "fp8_linear":
        values, every, _ = _exact_fp8(s["x"])
        w = s["w_codes"].to(torch.float32).to(f64)
        row, col = torch.arange(n, device=dev) // 128, torch.arange(k, device=dev) // 128
        y = (values * every) @ (w * s["w_scale"].to(f64)[row][:, col]).T
        return y + s["bias"].to(f64) if s["bias"] is not None else y

    def base(w):
        codes, absmax, absmax_q, absmax_scale = w
        two = torch.empty((codes.numel(), 2), dtype=torch.uint8, device=dev)
        two[:, 0], two[:, 1] = codes // 16, codes % 16
        scale = absmax if absmax is not None else absmax_q.to(torch.float32) * absmax_scale
        element = torch.arange(n * k, device=dev)
        v = _levels(dev)[two.view(-1).long()] * scale[element.div(case["block"], rounding_mode="floor")]  # one fp32 product,
        return v.to(s["dt"]).to(f64).view(n, k)  # rounded to the compute type

    alpha = s["alpha"] / case["r"]
    A, B = s["A"].to(f64), s["B"].to(f64)
    if case["op"] == "gated_fwd":
        t = torch.einsum("mk,prk->pmr", x, A) * alpha
        pre = torch.einsum("pmr,pnr->pmn", t, B)
        pre[0] += x @ base(s["gate"]).T
        pre[1] += x @ base(s["up"]).T
        if s["bias"] is not None:
            pre += s["bias"].to(f64)[:, None]
        h = _exact_act(pre[0], case["act"])[0] * pre[1]
        return {"h": h, "pre": pre, "t": t} if case["save"] else {"h": h}
    dh, g, u = s["dh"].to(f64), s["pre"][0].to(f64), s["pre"][1].to(f64)
    value, slope = _exact_act(g, case["act"])
    d = torch.stack((dh * u * slope, dh * value))
    v = torch.einsum("pmn,pnr->pmr", d, B) * alpha
    dx = d[0] @ base(s["gate"]) + d[1] @ base(s["up"]) + torch.einsum("pmr,prk->mk", v, A)
    return {"dA": torch.einsum("pmr,mk->prk", v, x), "dB": torch.einsum("pmn,pmr->pnr", d, s["t"].to(f64)), "dx": dx}
