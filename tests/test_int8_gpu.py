"""GPU parity of the 8-bit integer quantizer and linear against their definitions in 64 bits.

Codes and scales are exact.  The linear's sums are exact integers, so with the
same codes y is off by its fp32 steps alone: the sum to fp32 (2^-24), two scale
products, the bias add, and one rounding to the output type.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def _Q():
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    return Q


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _quantize64(x):
    """(codes, scale) from the definition: x fp64 holding the input's values."""
    top = np.abs(x).max(axis=1, initial=0.0)
    scale = (top / 127.0).astype(np.float32)      # x is at most 24 bits: one rounding
    s = scale.astype(np.float64)[:, None]
    q = np.divide(x, s, out=np.zeros_like(x), where=s > 0)
    return np.clip(np.rint(q), -127, 127).astype(np.int8), scale


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 17), (5, 8), (7, 1000), (64, 4096), (2, 4100), (33, 11008),
                                       (1, 40000), (2, 30001), (1000, 64)])
def test_quantize(cuda_device, dtype, rows, cols):
    import torch
    Q = _Q()
    gen = torch.Generator().manual_seed(rows * 100003 + cols)
    x = (torch.randn(rows, cols, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen))).to(_dt(dtype))
    m = Q.int8_quantize(x.to(cuda_device))
    codes, scale = _quantize64(x.double().numpy())
    assert np.array_equal(m.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    assert np.array_equal(m.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_next_to_halves(cuda_device, dtype):
    """Values at and beside every half step (half of the largest value lies next to 63.5 steps)."""
    import torch
    Q = _Q()
    rows = []
    for top in (127.0, 1.0, 3.7, 0.33, 254.0, 100.0, 1.984375):
        tops = torch.tensor(top).to(_dt(dtype))
        half = (torch.arange(0, 127) + 0.5) * (float(tops) / 127)
        h = half.to(_dt(dtype)).float()
        near = torch.cat([h, torch.nextafter(h, torch.tensor(1e9)), torch.nextafter(h, torch.tensor(-1e9))])
        row = torch.cat([tops.float().reshape(1), near, -near, tops.float().reshape(1) / 2])
        rows.append(row.clamp(-float(tops), float(tops)))
    x = torch.stack(rows).to(_dt(dtype))
    m = Q.int8_quantize(x.to(cuda_device))
    codes, scale = _quantize64(x.double().numpy())
    assert np.array_equal(m.scale.cpu().numpy(), scale)
    assert np.array_equal(m.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("cols", [24, 25])
def test_quantize_edges(cuda_device, cols):
    """Zero rows, rows whose scale is subnormal or 0, the largest finite values, and NaN / Inf rows."""
    import torch
    Q = _Q()
    base = torch.linspace(-1, 1, cols)
    rows = [base * 0, base * 1e-38, base * 1e-40, base * 1e-43, base * 1e-45, base * 3.4e38, base]
    x = torch.stack(rows).float()
    m = Q.int8_quantize(x.to(cuda_device))
    codes, scale = _quantize64(x.double().numpy())
    assert np.array_equal(m.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    assert np.array_equal(m.codes.cpu().numpy(), codes)
    bad = base.repeat(4, 1)
    bad[0, 3], bad[1, cols - 1], bad[2, 0] = float("nan"), float("inf"), float("-inf")
    m = Q.int8_quantize(bad.to(cuda_device))
    assert m.scale[:3].isnan().all() and not m.codes[:3].any()
    assert m.scale[3].isfinite() and m.codes[3].any()


def test_quantize_empty(cuda_device):
    import torch
    Q = _Q()
    m = Q.int8_quantize(torch.zeros(0, 16, device=cuda_device))
    assert m.codes.shape == (0, 16)
    m = Q.int8_quantize(torch.zeros(3, 0, device=cuda_device))
    assert not m.scale.any()


def _check_linear(cuda_device, m, n, k, dtype, bias, given=False, seed=0):
    import torch
    Q = _Q()
    gen = torch.Generator().manual_seed(seed + m + 7 * n + 13 * k)
    dt = _dt(dtype)
    x = torch.randn(m, k, generator=gen).to(dt)
    wc = torch.randint(-127, 128, (n, k), generator=gen, dtype=torch.int8)
    ws = torch.rand(n, generator=gen) * 0.01 + 0.001
    b = torch.randn(n, generator=gen).to(dt) if bias else None
    w = Q.Int8Matrix(wc.to(cuda_device), ws.to(cuda_device))
    space = Q.Workspace(cuda_device)
    xg = x.to(cuda_device)
    bg = None if b is None else b.to(cuda_device)
    if given:
        y = Q.int8_linear_fwd(w, Q.int8_quantize(xg), bias=bg, out_dtype=dt, workspace=space)
    else:
        y = Q.int8_linear_fwd(w, xg, bias=bg, workspace=space)
    assert y.dtype == dt and space.read_status() == 0
    codes, scale = _quantize64(x.double().numpy())
    core = (codes.astype(np.float64) @ wc.numpy().astype(np.float64).T) * scale.astype(np.float64)[:, None] * ws.double().numpy()
    bn = 0.0 if b is None else b.double().numpy()
    want = core + bn
    fp32 = 4 * 2.0 ** -24 * np.abs(core) + 2.0 ** -24 * np.abs(want)
    bound = fp32 + HALF[dtype] * (np.abs(want) + fp32) + (2.0 ** -25 if dtype == "f16" else 0.0)
    got = y.double().cpu().numpy()
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[:4].tolist()}"
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k,bias", [
    (1, 8, 16, False), (1, 64, 64, True), (1, 4096, 4096, False), (2, 1000, 2064, True), (5, 136, 48, False),
    (8, 264, 1040, True), (9, 128, 4096, False), (16, 4096, 1024, False), (17, 520, 112, True), (31, 1000, 528, False),
    (32, 256, 512, False), (33, 256, 512, True), (64, 392, 4112, False), (65, 128, 128, False), (127, 1032, 80, True),
    (128, 128, 256, False), (129, 264, 272, False), (255, 8, 4096, True), (300, 1000, 1040, False), (513, 776, 400, True),
])
def test_linear(cuda_device, m, n, k, bias, dtype):
    _check_linear(cuda_device, m, n, k, dtype, bias)
    _check_linear(cuda_device, m, n, k, dtype, bias, given=True)


def test_linear_largest_sums(cuda_device):
    """All codes at +-127 over the longest K: the int32 sums come within 2 % of their range."""
    import torch
    Q = _Q()
    k = 131072
    for m in (2, 40, 200):
        xc = torch.full((m, k), 127, dtype=torch.int8, device=cuda_device)
        wc = torch.full((16, k), 127, dtype=torch.int8, device=cuda_device)
        wc[1::2] = -127
        one = lambda c: torch.ones(c, device=cuda_device)
        y = Q.int8_linear_fwd(Q.Int8Matrix(wc, one(16)), Q.Int8Matrix(xc, one(m)), out_dtype=torch.float32)
        want = np.float32(127 * 127 * k)
        assert (y[:, 0::2] == want).all() and (y[:, 1::2] == -want).all()


@pytest.mark.parametrize("m", [3, 150])
def test_linear_non_finite_rows(cuda_device, m):
    """A row with NaN or Inf gives a NaN row; the others keep their bits."""
    import torch
    Q = _Q()
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    w = Q.int8_quantize(torch.randn(264, 512, generator=gen, device=cuda_device))
    x = torch.randn(m, 512, generator=gen, device=cuda_device).to(torch.bfloat16)
    y = Q.int8_linear_fwd(w, x)
    x[1, 5] = float("inf")
    y2 = Q.int8_linear_fwd(w, x)
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(y[keep], y2[keep]) and y2[1].isnan().all()


@pytest.mark.parametrize("m", [1, 20, 200])
def test_linear_repeats_streams_and_graphs(cuda_device, m):
    import torch
    Q = _Q()
    gen = torch.Generator(device=cuda_device).manual_seed(2)
    ws = [Q.int8_quantize(torch.randn(1000, 2064, generator=gen, device=cuda_device)) for _ in range(2)]
    xs = [torch.randn(m, 2064, generator=gen, device=cuda_device).to(torch.float16) for _ in range(2)]
    want = [Q.int8_linear_fwd(w, x) for w, x in zip(ws, xs)]
    for _ in range(10):
        assert all(torch.equal(Q.int8_linear_fwd(w, x), y) for w, x, y in zip(ws, xs, want))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = Q.int8_linear_fwd(ws[0], xs[0], stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    graphs, outs = [], []
    for w, x in zip(ws, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(Q.int8_linear_fwd(w, x))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        Q.int8_linear_fwd(ws[0], xs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, y) for o, y in zip(outs, want))


def test_experts_to_int8(cuda_device):
    """The operators as they are used in a row: two expert layers forward and backward with an adapter update, each
    expert then merged dense, brought to 8 bits and served on its rows.  The served result is held to the 8-bit
    steps of both operands."""
    import torch
    Q = _Q()
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(9)
    e, h, f, r, tokens = 4, 256, 512, 16, 96
    mk = lambda *s, sigma=1.0: torch.randn(s, generator=gen, device=dev) * sigma
    up, down = (Q.quantize(mk(e * a, b, sigma=0.02), 64, True) for a, b in ((f, h), (h, f)))
    bf = torch.bfloat16
    Au, Bu, Ad, Bd = mk(e, r, h, sigma=h ** -0.5).to(bf), mk(e, f, r, sigma=0.01).to(bf), mk(e, r, f, sigma=f ** -0.5).to(bf), mk(e, h, r, sigma=0.01).to(bf)
    x = mk(tokens, h).to(bf)
    top = mk(tokens, e).topk(2, dim=1).indices                       # a router's choice: two experts a token
    order = torch.argsort(top.reshape(-1), stable=True)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(torch.bincount(top.reshape(-1), minlength=e), 0).to(torch.int32)
    rows = x[order // 2].contiguous()

    def forward():
        hid, t1 = Q.grouped_fwd(up, rows, offsets, Au, Bu, 32.0)
        act = torch.relu(hid)
        y, t2 = Q.grouped_fwd(down, act, offsets, Ad, Bd, 32.0)
        return hid, t1, act, t2, y

    hid, t1, act, t2, y = forward()
    dy = mk(2 * tokens, h).to(bf)
    dAd, dBd, dact = Q.grouped_bwd(down, act, offsets, Ad, Bd, 32.0, dy, t=t2)
    dAu, dBu, dx = Q.grouped_bwd(up, rows, offsets, Au, Bu, 32.0, (dact * (hid > 0)).to(bf), t=t1)
    assert all(v.isfinite().all() for v in (dAd, dBd, dAu, dBu)) and dx.float().isfinite().all()
    for p, g in ((Ad, dAd), (Bd, dBd), (Au, dAu), (Bu, dBu)):
        p.copy_((p.float() - 1e-4 * g).to(bf))
    y = forward()[-1]
    off = offsets.tolist()
    for i in range(e):
        sel = rows[off[i]:off[i + 1]].contiguous()
        if not len(sel):
            continue
        part = lambda q, n, k: Q.QuantizedWeight(q.codes[i * n * k // 2:(i + 1) * n * k // 2], None,
                                                 q.absmax_q[i * n * k // 64:(i + 1) * n * k // 64], q.absmax_scale, n, k, 64, True)
        wu = Q.int8_quantize(Q.merge(part(up, f, h), Au[i], Bu[i], 32.0, "f32"))
        wd = Q.int8_quantize(Q.merge(part(down, h, f), Ad[i], Bd[i], 32.0, "f32"))
        a = torch.relu(Q.int8_linear_fwd(wu, sel))
        served = Q.int8_linear_fwd(wd, a)
        # every operand is off by at most half a step of 1/127 of its row's largest value (x and W of both layers)
        am, wm = a.double(), wd.dequantize().double().abs()
        xm, um = sel.double().abs(), wu.dequantize().double().abs()
        half = lambda v: v.abs().amax(1, keepdim=True) / 254
        err1 = xm @ half(um).expand_as(um).T + half(xm).expand_as(xm) @ um.T + 2.0 ** -6 * (xm @ um.T)
        err2 = (am.abs() + err1) @ (half(wm).expand_as(wm)).T + (half(am).expand_as(am) + err1) @ wm.T + 2.0 ** -6 * (am.abs() @ wm.T)
        assert ((served.double() - y[off[i]:off[i + 1]].double()).abs() <= err2).all()
