"""GPU parity of the 8-bit floating point quantizer, its inverse and the linear against their
definitions in 64 bits.

Codes, scales and dequantized values are exact.  With the same codes a linear's y is off by
its fp32 steps alone, f = 2^-23 each (the tensor core may truncate when it adds): K adds
inside the blocks, three operations a block (the scales' product, scaling, adding; the warps
of the few-token kernel add eight sums more), the bias, and one rounding to the output type.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
F = 2.0 ** -23


def _Q():
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    return Q


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def spread(scale, block_rows, rows, cols):
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def quantize64(x, block_rows):
    """(values of the codes, scales) from the definition: x in fp64 holding the input's values."""
    import torch
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    pad = torch.nn.functional.pad(x, (0, bc * 128 - cols, 0, br * block_rows - rows)).view(br, block_rows, bc, 128)
    scale = (pad.abs().amax((1, 3)) / 448).float()
    s = spread(scale.double(), block_rows, rows, cols)
    v = torch.where(s > 0, x / s, torch.zeros_like(x)).float().double()     # the fp32 quotient
    step = torch.exp2(torch.frexp(v)[1].double().sub(1).clamp(min=-6) - 3)  # e4m3: three bits after the leading one
    return (torch.round(v / step) * step).clamp(-448, 448), scale


def check_codes(m, x, block_rows):
    import torch
    codes, scale = quantize64(x.double().to(m.codes.device), block_rows)
    assert m.scale.view(torch.int32).equal(scale.view(torch.int32))
    assert m.codes.float().double().equal(codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 17), (5, 8), (7, 1000), (129, 4096), (2, 4100), (127, 260),
                                       (128, 128), (300, 387), (1000, 64)])
def test_quantize(cuda_device, dtype, block_rows, rows, cols):
    import torch
    Q = _Q()
    gen = torch.Generator().manual_seed(rows * 100003 + cols)
    x = (torch.randn(rows, cols, generator=gen) * torch.exp(2 * torch.randn(rows, 1, generator=gen))).to(_dt(dtype)).to(cuda_device)
    m = Q.fp8_quantize(x, block_rows)
    check_codes(m, x, block_rows)
    want = m.codes.float() * spread(m.scale, block_rows, rows, cols)
    for out in ("f32", "bf16", "f16"):
        assert Q.fp8_dequantize(m, _dt(out)).equal(want.to(_dt(out)))


def test_quantize_next_to_halves(cuda_device):
    """Quotients at and beside every half step, subnormal codes among them."""
    import torch
    Q = _Q()
    grid = torch.arange(0, 126, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    half = (grid[:-1] + grid[1:]) / 2
    rows = []
    for scale in (1.0, 2.0 ** -9, 0.37, 3.1e-5, 1.9e4):
        h = half * scale
        near = torch.cat([h, torch.nextafter(h, torch.tensor(1e9)), torch.nextafter(h, torch.tensor(-1e9))])
        row = torch.zeros(4 * 128)
        for b in range(4):   # a block's largest value sets its scale
            part = near[b * 127:(b + 1) * 127]
            row[b * 128:b * 128 + len(part)] = part
            row[b * 128 + 127] = 448 * scale
        rows += [row, -row]
    x = torch.stack(rows).to(cuda_device)
    check_codes(Q.fp8_quantize(x, 1), x, 1)


@pytest.mark.parametrize("dtype,cols", [("f32", 128), ("f32", 131), ("bf16", 136), ("f16", 130)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_edges(cuda_device, dtype, cols, block_rows):
    """Zeros, scales that are subnormal or 0, the largest finite values; NaN and infinities."""
    import torch
    Q = _Q()
    top = torch.finfo(_dt(dtype)).max
    for factor in (0.0, 1e-36, 1e-38, 1e-40, 1e-43, 1e-45, 1.0):
        x = (torch.linspace(-1, 1, cols).repeat(3, 1) * factor).to(_dt(dtype)).to(cuda_device)
        check_codes(Q.fp8_quantize(x, block_rows), x, block_rows)
    x = torch.full((3, cols), top, dtype=_dt(dtype), device=cuda_device)
    check_codes(Q.fp8_quantize(x, block_rows), x, block_rows)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.ones((130, cols), dtype=_dt(dtype), device=cuda_device)
        x[1, 3] = bad
        m = Q.fp8_quantize(x, block_rows)
        nan = m.scale.isnan()
        assert nan[1 if block_rows == 1 else 0, 0] and int(nan.sum()) == 1
        hit = spread(nan.float(), block_rows, 130, cols) > 0
        assert not m.codes.float()[hit].any() and (m.codes.float()[~hit] == 448).all()
        assert Q.fp8_dequantize(m)[hit].isnan().all()


class Lin:
    def __init__(self, dev, m, n, k, dtype="bf16", bias=False, seed=0):
        import torch
        gen = torch.Generator().manual_seed(seed + 31 * m + 7 * n + k)
        randn = lambda *s: torch.randn(*s, generator=gen)
        self.m, self.n, self.k, self.dtype = m, n, k, dtype
        self.x = (randn(m, k) * (1 + 9 * (torch.rand(k, generator=gen) < 0.02))).to(_dt(dtype)).to(dev)
        self.w = _Q().fp8_quantize((randn(n, k) * 0.02).to(dev), 128)
        self.bias = randn(n).to(_dt(dtype)).to(dev) if bias else None

    def check(self, y, q=None, rows=slice(None)):
        import torch
        q = q if q is not None else _Q().fp8_quantize(self.x, 1)
        xv = q.codes.float().double() * spread(q.scale.double(), 1, self.m, self.k)
        wv = self.w.codes.float().double() * spread(self.w.scale.double(), 128, self.n, self.k)
        xv = xv[rows]
        b = 0.0 if self.bias is None else self.bias.double()
        want = xv @ wv.T + b
        mag = xv.abs() @ wv.abs().T + (0.0 if self.bias is None else b.abs())
        h = HALF[self.dtype]
        bound = h * want.abs() + (1 + h) * (self.k + 3 * -(-self.k // 128) + 12) * F * mag + (2.0 ** -25 if self.dtype == "f16" else 0.0)
        got = y[rows].double()
        assert got.shape == want.shape and torch.isfinite(got).all()
        off = (got - want).abs() - bound
        assert off.max() <= 0, f"off by {(got - want).abs().max():.3e}"


@pytest.mark.parametrize("m,n,k,dtype,bias", [
    (1, 8, 16, "bf16", False), (1, 4096, 4096, "bf16", False), (1, 1000, 144, "f16", True), (2, 136, 128, "f32", True),
    (3, 24, 11008, "bf16", False), (8, 520, 2064, "f16", False), (9, 72, 256, "bf16", True), (16, 2056, 1024, "f32", False),
    (17, 128, 512, "bf16", False), (24, 256, 4096, "bf16", True), (32, 264, 3056, "f16", True), (32, 64, 16, "bf16", False),
    (33, 256, 384, "bf16", False), (64, 8, 144, "f32", True), (128, 1000, 2064, "f16", False), (129, 640, 272, "bf16", True),
    (257, 72, 1040, "bf16", False), (333, 1000, 2064, "f16", True), (500, 4104, 128, "f32", True), (1000, 5000, 400, "bf16", True),
    (2100, 2312, 640, "f32", False), (2048, 2560, 1152, "f16", False)])
def test_linear(cuda_device, m, n, k, dtype, bias):
    Q = _Q()
    L = Lin(cuda_device, m, n, k, dtype, bias)
    y = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias)
    assert y.dtype == _dt(dtype)
    L.check(y)
    q = Q.fp8_quantize(L.x, 1)
    y2 = Q.fp8_linear_fwd(L.w, q, bias=L.bias, out_dtype=_dt(dtype))
    assert y2.equal(y)                       # quantized in the call or before: the same codes
    assert Q.read_status() == 0


@pytest.mark.parametrize("m", [2, 40, 300])
def test_tokens_that_are_not_finite_stay_alone(cuda_device, m):
    import torch
    Q = _Q()
    L = Lin(cuda_device, m, 264, 400)
    x = L.x.clone()
    x[1, 5], clean = float("inf"), L.x
    if m > 2:
        x[m - 1, 399] = float("nan")
    y = Q.fp8_linear_fwd(L.w, x)
    bad = torch.zeros(m, dtype=torch.bool, device=cuda_device)
    bad[1] = True
    if m > 2:
        bad[m - 1] = True
    assert y[bad].isnan().all()
    assert y[~bad].equal(Q.fp8_linear_fwd(L.w, clean)[~bad])


def test_weight_block_that_is_not_finite(cuda_device):
    """NaN outputs for the 128 rows of the block, the others untouched."""
    import torch
    Q = _Q()
    for m in (1, 200):
        L = Lin(cuda_device, m, 520, 512)
        want = Q.fp8_linear_fwd(L.w, L.x)
        w = Q.Fp8Matrix(L.w.codes, L.w.scale.clone(), 128)
        w.scale[1, 2] = float("nan")
        y = Q.fp8_linear_fwd(w, L.x)
        assert y[:, 128:256].isnan().all()
        rest = torch.cat([y[:, :128], y[:, 256:]], 1)
        assert rest.equal(torch.cat([want[:, :128], want[:, 256:]], 1))


def test_rows_behind_the_batch_stay(cuda_device):
    import torch
    Q = _Q()
    for m, n in ((5, 264), (77, 264), (300, 5000)):
        for dtype in ("bf16", "f32"):
            L = Lin(cuda_device, m, n, 256, dtype)
            big = torch.full((m + 40, n), 7.0, dtype=_dt(dtype), device=cuda_device)
            Q.fp8_linear_fwd(L.w, L.x, out=big[:m])
            L.check(big[:m])
            assert (big[m:] == 7).all()


@pytest.mark.parametrize("m", [1, 6, 40, 300])
def test_captured_and_on_another_stream(cuda_device, m):
    import torch
    Q = _Q()
    L = Lin(cuda_device, m, 520, 400, bias=True)
    want = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias)
    q = Q.fp8_quantize(L.x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias, stream=side)
    side.synchronize()
    assert y.equal(want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias)
            codes = Q.fp8_quantize(L.x)
            back = Q.fp8_dequantize(codes, torch.bfloat16)
        graphs.append((g, out, codes, back))
    for _ in range(3):
        for g, out, codes, back in graphs:
            g.replay()
        between = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias)
        torch.cuda.synchronize()
        assert between.equal(want)
        for g, out, codes, back in graphs:
            assert out.equal(want) and codes.codes.view(torch.uint8).equal(q.codes.view(torch.uint8)) and codes.scale.equal(q.scale)
            assert back.equal(Q.fp8_dequantize(q, torch.bfloat16))
    assert Q.read_status() == 0 and Q.read_status(side) == 0


def test_a_merged_weight(cuda_device):
    """What serves a trained adapter: merge, quantize, linear.  Against the merged weight itself a product is off by at
    most half a step of each operand, 2^-4 of it (or 2^-10 scales where e4m3 is subnormal)."""
    import torch
    Q = _Q()
    gen = torch.Generator().manual_seed(5)
    n, k, r = 264, 320, 16
    q = Q.quantize((torch.randn(n, k, generator=gen) * 0.02).to(cuda_device), 64, True)
    A, B = ((torch.randn(*s, generator=gen) * 0.05).to(torch.bfloat16).to(cuda_device) for s in ((r, k), (n, r)))
    dense = Q.merge(q, A, B, 32.0, "f32")
    w = Q.fp8_quantize(dense, 128)
    back = Q.fp8_dequantize(w).double()
    step = torch.maximum(dense.double().abs() * 2.0 ** -4, spread(w.scale.double(), 128, n, k) * 2.0 ** -10)
    assert ((back - dense.double()).abs() <= step * (1 + 2.0 ** -20)).all()
    for m in (1, 100):
        x = torch.randn(m, k, generator=gen).to(torch.bfloat16).to(cuda_device)
        y = Q.fp8_linear_fwd(w, x).double()
        xa, wa = x.double().abs(), dense.double().abs()
        sx = spread(Q.fp8_quantize(x).scale.double(), 1, m, k)
        ex = torch.maximum(xa * 2.0 ** -4, sx * 2.0 ** -10)
        bound = ex @ (wa + step).T + xa @ step.T
        want = x.double() @ dense.double().T
        assert ((y - want).abs() <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_more_than_two_to_the_31_elements(cuda_device, block_rows):
    """Offsets past 32 bits: the last rows of a matrix are those of the same rows by themselves."""
    import torch
    Q = _Q()
    rows, cols = 128 * 513 + 41, 32_776
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    gen = torch.Generator(device=cuda_device).manual_seed(2)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda_device)
    x[-169:] = torch.randn(169, cols, generator=gen, device=cuda_device).to(torch.bfloat16)
    q, last = Q.fp8_quantize(x, block_rows), Q.fp8_quantize(x[-169:].clone(), block_rows)
    del x
    assert q.codes[-169:].view(torch.uint8).equal(last.codes.view(torch.uint8))
    assert q.scale[-last.scale.shape[0]:].equal(last.scale)
    back = Q.fp8_dequantize(q, torch.bfloat16)
    assert back[-169:].equal(Q.fp8_dequantize(last, torch.bfloat16))
    del back, q
    torch.cuda.empty_cache()


def test_linear_with_more_than_two_to_the_31_results(cuda_device):
    import torch
    Q = _Q()
    m, n, k = 70_041, 32_776, 144
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    w = Q.fp8_quantize(torch.randn(n, k, generator=gen, device=cuda_device), 128)
    x = torch.randn(m, k, generator=gen, device=cuda_device).to(torch.bfloat16)
    y = Q.fp8_linear_fwd(w, x)
    for rows in (slice(0, 130), slice(m // 2, m // 2 + 130), slice(m - 130, m)):
        assert y[rows].equal(Q.fp8_linear_fwd(w, x[rows].clone()))
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(9, 1024, 8192), (16, 264, 4096), (40, 520, 11008), (127, 136, 6000), (129, 1000, 4112), (200, 72, 16384),
                                   (64, 11008, 512), (33, 4104, 4096)])
def test_few_tiles_share_a_long_sum(cuda_device, m, n, k, dtype):
    import torch
    Q = _Q()
    L = Lin(cuda_device, m, n, k, dtype, bias=True)
    big = torch.full((m + 5, n), 7.0, dtype=L.x.dtype, device=cuda_device)
    y = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias, out=big[:m])
    L.check(y)
    assert (big[m:] == 7).all()
    for _ in range(3):
        assert Q.fp8_linear_fwd(L.w, L.x, bias=L.bias).equal(y)
    x = L.x.clone()
    x[1, 5] = float("nan")
    z = Q.fp8_linear_fwd(L.w, x, bias=L.bias)
    rows = torch.arange(m, device=cuda_device) != 1
    assert z[rows].equal(y[rows]) and not torch.isfinite(z[1]).any()
    assert Q.read_status() == 0
