"""GPU parity of the expert (grouped) QLoRA linear, forward and backward, against
its formulas in 64 bits on the same inputs.

Bounds per element, with e = half a step of the compute type (bf16 2^-8, f16
2^-11, fp32 2^-24), f = 2^-23 per fp32 add (the tensor core may truncate) and
|.| products taken with absolute values:
  T   e |T| + s (K + 2) f |x||A|
  y   e |y| + e |T||B| + (K + r + 3) f (|x||W'| + |T||B| + |bias|) + the T sum's own error times |B|
  dB  (c + 2) f |dy||T|                         (c rows; t is an input)
  dA  (u + (N + 2) f) s |dy||B||x| + (c + 2) f |U||x|,  u what the terms of the compute type lose of U:
      2^-23 (three terms of bf16), 2^-21 (two of f16), 2^-23 (fp32)
  dx  e |dx| + e |U||A| + (N + r + 3) f (|dy||W'| + |U||A|) + the U sum's own error times |A|
"""
import numpy as np
import pytest

from oracle import nf4_oracle as O

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SPLIT = {"bf16": 2.0 ** -23, "f16": 2.0 ** -21, "f32": 2.0 ** -23}
F = 2.0 ** -23


def _Q():
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    return Q


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


class Stack:
    """A stack of experts with ragged rows, on the GPU and in 64 bits."""

    def __init__(self, dev, counts, n, k, r, dtype="bf16", block=64, dq=True, bias=False, lead=0, pad=0,
                 seed=0, zero_w=False):
        import torch
        Q = _Q()
        self.dev, self.counts, self.n, self.k, self.r, self.dtype = dev, counts, n, k, r, dtype
        self.e = len(counts)
        self.m = lead + sum(counts) + pad
        off = np.cumsum([lead] + list(counts))
        self.off = off
        self.offsets = torch.tensor(off, dtype=torch.int32, device=dev)
        self.alpha = 2.0 * r
        self.s = self.alpha / r
        rng = np.random.default_rng(seed + 7 * n + k)
        w = (rng.standard_normal((self.e * n, k)) * (0.0 if zero_w else 0.02)).astype(np.float32)
        ref = O.quantize(w, block, double=dq)
        self.q = Q.quantize(torch.from_numpy(w).to(dev), block, dq)
        dt = _dt(dtype)
        t = lambda *shape, sigma=1.0: torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(dt)
        self.x, self.A, self.B = t(self.m, k), t(self.e, r, k, sigma=k ** -0.5), t(self.e, n, r, sigma=0.05)
        self.dy = t(self.m, n)
        self.bias = t(self.e, n) if bias else None
        f64 = lambda v: None if v is None else v.double().numpy()
        self.xn, self.An, self.Bn, self.dyn, self.biasn = map(f64, (self.x, self.A, self.B, self.dy, self.bias))
        wd = torch.from_numpy(np.ascontiguousarray(O.dequantize(ref, "f32"))).reshape(self.e, n, k)
        self.W = wd.to(dt).double().numpy()
        self.x, self.A, self.B, self.dy = (v.to(dev) for v in (self.x, self.A, self.B, self.dy))
        self.bias = None if self.bias is None else self.bias.to(dev)

    def rows(self, e):
        return slice(int(self.off[e]), int(self.off[e + 1]))

    def fwd(self, **kw):
        return _Q().grouped_fwd(self.q, self.x, self.offsets, self.A, self.B, self.alpha, bias=self.bias, **kw)

    def bwd(self, **kw):
        return _Q().grouped_bwd(self.q, self.x, self.offsets, self.A, self.B, self.alpha, self.dy, **kw)

    def check_fwd(self, y, t, experts=None):
        h = HALF[self.dtype]
        y, t = y.double().cpu().numpy(), t.double().cpu().numpy()
        for e in range(self.e) if experts is None else experts:
            x, A, B, W = self.xn[self.rows(e)], self.An[e], self.Bn[e], self.W[e]
            if not len(x):
                continue
            tw = self.s * (x @ A.T)
            t_sum = self.s * (self.k + 2) * F * (abs(x) @ abs(A).T)
            _within("T", t[self.rows(e)], tw, h * abs(tw) + (1 + h) * t_sum)
            b = 0.0 if self.biasn is None else self.biasn[e]
            yw = x @ W.T + tw @ B.T + b
            ta = abs(tw) @ abs(B).T
            bound = (h * abs(yw) + h * ta + (1 + h) ** 2 * (t_sum @ abs(B).T) +
                     (1 + h) * (self.k + self.r + 3) * F * (abs(x) @ abs(W).T + (1 + h) * ta + abs(b)))
            _within("y", y[self.rows(e)], yw, bound)

    def check_bwd(self, dA, dB, dx, t, experts=None):
        h = HALF[self.dtype]
        dA, dB, t = dA.double().cpu().numpy(), dB.double().cpu().numpy(), t.double().cpu().numpy()
        dx = None if dx is None else dx.double().cpu().numpy()
        for e in range(self.e) if experts is None else experts:
            rows = self.rows(e)
            x, dy, te = self.xn[rows], self.dyn[rows], t[rows]
            A, B, W = self.An[e], self.Bn[e], self.W[e]
            c = len(x)
            if c == 0:
                assert not dA[e].any() and not dB[e].any(), "an expert without rows has zero gradients"
                continue
            u = self.s * (dy @ B)
            ua = self.s * (abs(dy) @ abs(B))
            u_sum = (self.n + 2) * F * ua
            _within("dB", dB[e], dy.T @ te, (c + 2) * F * (abs(dy).T @ abs(te)) + 1e-30)
            u_err = SPLIT[self.dtype] * (abs(u) + u_sum) + u_sum
            if self.dtype == "f16":
                u_err = u_err + 2.0 ** -36   # the second term's smallest step, 2^-24 over 2^11, halved
            _within("dA", dA[e], u.T @ x, u_err.T @ abs(x) + (c + 2) * F * ((abs(u) + u_err).T @ abs(x)))
            if dx is None:
                continue
            want = dy @ W + u @ A
            aa = abs(u) @ abs(A)
            bound = (h * abs(want) + h * aa + (1 + h) ** 2 * (u_sum @ abs(A)) +
                     (1 + h) * (self.n + self.r + 3) * F * (abs(dy) @ abs(W) + (1 + h) * aa))
            _within("dx", dx[rows], want, bound)


def _within(name, got, want, bound):
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    bad = np.abs(got - want) > bound
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.max(np.abs(got - want) / np.maximum(bound, 1e-300)):.3g} times the bound at "
                           f"{np.unravel_index(np.argmax(np.abs(got - want) / np.maximum(bound, 1e-300)), got.shape)}")


SHAPES = [
    # counts, n, k, r
    ([1], 64, 64, 8),
    ([1, 0, 1], 136, 128, 16),
    ([0, 3, 0, 0, 5, 0], 264, 320, 24),
    ([33, 1, 64, 0, 17], 200, 192, 40),
    ([127, 128, 129], 256, 256, 64),
    ([300, 0, 5, 255, 257], 392, 320, 16),
    ([700], 520, 448, 128),
    ([2, 2, 2, 2], 1032, 1088, 16),
    ([20, 70], 128, 4160, 256),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts,n,k,r", SHAPES)
def test_forward_backward(cuda_device, counts, n, k, r, dtype):
    """Ragged rows, empty experts, sizes off every tile, both directions."""
    g = Stack(cuda_device, counts, n, k, r, dtype, dq=len(counts) % 2 == 1, bias=len(counts) > 2, seed=len(counts))
    ws = _Q().Workspace(cuda_device)
    y, t = g.fwd(workspace=ws)
    g.check_fwd(y, t)
    dA, dB, dx = g.bwd(t=t, workspace=ws)
    g.check_bwd(dA, dB, dx, t)
    assert ws.read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_adapter_alone(cuda_device, dtype):
    """A zero base leaves the adapter terms, which the base would drown."""
    g = Stack(cuda_device, [40, 0, 9, 300], 264, 320, 24, dtype, zero_w=True, seed=3)
    y, t = g.fwd()
    g.check_fwd(y, t)
    g.check_bwd(*g.bwd(t=t), t)


@pytest.mark.parametrize("block,dq", [(64, False), (128, True), (256, False), (4096, True)])
def test_block_sizes(cuda_device, block, dq):
    """Blocks that run over rows and, at 4096, over the border of two experts."""
    g = Stack(cuda_device, [3, 70, 0, 130], 40, 192, 8, block=block, dq=dq, seed=block)
    y, t = g.fwd()
    g.check_fwd(y, t)
    g.check_bwd(*g.bwd(t=t), t)


@pytest.mark.parametrize("counts", [[0] * 63 + [1], [1] * 64, list(range(64)), [0, 0, 500] + [0] * 61, [2] * 511 + [0]])
def test_many_experts(cuda_device, counts):
    g = Stack(cuda_device, counts, 64, 128, 8, seed=len(counts))
    y, t = g.fwd()
    g.check_fwd(y, t)
    g.check_bwd(*g.bwd(t=t), t)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[3, 0, 2], [150, 0, 70, 300]])
def test_rows_of_no_expert(cuda_device, dtype, counts):
    """Rows before the first offset and behind the last stay as they were, and what
    they hold (NaN here) reaches nothing."""
    import torch
    g = Stack(cuda_device, counts, 136, 192, 16, dtype, lead=5, pad=67, seed=11)
    outside = torch.ones(g.m, dtype=torch.bool)
    outside[g.off[0]:g.off[-1]] = False
    g.x[outside.to(cuda_device)] = float("nan")
    g.dy[outside.to(cuda_device)] = float("nan")
    mk = lambda c: torch.full((g.m, c), 7.0, dtype=_dt(dtype), device=cuda_device)
    y, t = g.fwd(out=mk(136), t_out=mk(16))
    g.check_fwd(y, t)
    t[outside.to(cuda_device)] = float("inf")
    dA, dB, dx = g.bwd(t=t, dx=mk(192))
    g.check_bwd(dA, dB, dx, t)
    assert (y.cpu()[outside] == 7).all() and (dx.cpu()[outside] == 7).all()
    y2, _ = g.fwd(out=mk(136), want_t=False)
    assert torch.equal(y2, y)
    dA2, dB2, none = g.bwd(t=None, want_dx=False)
    assert none is None
    assert torch.equal(dA2, dA) and torch.equal(dB2, dB)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_non_finite_values_stay_in_their_expert(cuda_device, dtype):
    """NaN and Inf in one expert's rows, adapters and bias: the others' results keep their bits."""
    import torch
    g = Stack(cuda_device, [30, 10, 90], 72, 128, 8, dtype, bias=True, seed=5)
    y, t = g.fwd()
    dA, dB, dx = g.bwd(t=t)
    r = slice(30, 40)
    g.x[r] = float("nan")
    g.dy[r] = float("inf")
    g.A[1] = float("inf")
    g.B[1] = float("nan")
    g.bias[1] = float("nan")
    y2, t2 = g.fwd()
    dA2, dB2, dx2 = g.bwd(t=t2)
    keep = [i for i in range(130) if not 30 <= i < 40]
    for a, b in ((y, y2), (t, t2), (dx, dx2)):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(b[r].float()).any()
    for a, b in ((dA, dA2), (dB, dB2)):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    # one bad row inside an expert leaves the expert's other rows
    g = Stack(cuda_device, [30, 10, 90], 72, 128, 8, dtype, seed=5)
    y, t = g.fwd()
    _, _, dx = g.bwd(t=t)
    g.x[33] = float("nan")
    g.dy[33] = float("nan")
    y2, t2 = g.fwd()
    _, _, dx2 = g.bwd(t=t2)
    keep = [i for i in range(130) if i != 33]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(t[keep], t2[keep]) and torch.equal(dx[keep], dx2[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_offsets_are_clamped_and_reported(cuda_device, dtype):
    """Offsets that fall, leave the matrix or are negative reach no memory out of bounds: each counts as at
    least the ones before it and at most M, and the status word says so."""
    import torch
    Q = _Q()
    g = Stack(cuda_device, [5, 6, 7], 64, 128, 8, dtype, seed=2)
    for bad, as_if in (([0, 9, 4, 18], [0, 9, 9, 18]), ([-3, 5, 11, 18], [0, 5, 11, 18]),
                       ([0, 5, 11, 1 << 30], [0, 5, 11, 18]), ([0, 99, 5, 6], [0, 18, 18, 18]),
                       ([-2 ** 31, 2 ** 31 - 1, 0, 0], [0, 18, 18, 18])):
        for small in (True, False):
            res = []
            for off in (bad, as_if):
                ws = Q.Workspace(cuda_device)
                g.offsets = torch.tensor(off, dtype=torch.int32, device=cuda_device)
                out = torch.zeros(18, 64, dtype=_dt(dtype), device=cuda_device)
                y, t = g.fwd(out=out, workspace=ws)
                dA, dB, dx = g.bwd(t=t, workspace=ws)
                res.append((y, t, dA, dB, dx))
                assert ws.read_status() == (1 if off is bad else 0)
            assert all(torch.equal(a, b) for a, b in zip(*res))


def test_no_rows(cuda_device):
    """M = 0: the forward enqueues nothing, the backward clears every gradient."""
    import torch
    g = Stack(cuda_device, [0, 0], 64, 64, 8)
    y, t = g.fwd()
    assert y.shape == (0, 64) and t.shape == (0, 8)
    dA = torch.full((2, 8, 64), 3.0, device=cuda_device)
    dB = torch.full((2, 64, 8), 3.0, device=cuda_device)
    g.bwd(t=t, dA=dA, dB=dB)
    assert not dA.any() and not dB.any()
    # rows, but none of them any expert's
    g = Stack(cuda_device, [0, 0], 64, 64, 8, lead=3, pad=4)
    y, t = g.fwd(out=torch.full((7, 64), 2.0, dtype=torch.bfloat16, device=cuda_device))
    assert (y == 2).all()
    dA.fill_(3), dB.fill_(3)
    g.bwd(t=t, dA=dA, dB=dB)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_same_bits_every_time(cuda_device, dtype):
    import torch
    g = Stack(cuda_device, [9, 0, 300, 41, 1], 264, 448, 24, dtype, seed=8)
    first = None
    for _ in range(12):
        y, t = g.fwd()
        got = (y, t) + g.bwd(t=t)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("counts,n,k,r", [([2, 1, 2, 2], 1768, 6528, 64), ([40, 90], 6528, 1792, 24), ([3, 0, 5], 4096, 1024, 8)])
def test_weight_bound_calls_repeated(cuda_device, counts, n, k, r):
    """Few tokens an expert: the tensor core waits for every weight tile, so a tile that is read before it is whole, or
    made from codes already overwritten, shows.  Such a race needs its timing; many calls must give the same bits."""
    import torch
    g = Stack(cuda_device, counts, n, k, r, dq=False, block=128, seed=6)
    y, t = g.fwd()
    g.check_fwd(y, t)
    dA, dB, dx = g.bwd(t=t)
    g.check_bwd(dA, dB, dx, t)
    for _ in range(150):
        again = g.fwd()[:1] + g.bwd(t=t)
        assert all(torch.equal(a, b) for a, b in zip(again, (y, dA, dB, dx)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,r", [([1500, 1000, 100], 72), ([2331, 17, 257], 8), ([0, 2800], 64)])
def test_many_rows_an_expert(cuda_device, counts, r, dtype):
    """Tiles of up to 512 tokens, two products of a decoded weight tile: tiles with both and with one of them, odd
    halves; and the same bits every time."""
    import torch
    g = Stack(cuda_device, counts, 2040, 1984, r, dtype, dq=r == 8, bias=r == 72, seed=12)
    y, t = g.fwd()
    g.check_fwd(y, t)
    dA, dB, dx = g.bwd(t=t)
    g.check_bwd(dA, dB, dx, t)
    for _ in range(60):
        again = g.fwd()[:1] + g.bwd(t=t)
        assert all(torch.equal(a, b) for a, b in zip(again, (y, dA, dB, dx)))


@pytest.mark.parametrize("n,k,r", [(2040, 64, 8), (64, 1984, 8), (8, 1984, 256), (2040, 64, 256)])
def test_many_rows_of_short_sums(cuda_device, n, k, r):
    """The same tiles where a tile has fewer steps than the ring has stages, or more adapter steps than others."""
    import torch
    g = Stack(cuda_device, [2600, 0, 3, 290], n, k, r, seed=14)
    y, t = g.fwd()
    g.check_fwd(y, t)
    dA, dB, dx = g.bwd(t=t)
    g.check_bwd(dA, dB, dx, t)
    for _ in range(100):
        again = g.fwd()[:1] + g.bwd(t=t)
        assert all(torch.equal(a, b) for a, b in zip(again, (y, dA, dB, dx)))


@pytest.mark.parametrize("counts", [[1, 0, 2], [80, 200, 3]])
def test_one_expert_equals_the_dense_layer(cuda_device, counts):
    """Each expert's rows give what the dense layer gives on that expert's weight, to rounding."""
    import torch
    Q = _Q()
    g = Stack(cuda_device, counts, 256, 256, 16, dq=False, seed=4)
    y, t = g.fwd()
    for e, c in enumerate(counts):
        if not c:
            continue
        sl = slice(e * 256 * 256 // 2, (e + 1) * 256 * 256 // 2)
        ab = slice(e * 1024, (e + 1) * 1024)
        q = Q.QuantizedWeight(g.q.codes[sl], g.q.absmax[ab], None, None, 256, 256, 64, False)
        yd, _ = Q.linear_fwd(q, g.x[g.rows(e)].contiguous(), g.A[e], g.B[e], g.alpha)
        torch.testing.assert_close(y[g.rows(e)].float(), yd.float(), rtol=2 ** -7, atol=2 ** -7 * float(yd.abs().max()))


def test_gradients_against_differences(cuda_device):
    """dA, dB and dx of L = sum(dy * y) against central differences of the fp32 mode's own forward: y is linear in
    each of A, B and x, so a difference of any width is the derivative up to the sums' rounding."""
    import torch
    g = Stack(cuda_device, [7, 0, 12], 64, 64, 8, "f32", seed=21)
    y, t = g.fwd()
    dA, dB, dx = g.bwd(t=t)
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    loss = lambda: float((g.fwd()[0].double() * g.dy.double()).sum())
    W = torch.from_numpy(g.W).to(cuda_device).abs()

    def loss_error():
        """What the sums of K and of r products in fp32 may be off in the loss, two steps for every product."""
        x, A, B, dy = (v.double().abs() for v in (g.x, g.A, g.B, g.dy))
        total = 0.0
        for e in range(g.e):
            r = g.rows(e)
            total += float((dy[r] * (x[r] @ W[e].T + 2 * g.s * (x[r] @ A[e].T) @ B[e].T)).sum())
        return (64 + 8 + 4) * 2.0 ** -23 * total

    for param, grad, terms in ((g.A, dA, 12 + 64), (g.B, dB, 12 + 64), (g.x, dx, 64 + 8 + 64)):
        d = torch.randn(param.shape, generator=gen, device=cuda_device)
        keep = param.clone()
        param.copy_(keep + 0.5 * d)
        up, err, high = loss(), loss_error(), param.double()
        param.copy_(keep - 0.5 * d)
        down, err, low = loss(), err + loss_error(), param.double()
        param.copy_(keep)
        want = float((grad.double() * (high - low)).sum())
        # the gradient's own sums, of `terms` products, relative to the products' absolute sums
        x, A, B, dy = (v.double().abs() for v in (g.x, g.A, g.B, g.dy))
        step = (high - low).abs()
        for e in range(g.e):
            r = g.rows(e)
            u = g.s * (dy[r] @ B[e])
            size = (u.T @ x[r] if param is g.A else dy[r].T @ (g.s * x[r] @ A[e].T) if param is g.B else dy[r] @ W[e] + u @ A[e])
            err += 2 * terms * 2.0 ** -23 * float((size * (step[r] if param is g.x else step[e])).sum())
        assert abs((up - down) - want) <= err, (up - down, want, err)


@pytest.mark.parametrize("counts", [[2, 0, 1, 3], [100, 7, 260, 33]])
def test_streams_and_graphs(cuda_device, counts):
    """Calls on another stream, two captured graphs and an eager call between their replays share no scratch."""
    import torch
    stacks = [Stack(cuda_device, counts, 264, 320, 16, seed=s) for s in (1, 2)]
    want = []
    for g in stacks:
        y, t = g.fwd()
        want.append((y, t) + g.bwd(t=t))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, t = stacks[0].fwd()
        got = (y, t) + stacks[0].bwd(t=t)
    other = stacks[1].fwd(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    assert torch.equal(other[0], want[1][0])
    graphs, outs = [], []
    for g in stacks:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, t = g.fwd()
            out = (y, t) + g.bwd(t=t)
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for out in outs:
            for v in out:
                v.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        stacks[0].fwd()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_codes_on_a_16_byte_boundary(cuda_device):
    """Codes that start on a 16-byte boundary and no larger one (a slice of a bigger buffer)."""
    import torch
    for counts in ([3, 0, 2], [90, 0, 200]):
        g = Stack(cuda_device, counts, 264, 320, 16, dq=False, seed=13)
        y, t = g.fwd()
        want = (y, t) + g.bwd(t=t)
        buf = torch.empty(g.q.codes.numel() + 16, dtype=torch.uint8, device=cuda_device)
        assert buf.data_ptr() % 32 == 0
        buf[16:] = g.q.codes
        g.q.codes = buf[16:]
        y, t = g.fwd()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, t) + g.bwd(t=t)))


def test_two_threads(cuda_device):
    """Two host threads, each with a stream, on layers of their own."""
    import threading
    import torch
    stacks = [Stack(cuda_device, c, 264, 320, 16, seed=17) for c in ([2, 0, 1], [70, 5, 140])]
    want = []
    for g in stacks:
        y, t = g.fwd()
        want.append((y, t) + g.bwd(t=t))
    torch.cuda.synchronize()
    wrong = []

    def work(g, w):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(40):
                y, t = g.fwd()
                got = (y, t) + g.bwd(t=t)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    wrong.append(1)
    threads = [threading.Thread(target=work, args=a) for a in zip(stacks, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_large_offsets_in_the_stack(cuda_device):
    """A stack of more than 2^32 weight elements: the last expert's codes lie past 32-bit element indexes."""
    import torch
    Q = _Q()
    e, n, k, r = 260, 4096, 4096, 8     # 4.36e9 elements, 2.2 GB of codes
    codes = torch.randint(0, 256, (e * n * k // 2,), dtype=torch.uint8, device=cuda_device)
    absmax = torch.rand(e * n * k // 64, device=cuda_device) * 0.05
    q = Q.QuantizedWeight(codes, absmax, None, None, e * n, k, 64, False)
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    mk = lambda *s: torch.randn(s, generator=gen, device=cuda_device).to(torch.bfloat16)
    A, B = mk(e, r, k) * 0.02, mk(e, n, r) * 0.01
    for count in (3, 140):
        counts = [0] * e
        counts[0] = counts[-1] = count
        off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=cuda_device)
        x, dy = mk(2 * count, k), mk(2 * count, n)
        y, t = Q.grouped_fwd(q, x, off, A, B, 16.0)
        _, _, dx = Q.grouped_bwd(q, x, off, A, B, 16.0, dy, t=t)
        for i in (0, e - 1):
            rows = slice(0, count) if i == 0 else slice(count, 2 * count)
            one = Q.QuantizedWeight(codes[i * n * k // 2:(i + 1) * n * k // 2], absmax[i * n * k // 64:(i + 1) * n * k // 64],
                                    None, None, n, k, 64, False)
            yd, td = Q.linear_fwd(one, x[rows].contiguous(), A[i], B[i], 16.0)
            _, _, dxd = Q.linear_bwd(one, x[rows].contiguous(), A[i], B[i], 16.0, dy[rows].contiguous(), t=td)
            for a, b in ((y[rows], yd), (dx[rows], dxd)):
                err = float((a.double() - b.double()).norm() / b.double().norm())
                assert err < 2.0 ** -7, err      # two roundings to bf16 apart
