"""Edges of the gated feed-forward layer: empty batches, values that are not finite, far
pre-activations, given outputs, streams, captured graphs, host threads, the block it is part
of, and gradients against differences."""
import math

import pytest

from tests.test_gated_gpu import F, HALF, Layer, _Q, _dt, logistic_parts, ok_status
from tests.test_scratch_gpu import _together

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_empty_batch(cuda_device, dtype):
    import torch
    Q = _Q()
    L = Layer(cuda_device, 4, 72, 128, 16, dtype)
    L.x, L.dh = L.x[:0], L.dh[:0]
    h, saved = L.fwd()
    assert h.shape == (0, 72) and saved.pre.shape == (2, 0, 72) and saved.t.shape == (2, 0, 16)
    dA, dB = (torch.full(s, 7.0, device=cuda_device) for s in ((2, 16, 128), (2, 72, 16)))
    a, b, dx = L.bwd(saved, dA=dA, dB=dB)
    assert a is dA and b is dB and dx.shape == (0, 128)
    assert not dA.any() and not dB.any()
    ok_status()


@pytest.mark.parametrize("m", [3, 20, 40, 300])
def test_tokens_that_are_not_finite_stay_alone(cuda_device, m):
    import torch
    L = Layer(cuda_device, m, 264, 192, 24)
    want, saved = L.fwd()
    good = L.bwd(saved)[2]
    x = L.x.clone()
    x[1, 5], x[m - 1, 100] = float("inf"), float("nan")
    L.x = x
    h, bad = L.fwd()
    rows = torch.ones(m, dtype=torch.bool, device=cuda_device)
    rows[1] = rows[m - 1] = False
    assert h[rows].equal(want[rows]) and bad.pre[:, rows].equal(saved.pre[:, rows]) and bad.t[:, rows].equal(saved.t[:, rows])
    assert not torch.isfinite(h[~rows]).any()
    dx = L.bwd(bad)[2]
    assert dx[rows].equal(good[rows]) and not torch.isfinite(dx[~rows]).any()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,dtype", [(2, "bf16"), (40, "bf16"), (40, "f16"), (300, "bf16"), (5, "f32")])
def test_far_pre_activations(cuda_device, act, m, dtype):
    """Biases that take g from far below to far above what the exponential covers."""
    import torch
    L = Layer(cuda_device, m, 256, 64, 8, dtype, bias=True, act=act)
    far = [0.0, 1e-3, 5.0, 20.0, 40.0, 80.0, 87.5, 90.0, 104.0, 200.0, 3e4]
    L.bias[0] = torch.tensor([s * f for f in far for s in (1, -1)] * 12)[:256].to(L.bias.dtype)
    h, saved = L.fwd()
    L.check_fwd(h, saved)
    if dtype == "f16":
        L.dh /= 16      # du, up to 3e4 |dh|, stays within the type
    dA, dB, dx = L.bwd(saved)
    L.check_bwd(dA, dB, dx, saved)


def test_gradients_of_infinite_pre_activations(cuda_device):
    """d of an infinite value is infinite or NaN, in its token's dx alone, and in sums over tokens."""
    import torch
    for act in ("silu", "gelu_tanh"):
        L = Layer(cuda_device, 70, 136, 128, 16, act=act)
        _, saved = L.fwd()
        good = L.bwd(saved)
        saved.pre[1, 2, 3] = float("inf")          # u: dg is infinite
        dA, dB, dx = L.bwd(saved)
        rows = torch.arange(70, device=cuda_device) != 2
        assert dx[rows].equal(good[2][rows]) and not torch.isfinite(dx[2]).any()
        other = torch.arange(136, device=cuda_device) != 3
        assert dB[:, other].equal(good[1][:, other]) and dB[1].equal(good[1][1])
        assert not torch.isfinite(dB[0, 3]).any() and dB[0, 3].isinf().any()


@pytest.mark.parametrize("m,n", [(5, 264), (77, 264), (300, 5000)])
def test_given_outputs_and_rows_behind(cuda_device, m, n):
    import torch
    Q = _Q()
    L = Layer(cuda_device, m, n, 128, 16)
    want, kept = L.fwd()
    big = torch.full((m + 40, n), 7.0, dtype=torch.bfloat16, device=cuda_device)
    saved = Q.GatedSaved(torch.full_like(kept.pre, 7.0), None)      # T is left out
    h, got = L.fwd(out=big[:m], saved=saved)
    assert got is saved and h.data_ptr() == big.data_ptr()
    assert h.equal(want) and saved.pre.equal(kept.pre) and (big[m:] == 7).all()
    grads = L.bwd(kept)
    wide = torch.full((m + 40, 128), 7.0, dtype=torch.bfloat16, device=cuda_device)
    again = L.bwd(saved, dx=wide[:m])
    assert all(a.equal(b) for a, b in zip(grads, again)) and (wide[m:] == 7).all()


def test_same_inputs_same_bits(cuda_device):
    for m, n, k, r, dtype in ((1, 520, 2048, 16, "bf16"), (13, 2056, 1024, 72, "f16"), (70, 4000, 512, 128, "bf16"),
                              (600, 3000, 1024, 64, "bf16")):
        L = Layer(cuda_device, m, n, k, r, dtype)
        first, saved = L.fwd()
        grads = L.bwd(saved)
        for _ in range(5):
            h, s = L.fwd()
            assert h.equal(first) and s.pre.equal(saved.pre) and s.t.equal(saved.t)
            assert all(a.equal(b) for a, b in zip(grads, L.bwd(saved)))


@pytest.mark.parametrize("m", [2, 50, 400])
def test_other_stream(cuda_device, m):
    import torch
    L = Layer(cuda_device, m, 520, 256, 16)
    want, saved = L.fwd()
    grads = L.bwd(saved)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h, s = L.fwd(stream=side)
    got = L.bwd(s, stream=side)
    side.synchronize()
    assert h.equal(want) and all(a.equal(b) for a, b in zip(grads, got))
    assert _Q().read_status(side) == 0


@pytest.mark.parametrize("m", [2, 50, 400])
def test_captured_calls(cuda_device, m):
    """Two graphs, each a forward and a backward, replayed in turn with eager calls between."""
    import torch
    Ls = [Layer(cuda_device, m, 520, 256, 16, seed=s) for s in range(2)]
    eager = [(lambda h, s: (h,) + L.bwd(s))(*L.fwd()) for L in Ls]
    torch.cuda.synchronize()
    graphs = []
    for L in Ls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h, s = L.fwd()
            out = (h,) + L.bwd(s)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
        between = Ls[0].fwd()[0]
        torch.cuda.synchronize()
        assert between.equal(eager[0][0])
        for (g, out), want in zip(graphs, eager):
            assert all(a.equal(b) for a, b in zip(out, want))
    for L, (g, out) in zip(Ls, graphs):      # other inputs in the same tensors
        L.x.copy_(L.x.flip(0))
        g.replay()
        h, s = L.fwd()
        torch.cuda.synchronize()
        assert out[0].equal(h)
    ok_status()


def test_threads_on_one_stream(cuda_device):
    import torch
    Q = _Q()
    ws = Q.Workspace(cuda_device)
    Ls = [Layer(cuda_device, m, 520, 256, 16, seed=m) for m in (3, 40, 300)]
    saved = [L.fwd()[1] for L in Ls]
    w8 = Q.fp8_quantize(torch.randn(264, 320, device=cuda_device), 128)
    x8 = [torch.randn(m, 320, device=cuda_device).to(torch.bfloat16) for m in (2, 7, 130)]
    for space in (None, ws):
        jobs = [lambda L=L: L.fwd(want_saved=False, workspace=space)[:1] for L in Ls]
        jobs += [lambda L=L, s=s: L.bwd(Q.GatedSaved(s.pre, None), workspace=space) for L, s in zip(Ls, saved)]
        jobs += [lambda x=x: (Q.fp8_linear_fwd(w8, x, workspace=space),) for x in x8]
        _together(jobs, 15)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(cuda_device, act):
    """fp32 mode: the derivative along a direction against central differences of the loss.  With step 2^-6 the
    differences are off by their third-order term, step^2 / 6 times a third derivative, and by the loss's rounding:
    2e-3 of the size of what is summed covers both (the layer's values are of order 1)."""
    import torch
    L = Layer(cuda_device, 37, 72, 64, 8, "f32", act=act)
    _, saved = L.fwd()
    dA, dB, dx = L.bwd(saved)
    eps = 2.0 ** -6
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    for name, grad in (("A", dA), ("B", dB), ("x", dx)):
        base = getattr(L, name)
        way = torch.randn(base.shape, generator=gen, device=cuda_device) * base.abs().mean()
        loss = []
        for sign in (1, -1):
            setattr(L, name, base + sign * eps * way)
            loss.append((L.fwd(want_saved=False)[0].double() * L.dh.double()).sum().item())
        setattr(L, name, base)
        parts = grad.double() * way.double()
        got = (loss[0] - loss[1]) / (2 * eps)
        assert abs(got - parts.sum().item()) <= 2e-3 * parts.abs().sum().item(), name


def test_feed_forward_block(cuda_device):
    """A block as it is trained: gate and up with the product (gated_fwd), down (linear_fwd), and backwards, against
    autograd in 64 bits with the same dequantized weights.  The steps between round to bf16 (h, g and u, T, dh, dg and
    du, U), half a step 2^-8 each and at most eight of them on a path, so the error's norm is within 8 * 2^-8 of the
    result's where the sums do not cancel; the norms of sums of random signs do not."""
    import torch
    Q = _Q()
    m, n, k, r = 200, 576, 256, 16
    L = Layer(cuda_device, m, n, k, r)
    gen = torch.Generator().manual_seed(3)
    t = lambda *s, sigma=1.0: (torch.randn(*s, generator=gen) * sigma).to(torch.bfloat16).to(cuda_device)
    down = Q.quantize((torch.randn(k, n, generator=gen) * 0.04).to(cuda_device), 64, True)
    Ad, Bd, dy = t(r, n, sigma=n ** -0.5), t(k, r, sigma=0.05), t(m, k)
    h, saved = L.fwd()
    y, td = Q.linear_fwd(down, h, Ad, Bd, L.alpha)
    dAd, dBd, dh = Q.linear_bwd(down, h, Ad, Bd, L.alpha, dy, t=td)
    L.dh = dh
    dA, dB, dx = L.bwd(saved)

    f64 = lambda v: v.double().clone().requires_grad_(True)
    x, A, B, a, b = map(f64, (L.x, L.A, L.B, Ad, Bd))
    Wd = Q.dequantize(down, "bf16").double()
    g, u = (x @ L.W[i].T + L.s * (x @ A[i].T) @ B[i].T for i in range(2))
    hw = g * torch.sigmoid(g) * u
    yw = hw @ Wd.T + L.s * (hw @ a.T) @ b.T
    (yw * dy.double()).sum().backward()
    for name, got, want in (("y", y, yw), ("dA down", dAd, a.grad), ("dB down", dBd, b.grad), ("dA", dA, A.grad),
                            ("dB", dB, B.grad), ("dx", dx, x.grad)):
        off = (got.double() - want).norm() / want.norm()
        assert off <= 8 * 2.0 ** -8, f"{name}: {off:.2e}"
    ok_status()


@pytest.mark.parametrize("m,n,k,r,dtype,act", [(33, 72, 4096, 8, "bf16", "silu"), (64, 1000, 2048, 24, "f16", "gelu_tanh"),
                                               (129, 136, 8192, 72, "bf16", "silu"), (257, 520, 1600, 256, "f16", "silu"),
                                               (300, 264, 4160, 16, "bf16", "gelu_tanh")])
def test_long_reductions_of_few_tiles(cuda_device, m, n, k, r, dtype, act):
    """Few output tiles share a long reduction over K among several CTA pairs, forward and (N long) backward."""
    import torch
    Q = _Q()
    L = Layer(cuda_device, m, n, k, r, dtype, bias=True, act=act)
    big = torch.full((m + 3, n), 7.0, dtype=_dt(dtype), device=cuda_device)
    h, saved = L.fwd(out=big[:m])
    L.check_fwd(h, saved)
    assert (big[m:] == 7).all()
    assert L.fwd(want_saved=False)[0].equal(h)
    L = Layer(cuda_device, m, k, 64, r, dtype, act=act)
    saved = L.fwd()[1]
    L.check_bwd(*L.bwd(saved), saved)
    ok_status()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_more_than_two_to_the_31_elements(cuda_device, dtype):
    """Offsets past 32 bits in h, g, u, dh, dg and du: the last rows, which alone have gradients, are checked."""
    import torch
    m, n, k = 70_041, 32_776, 64
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    L = Layer(cuda_device, 8, n, k, 8, dtype)
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    L.x = torch.randn(m, k, generator=gen, device=cuda_device).to(_dt(dtype))
    L.dh = torch.zeros(m, n, dtype=_dt(dtype), device=cuda_device)
    L.dh[-45:] = torch.randn(45, n, generator=gen, device=cuda_device).to(_dt(dtype))
    h, saved = L.fwd()
    for rows in (slice(0, 40), slice(m // 2, m // 2 + 40), slice(m - 45, m)):
        L.check_fwd(h, saved, rows)
    del h
    dA, dB, dx = L.bwd(saved)
    L.check_bwd(dA, dB, dx, saved, slice(m - 45, m))
    assert not dx[:-45].any()
    ok_status()
    del L, saved, dx
    torch.cuda.empty_cache()
