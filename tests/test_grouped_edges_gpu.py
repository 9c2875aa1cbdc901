"""Edges of the expert layer: calls without a live row, special values, and the two widths of the decode kernel."""
import pytest

from tests.test_grouped_gpu import Stack, _dt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_no_live_row_among_many(cuda_device, dtype):
    """Rows enough for the GEMM, none of them an expert's; the offsets are overwritten right behind the calls.

    The GEMM is launched while the kernel before it still runs.  With no tile to compute it has to wait for that
    kernel all the same: the copy into the offsets is ordered behind the GEMM alone."""
    import torch
    g = Stack(cuda_device, [0, 0, 0], 136, 192, 16, dtype, lead=40, pad=60, seed=3)
    empty, full = g.offsets.clone(), torch.tensor([0, 30, 60, 100], dtype=torch.int32, device=cuda_device)
    sevens = lambda c: torch.full((100, c), 7.0, dtype=_dt(dtype), device=cuda_device)
    y, t, dx = sevens(136), sevens(16), sevens(192)
    for _ in range(50):
        g.offsets.copy_(empty)
        g.fwd(out=y, t_out=t)
        g.offsets.copy_(full)
        g.offsets.copy_(empty)
        dA, dB, _ = g.bwd(t=t, dx=dx)
        g.offsets.copy_(full)
        assert not dA.any() and not dB.any()
        assert (y == 7).all() and (t == 7).all() and (dx == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[3, 0, 2], [150, 0, 70]])
def test_infinite_gradients_keep_their_sign(cuda_device, dtype, counts):
    """One infinite dy: U's row is infinite, and dA is then infinite with the sign of U x, as the formula gives."""
    import numpy as np
    import torch
    g = Stack(cuda_device, counts, 72, 128, 8, dtype, seed=9)
    _, t = g.fwd()
    g.dy[1, 5] = float("inf")
    g.dyn[1, 5] = np.inf
    assert (g.Bn[0][5] != 0).all() and (g.xn[1] != 0).all()
    dA, dB, dx = g.bwd(t=t)
    u = g.s * (g.dyn[g.rows(0)] @ g.Bn[0])
    with np.errstate(invalid="ignore"):
        want = u.T @ g.xn[g.rows(0)]
    assert np.isinf(want).all()
    assert np.array_equal(dA[0].double().cpu().numpy(), want)
    assert torch.isfinite(dA[2]).all()
    te = t.double().cpu().numpy()[g.rows(0)]
    assert (te[1] != 0).all()
    assert np.array_equal(np.isinf(dB[0].cpu().numpy()), np.isinf(g.dyn[g.rows(0)].T @ te))


@pytest.mark.parametrize("counts", [[3, 0, 2], [150, 0, 70]])
def test_f16_gradients_past_the_range(cuda_device, counts):
    """|U| above f16's largest value counts as infinite; it makes no NaN."""
    import torch
    g = Stack(cuda_device, counts, 72, 128, 8, "f16", seed=10)
    _, t = g.fwd()
    g.B[0, 5] = 40.0
    g.dy[1, 5] = 4096.0                      # U of that row: 2 * 4096 * 40 = 327,680, and little more
    g.dy[1, 6:] = 0
    dA, _, _ = g.bwd(t=t)
    assert torch.equal(dA[0], torch.sign(g.x[1].float()).expand(8, 128) * float("inf"))


@pytest.mark.parametrize("counts", [[3, 0, 2], [150, 0, 70]])
def test_f16_small_gradients(cuda_device, counts):
    """U around 2^-20, below f16's normal range: dA within U's absolute step, 2^-36."""
    g = Stack(cuda_device, counts, 72, 128, 8, "f16", seed=12)
    for v in (g.dy, g.B):
        v.mul_(2.0 ** -9)
    g.dyn, g.Bn = g.dy.double().cpu().numpy(), g.B.double().cpu().numpy()
    _, t = g.fwd()
    g.check_bwd(*g.bwd(t=t, want_dx=False), t)
