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
