"""The expert layer with few rows an expert (M <= 16 E), where the weights are streamed: both row widths (8 rows a pass
for M <= 8 or M <= 6 E, 16 else), shares that split tiles, rows of no expert, special values, bad offsets.  Bounds as
in test_grouped_gpu."""
import pytest

from tests.test_grouped_gpu import Stack, _Q, _dt

pytestmark = pytest.mark.gpu

# counts (M, M / E decide the width), n, k, r
WIDE = [
    ([12, 0, 16, 9], 264, 320, 24),            # one pass an expert, N and K off the tile and chunk
    ([30, 0, 3, 20], 1032, 1088, 72),          # several passes, 225 units: shares split tiles
    ([7, 8, 9, 10, 11, 12, 13, 14], 136, 64, 8),   # one chunk a row
    ([1, 0, 0, 31], 2056, 2048, 16),           # whole chunks, vector scales, rings that wrap
    ([16] * 8, 520, 4160, 256),                # every pass full, the widest adapter
    ([17, 0, 0, 0, 30, 1], 8, 6528, 40),       # one 128-row tile, many chunks: one tile over many shares
]
NARROW = [
    ([8], 264, 320, 24),
    ([3, 0, 2, 7], 1032, 1088, 72),
    ([6] * 8, 136, 64, 8),
    ([1, 0, 0, 9], 2056, 2048, 16),
    ([5, 6, 0, 7], 520, 4160, 256),
    ([0, 0, 20, 0, 3, 1], 8, 6528, 40),
]


def _np(counts):
    m, e = sum(counts), len(counts)
    assert m <= 16 * e
    return 8 if m <= 8 or m <= 6 * e else 16


def test_the_cases_reach_both_widths():
    assert all(_np(c) == 16 for c, *_ in WIDE) and all(_np(c) == 8 for c, *_ in NARROW)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dq", [False, True])
@pytest.mark.parametrize("counts,n,k,r", WIDE + NARROW)
def test_forward(cuda_device, counts, n, k, r, dq, dtype):
    import torch
    g = Stack(cuda_device, counts, n, k, r, dtype, dq=dq, bias=True, seed=len(counts) + dq)
    ws = _Q().Workspace(cuda_device)
    y, t = g.fwd(workspace=ws)
    g.check_fwd(y, t)
    for _ in range(10):
        again, _ = g.fwd(workspace=ws)
        assert torch.equal(again, y)
    assert ws.read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block,dq", [(128, False), (512, True), (4096, False)])
@pytest.mark.parametrize("counts", [[12, 0, 16, 9], [3, 0, 2, 7]])
def test_blocks_over_rows_and_experts(cuda_device, counts, block, dq, dtype):
    g = Stack(cuda_device, counts, 40, 1088, 8, dtype, block=block, dq=dq, seed=block)
    y, t = g.fwd()
    g.check_fwd(y, t)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[3, 0, 2, 1, 0, 4, 2, 1], [9, 0, 12, 3, 20, 4, 2, 11]])
def test_rows_of_no_expert(cuda_device, counts, dtype):
    """NaN rows before the first and behind the last expert stay as they are and reach nothing; so does a row's
    neighbour in the same pass."""
    import torch
    g = Stack(cuda_device, counts, 1032, 1088, 24, dtype, lead=5, pad=7, seed=11)
    assert _np([g.m] + [0] * 7) == (8 if g.m < 48 else 16)
    outside = torch.ones(g.m, dtype=torch.bool)
    outside[g.off[0]:g.off[-1]] = False
    dev_out = outside.to(cuda_device)
    clean, _ = g.fwd(out=torch.full((g.m, 1032), 7.0, dtype=_dt(dtype), device=cuda_device))
    g.x[dev_out] = float("nan")
    mk = lambda c: torch.full((g.m, c), 7.0, dtype=_dt(dtype), device=cuda_device)
    y, t = g.fwd(out=mk(1032), t_out=mk(24))
    g.check_fwd(y, t)
    assert torch.equal(y, clean)
    assert (y[dev_out] == 7).all() and (t[dev_out] == 7).all()
    row = int(g.off[0]) + 1                       # one bad row of the first expert
    g.x[row] = float("inf")
    y2, t2 = g.fwd(out=mk(1032), t_out=mk(24))
    keep = [i for i in range(g.m) if i != row]
    assert torch.equal(y2[keep], y[keep]) and torch.equal(t2[keep], t[keep])
    assert not torch.isfinite(y2[row].float()).any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[9, 10, 11], [5, 6, 7], [40, 50, 60]])
def test_bad_offsets(cuda_device, counts, dtype):
    """Clamped and reported by both widths and by the GEMM, forward and backward."""
    import torch
    Q = _Q()
    g = Stack(cuda_device, counts, 264, 320, 16, dtype, seed=2)
    m, a, b = g.m, counts[0], counts[0] + counts[1]
    for bad, as_if in (([0, b, a, m], [0, b, b, m]), ([-3, a, b, m], [0, a, b, m]), ([0, a, b, 1 << 30], [0, a, b, m]),
                       ([0, m + 9, a, b], [0, m, m, m]), ([-2 ** 31, 2 ** 31 - 1, 0, 0], [0, m, m, m])):
        res = []
        for off in (bad, as_if):
            ws = Q.Workspace(cuda_device)
            g.offsets = torch.tensor(off, dtype=torch.int32, device=cuda_device)
            y, t = g.fwd(out=torch.zeros(m, 264, dtype=_dt(dtype), device=cuda_device), workspace=ws)
            code = ws.read_status()
            dA, dB, dx = g.bwd(t=t, workspace=ws)
            res.append((y, t, dA, dB, dx))
            assert code == ws.read_status() == (1 if off is bad else 0)
        assert all(torch.equal(u, v) for u, v in zip(*res))


@pytest.mark.parametrize("counts", [[128, 0, 0, 0, 0, 0, 0, 0], [0] * 7 + [100], [64, 64, 0, 0, 0, 0, 0, 0]])
def test_all_rows_on_few_experts(cuda_device, counts):
    """The rule goes by the average; an expert may have all the rows."""
    g = Stack(cuda_device, counts, 1032, 1088, 16, seed=4)
    y, t = g.fwd()
    g.check_fwd(y, t)


def test_captured_split_tiles(cuda_device):
    """The counters of split tiles are cleared in every replay, whichever kernel made T."""
    import torch
    for counts, r in (([30, 0, 3, 20], 72), ([1, 0, 0, 2], 8)):
        g = Stack(cuda_device, counts, 1032, 2112, r, seed=5)
        want, _ = g.fwd()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y1, _ = g.fwd()
            y2, _ = g.fwd(want_t=False)
        for _ in range(5):
            y1.zero_(), y2.zero_()
            graph.replay()
            assert torch.equal(y1, want) and torch.equal(y2, want)
