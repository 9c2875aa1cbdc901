"""What the GPU found in calls made without a workspace: eager ones, captured ones, and after scratch has grown."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from tests.test_grouped_gpu import Stack, _Q

pytestmark = pytest.mark.gpu


def _stack(dev, counts=(5, 6, 7)):
    return Stack(dev, list(counts), 64, 128, 8, seed=2)


@pytest.mark.parametrize("counts", [(5, 6, 7), (90, 60, 70)])
def test_eager_calls(cuda_device, counts):
    import torch
    Q = _Q()
    g = _stack(cuda_device, counts)
    Q.read_status()
    y, t = g.fwd()
    g.bwd(t=t)
    assert Q.read_status() == 0
    g.offsets[1] = g.m + 1
    for call in (lambda: g.fwd(), lambda: g.bwd(t=t)):
        call()
        assert Q.read_status() == 1 and Q.read_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.fwd(stream=side)
    assert Q.read_status() == 0 and Q.read_status(side) == 1 and Q.read_status(side) == 0


def test_growing_scratch_keeps_the_status(cuda_device):
    import torch
    Q = _Q()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g, big = _stack(cuda_device), _stack(cuda_device, (3000, 4000, 500))
        Q.read_status()
        good = g.offsets.clone()
        g.offsets[1] = 99
        g.bwd()
        g.offsets.copy_(good)
        big.bwd()
        assert Q.read_status() == 1 and Q.read_status() == 0


@pytest.mark.parametrize("counts", [(5, 6, 7), (90, 60, 70)])
def test_captured_calls(cuda_device, counts):
    """Every replay records again; a given workspace keeps its own word."""
    import torch
    Q = _Q()
    g = _stack(cuda_device, counts)
    good = g.offsets.clone()
    ws = Q.Workspace(cuda_device)
    _, t = g.fwd(workspace=ws)
    g.bwd(t=t, workspace=ws)
    Q.read_status()
    graphs = []
    for space in (None, ws):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, t = g.fwd(workspace=space)
            g.bwd(t=t, workspace=space)
        graphs.append((graph, y, t))
    bad = good.clone()
    bad[1] = g.m + 1
    for offsets, code in ((good, 0), (bad, 1), (bad, 1), (good, 0)):
        g.offsets.copy_(offsets)
        graphs[0][0].replay()
        assert ws.read_status() == 0 and Q.read_status() == code
        graphs[1][0].replay()
        assert Q.read_status() == 0 and ws.read_status() == code
    assert torch.equal(graphs[0][1], graphs[1][1])
    # an eager call with a workspace still records there
    g.offsets.copy_(bad)
    g.fwd(workspace=ws)
    assert Q.read_status() == 0 and ws.read_status() == 1


def test_first_call_of_a_process_is_captured():
    """No eager call before: the status word has to be there all the same."""
    code = """
import torch
from qlora_linear_layers_nf4_b200 import nf4qlora as Q
dev = torch.device("cuda:0")
q = Q.QuantizedWeight(torch.zeros(2 * 64 * 64, dtype=torch.uint8, device=dev), torch.ones(2 * 2 * 64, device=dev), None, None, 4 * 64, 64, 64, False)
bf = torch.bfloat16
x, A, B = torch.ones(9, 64, dtype=bf, device=dev), torch.ones(4, 8, 64, dtype=bf, device=dev), torch.ones(4, 64, 8, dtype=bf, device=dev)
off = torch.tensor([0, 4, 3, 9, 9], dtype=torch.int32, device=dev)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, t = Q.grouped_fwd(q, x, off, A, B, 16.0)
g.replay()
assert Q.read_status() == 1 and Q.read_status() == 0
off[2] = 5
g.replay()
assert Q.read_status() == 0
want, _ = Q.grouped_fwd(q, x, off, A, B, 16.0)
assert torch.equal(y, want)
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ), capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stdout + done.stderr
