"""CPU checks of the binding's scratch: what calls from several host threads are handed.

The library is replaced by one that records each call's workspace while the call runs; no GPU is touched.  A call
enqueues several kernels that hand results to each other through its scratch, so two calls that enqueue at the same
time must not hold the same memory, on one stream or on several."""
import threading
import time

import pytest
import torch

from qlora_linear_layers_nf4_b200 import nf4qlora as Q

E, N, K, R, M = 2, 64, 64, 8, 5


class RecordingLibrary:
    """Entry points that take a while; `shared` counts calls that ran while another held the same workspace."""

    def __init__(self):
        self.guard = threading.Lock()
        self.active = []
        self.shared = 0
        self.calls = 0

    def nf4_workspace_bytes(self, op, m, n, k, r, block_size, double_quant):
        return 256 + 64 * m

    def __getattr__(self, name):
        if name not in ("qlora_grouped_fwd", "qlora_grouped_bwd", "int8_linear_fwd", "qlora_linear_fwd", "qlora_linear_bwd",
                        "nf4_quantize"):
            raise AttributeError(name)

        def call(*args):
            ws = getattr(args[-3], "value", args[-3])
            with self.guard:
                self.shared += ws in self.active
                self.active.append(ws)
                self.calls += 1
            time.sleep(0.002)
            with self.guard:
                self.active.remove(ws)
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    fake = RecordingLibrary()
    stream = threading.local()
    monkeypatch.setattr(Q, "lib", lambda: fake)
    monkeypatch.setattr(Q, "_here", lambda device: getattr(stream, "handle", 0))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(Q, "_sizes", {})
    if hasattr(Q, "_stream_ws"):
        monkeypatch.setattr(Q, "_stream_ws", {})
    fake.stream = stream
    return fake


def _operands(m):
    bf = torch.bfloat16
    q = Q.QuantizedWeight(codes=torch.zeros(E * N * K // 2, dtype=torch.uint8), absmax=torch.zeros(E * N * K // 64),
                          absmax_q=None, absmax_scale=None, rows=E * N, cols=K, block_size=64, double_quant=False)
    off = torch.tensor([0, m // 2, m], dtype=torch.int32)
    return (q, torch.zeros(m, K, dtype=bf), off, torch.zeros(E, R, K, dtype=bf), torch.zeros(E, N, R, dtype=bf), 16.0)


def _calls(m, workspace=None):
    args = _operands(m)
    dy = torch.zeros(m, N, dtype=torch.bfloat16)
    w8 = Q.Int8Matrix(torch.zeros(N, K, dtype=torch.int8), torch.ones(N))
    return (lambda: Q.grouped_fwd(*args, workspace=workspace), lambda: Q.grouped_bwd(*args, dy, workspace=workspace),
            lambda: Q.int8_linear_fwd(w8, args[1], workspace=workspace))


def _run(fake, threads, handles, workspace=None):
    def work(i):
        fake.stream.handle = handles[i]
        for _ in range(5):
            for call in _calls(M * (i + 1), workspace):    # sizes differ, so scratch grows on the way
                call()
    pool = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    assert fake.calls == threads * 15


def test_threads_on_one_stream(recorder):
    _run(recorder, 4, [0] * 4)
    assert recorder.shared == 0


def test_threads_with_one_workspace(recorder):
    _run(recorder, 4, [0] * 4, Q.Workspace(torch.device("cpu")))
    assert recorder.shared == 0


def test_threads_on_their_own_streams(recorder):
    _run(recorder, 4, [1, 2, 3, 4])
    assert recorder.shared == 0


def test_growing_keeps_the_status():
    ws = Q.Workspace(torch.device("cpu"))
    ws.get(256)[0] = 8
    grown = ws.get(5000)
    assert grown.numel() == 5000 and grown[0] == 8 and not grown[1:].any()


def test_workspace_copies_have_their_own_lock():
    import copy
    ws = Q.Workspace(torch.device("cpu"))
    ws.get(300)[5] = 1
    other = copy.deepcopy(ws)
    assert other.lock is not ws.lock and torch.equal(other.buf, ws.buf) and other.buf is not ws.buf


def test_status_on_device_refuses():
    assert Q.lib().nf4_status_on_device(2) == 1 and Q.lib().nf4_status_on_device(-1) == 1
    assert Q.lib().nf4_status_on_device(0) == 0


@pytest.mark.parametrize("own_workspace", [False, True])
def test_threads_in_the_dense_calls(recorder, monkeypatch, own_workspace):
    """quantize, linear_fwd and linear_bwd on one stream, as above."""
    monkeypatch.setattr(Q, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(Q, "_default_ws", {})
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)   # quantize takes CUDA tensors only
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws = Q.Workspace(torch.device("cpu")) if own_workspace else None

    def work(i):
        bf, m = torch.bfloat16, M * (i + 1)
        q = Q.QuantizedWeight(codes=torch.zeros(N * K // 2, dtype=torch.uint8), absmax=torch.zeros(N * K // 64),
                              absmax_q=None, absmax_scale=None, rows=N, cols=K, block_size=64, double_quant=False)
        x, A, B, dy = (torch.zeros(s, dtype=bf) for s in ((m, K), (R, K), (N, R), (m, N)))
        for _ in range(5):
            Q.linear_fwd(q, x, A, B, 16.0, workspace=ws)
            Q.linear_bwd(q, x, A, B, 16.0, dy, workspace=ws)
            Q.quantize(torch.zeros(m, 64), 64, True, workspace=ws)
    pool = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    assert recorder.calls == 60 and recorder.shared == 0


def test_workspace_of_another_device_is_refused(recorder):
    """A pointer of another device, or of the host, would reach the kernels unseen."""
    elsewhere = Q.Workspace(torch.device("meta"))
    for call in _calls(M, elsewhere):
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert recorder.calls == 0
