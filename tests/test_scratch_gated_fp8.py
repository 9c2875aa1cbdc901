"""CPU checks of the scratch that the gated and 8-bit floating point calls are handed, by several host threads: no two calls
hold the same memory while they enqueue, and a workspace of another device is refused."""
import threading

import pytest
import torch

from qlora_linear_layers_nf4_b200 import nf4qlora as Q
from tests.test_scratch import K, M, N, R, RecordingLibrary

NAMES = ("qlora_gated_fwd", "qlora_gated_bwd", "fp8_linear_fwd")


class Library(RecordingLibrary):
    def __getattr__(self, name):
        if name not in NAMES:
            raise AttributeError(name)
        return super().__getattr__("qlora_grouped_fwd")   # any that it records


@pytest.fixture
def fake(monkeypatch):
    lib, stream = Library(), threading.local()
    monkeypatch.setattr(Q, "lib", lambda: lib)
    monkeypatch.setattr(Q, "_here", lambda device: getattr(stream, "handle", 0))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(Q, "_sizes", {})
    monkeypatch.setattr(Q, "_stream_ws", {})
    lib.stream = stream
    return lib


def _calls(m, workspace=None):
    bf = torch.bfloat16
    q = Q.QuantizedWeight(torch.zeros(N * K // 2, dtype=torch.uint8), torch.zeros(N * K // 64), None, None, N, K, 64, False)
    x, A, B, dh = (torch.zeros(s, dtype=bf) for s in ((m, K), (2, R, K), (2, N, R), (m, N)))
    saved = Q.GatedSaved(torch.zeros(2, m, N, dtype=bf), torch.zeros(2, m, R, dtype=bf))
    w8 = Q.Fp8Matrix(torch.zeros(N, K, dtype=torch.float8_e4m3fn), torch.ones(1, 1), 128)
    return (lambda: Q.gated_fwd(q, q, x, A, B, 16.0, workspace=workspace),
            lambda: Q.gated_bwd(q, q, x, A, B, 16.0, dh, saved, workspace=workspace),
            lambda: Q.fp8_linear_fwd(w8, x, workspace=workspace))


@pytest.mark.parametrize("handles,own", [([0] * 4, False), ([0] * 4, True), ([1, 2, 3, 4], False)])
def test_threads(fake, handles, own):
    ws = Q.Workspace(torch.device("cpu")) if own else None

    def work(i):
        fake.stream.handle = handles[i]
        for _ in range(5):
            for call in _calls(M * (i + 1), ws):    # sizes differ, so scratch grows on the way
                call()
    pool = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    assert fake.calls == 60 and fake.shared == 0


def test_workspace_of_another_device_is_refused(fake):
    for call in _calls(M, Q.Workspace(torch.device("meta"))):
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert fake.calls == 0
