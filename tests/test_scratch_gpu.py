"""Scratch of the expert and 8-bit calls on the GPU: several host threads on one stream, bits compared with the same
calls made alone."""
import threading

import pytest

from tests.test_grouped_gpu import Stack, _Q

pytestmark = pytest.mark.gpu


def _together(jobs, rounds):
    """Runs the jobs' calls in threads of their own that share the current stream; names what differed."""
    import torch
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    start, wrong = threading.Barrier(len(jobs)), []

    def work(i):
        try:
            with torch.cuda.stream(stream):
                torch.cuda.synchronize()   # the thread has used the device before
                start.wait(60)
                got = [jobs[i]() for _ in range(rounds)]
                torch.cuda.synchronize()
                if not all(torch.equal(a, b) for outs in got for a, b in zip(outs, want[i])):
                    wrong.append(i)
        except Exception as error:
            wrong.append((i, error))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("own_workspace", [False, True])
def test_threads_on_one_stream(cuda_device, own_workspace):
    """Decode, GEMM, backward (T recomputed) and 8-bit calls of different sizes."""
    import torch
    Q = _Q()
    ws = Q.Workspace(cuda_device) if own_workspace else None
    few, more, many = (Stack(cuda_device, c, 1032, 1088, 16, seed=s) for s, c in enumerate(([2, 0, 1, 2], [9, 30, 1, 16], [70, 5, 140, 33])))
    gen = torch.Generator(device=cuda_device).manual_seed(4)
    w8 = Q.int8_quantize(torch.randn(1032, 1088, generator=gen, device=cuda_device))
    x8 = [torch.randn(m, 1088, generator=gen, device=cuda_device).to(torch.bfloat16) for m in (9, 130)]
    jobs = [lambda g=g: g.fwd(want_t=False, workspace=ws)[:1] for g in (few, more, many)]
    jobs += [lambda g=g: g.bwd(workspace=ws) for g in (few, many)]
    jobs += [lambda x=x: (Q.int8_linear_fwd(w8, x, workspace=ws),) for x in x8]
    _together(jobs, 25)


def test_dense_calls_of_threads_on_one_stream(cuda_device):
    """The dense layer's calls, which share the device's default workspace."""
    import torch
    Q = _Q()
    g = Stack(cuda_device, [150, 70], 264, 320, 16, dq=False, seed=2)
    q = Q.QuantizedWeight(g.q.codes[:264 * 160], g.q.absmax[:264 * 5], None, None, 264, 320, 64, False)
    x, dy, A, B = g.x, g.dy, g.A[0], g.B[0]
    w = torch.randn(264, 320, device=cuda_device)
    jobs = [lambda m=m: Q.linear_fwd(q, x[:m], A, B, 32.0, want_t=False)[:1] for m in (4, 100, 220)]
    jobs += [lambda m=m: Q.linear_bwd(q, x[:m], A, B, 32.0, dy[:m]) for m in (40, 220)]
    jobs += [lambda m=m: (lambda r: (r.codes, r.absmax_q, r.absmax_scale))(Q.quantize(w[:m], 64, True)) for m in (30, 264)]
    _together(jobs, 25)
