"""The first library call of a host thread that has not used the GPU before."""
import threading

import pytest

from tests.test_grouped_gpu import Stack, _Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["grouped_decode", "grouped_gemm", "grouped_bwd", "int8_small", "int8_gemm",
                                  "int8_quantize", "dense_decode", "dense_gemm", "dense_bwd", "merge"])
def test_first_call_of_a_thread(cuda_device, name):
    import torch
    Q = _Q()
    few, many = Stack(cuda_device, [2, 0, 1], 264, 320, 16, dq=False), Stack(cuda_device, [70, 5, 140], 264, 320, 16, dq=False)
    w8, x = Q.int8_quantize(torch.randn(264, 320, device=cuda_device)), many.x
    dense = Q.QuantizedWeight(many.q.codes[:264 * 160], many.q.absmax[:264 * 5], None, None, 264, 320, 64, False)
    A, B = many.A[0], many.B[0]
    ws = Q.Workspace(cuda_device)
    call = {
        "grouped_decode": lambda: few.fwd(workspace=ws), "grouped_gemm": lambda: many.fwd(workspace=ws),
        "grouped_bwd": lambda: many.bwd(workspace=ws), "int8_small": lambda: (Q.int8_linear_fwd(w8, x[:2], workspace=ws),),
        "int8_gemm": lambda: (Q.int8_linear_fwd(w8, x, workspace=ws),),
        "int8_quantize": lambda: (Q.int8_quantize(x).codes,),
        "dense_decode": lambda: Q.linear_fwd(dense, x[:4], A, B, 32.0), "dense_gemm": lambda: Q.linear_fwd(dense, x, A, B, 32.0),
        "dense_bwd": lambda: Q.linear_bwd(dense, x, A, B, 32.0, many.dy), "merge": lambda: (Q.merge(dense, A, B, 32.0),),
    }[name]
    want = call()
    call()                   # leaves memory of the outputs' sizes with the allocator, so that the thread needs no more
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            got.extend(call())
        except Exception as error:
            failed.append(error)
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
