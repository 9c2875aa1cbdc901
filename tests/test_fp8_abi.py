"""CPU checks of the 8-bit floating point entry points: every refusal is made on the host, before the GPU is touched."""
import pytest

from qlora_linear_layers_nf4_b200 import nf4qlora as Q

FAKE = 0x10000   # aligned, never dereferenced: every call below fails validation first, or has nothing to do
BIG = 1 << 40


@pytest.mark.parametrize("call", [
    lambda x=FAKE, dt=1, rows=4, cols=16, br=1, c=FAKE, s=FAKE: Q.lib().fp8_quantize(x, dt, rows, cols, br, c, s, None),
    lambda x=FAKE, dt=1, rows=4, cols=16, br=1, c=FAKE, s=FAKE: Q.lib().fp8_dequantize(c, s, rows, cols, br, dt, x, None)])
def test_quantize_validation(call):
    assert call(dt=3) == 1 and call(dt=-1) == 1
    assert call(br=0) == 1 and call(br=64) == 1 and call(br=-128) == 1
    assert call(rows=-1) == 2 and call(cols=-1) == 2 and call(rows=(1 << 30) + 1) == 2 and call(cols=(1 << 30) + 1) == 2
    assert call(x=None) == 1 and call(c=None) == 1 and call(s=None) == 1
    assert call(x=FAKE + 8) == 3 and call(c=FAKE + 1) == 3 and call(s=FAKE + 2) == 3
    assert call(rows=0) == 0 and call(cols=0) == 0 and call(rows=0, x=None, c=None, s=None) == 0


def test_linear_validation():
    def lin(w=FAKE, s=FAKE, n=64, k=64, x=FAKE, xs=None, m=4, dt=1, bias=None, y=FAKE, ws=FAKE, wsb=BIG):
        return Q.lib().fp8_linear_fwd(w, s, n, k, x, xs, m, dt, bias, y, ws, wsb, None)

    assert lin(w=None) == 1 and lin(s=None) == 1 and lin(x=None) == 1 and lin(y=None) == 1
    assert lin(dt=3) == 1
    assert lin(n=60) == 2 and lin(n=0) == 2 and lin(k=24) == 2 and lin(k=0) == 2 and lin(k=(1 << 30) + 16) == 2
    assert lin(m=0) == 2 and lin(m=(1 << 30) + 1) == 2 and lin(n=(1 << 30) + 8) == 2
    assert lin(w=FAKE + 8) == 3 and lin(s=FAKE + 2) == 3 and lin(x=FAKE + 8) == 3 and lin(xs=FAKE + 1) == 3
    assert lin(y=FAKE + 8) == 3 and lin(bias=FAKE + 2) == 3
    assert lin(ws=None) == 5 and lin(ws=FAKE + 4) == 5
    need = Q.workspace_bytes(Q.OP_FP8_LINEAR, 4, 64, 64, 0, 0, False)
    assert need >= 256 + 4 * 64 + 4 * 4 and lin(wsb=need - 1) == 5
    assert Q.workspace_bytes(Q.OP_FP8_LINEAR, 33, 64, 272, 0, 0, False) >= 256 + 33 * 272 + 33 * 3 * 4


def test_binding_refusals():
    import torch
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    w = Q.Fp8Matrix(torch.zeros(264, 272, dtype=f8), torch.zeros(3, 3), 128)
    x = torch.zeros(5, 272, dtype=bf)
    q = Q.Fp8Matrix(torch.zeros(5, 272, dtype=f8), torch.zeros(5, 3), 1)
    for bad in (dict(x=x[0]), dict(block_rows=64), dict(codes=torch.zeros(5, 272, dtype=torch.uint8)), dict(scale=torch.zeros(5, 2)),
                dict(x=x.double()), dict(x=torch.zeros(5, 544, dtype=bf)[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            Q.fp8_quantize(**{**dict(x=x), **bad})
    for m in (Q.Fp8Matrix(q.codes, q.scale, 128), Q.Fp8Matrix(q.codes, torch.zeros(5, 2), 1), Q.Fp8Matrix(q.codes.view(torch.uint8), q.scale, 1),
              Q.Fp8Matrix(q.codes[0], q.scale, 1), Q.Fp8Matrix(q.codes, q.scale, 2)):
        with pytest.raises((ValueError, TypeError)):
            Q.fp8_dequantize(m)
    for bad in (dict(w=q), dict(w=Q.Fp8Matrix(w.codes, torch.zeros(3, 2), 128)), dict(x=x[:, :256]), dict(x=w), dict(x=x[0]),
                dict(x=Q.Fp8Matrix(q.codes, torch.zeros(4, 3), 1)), dict(bias=torch.zeros(264)), dict(bias=torch.zeros(263, dtype=bf)),
                dict(out=torch.zeros(5, 263, dtype=bf)), dict(out_dtype=torch.float16), dict(x=q, out_dtype=torch.int8),
                dict(x=torch.zeros(5, 272, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            Q.fp8_linear_fwd(**{**dict(w=w, x=x), **bad})
    for call in (lambda: Q.fp8_quantize(x), lambda: Q.fp8_dequantize(q), lambda: Q.fp8_linear_fwd(w, x), lambda: Q.fp8_linear_fwd(w, q)):
        with pytest.raises(ValueError, match="not the current CUDA device"):
            call()
