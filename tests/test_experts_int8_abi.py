"""CPU checks of the expert (grouped) and 8-bit entry points: every refusal is made on the host, before the GPU is
touched."""
import ctypes

import pytest

from qlora_linear_layers_nf4_b200 import nf4qlora as Q

FAKE = 0x10000   # aligned, never dereferenced: every call below fails validation first
BIG = 1 << 40


def _cw(rows=8 * 256, cols=256, bs=64, dq=1, codes=FAKE, absmax=FAKE):
    return Q.CWeight(codes=codes, absmax=absmax, absmax_q=FAKE, absmax_scale=FAKE, rows=rows, cols=cols,
                     block_size=bs, double_quant=dq)


def _fwd(cw=None, e=8, x=FAKE, m=16, off=FAKE, a=FAKE, b=FAKE, r=16, alpha=32.0, dt=1, bias=None, y=FAKE, t=None,
         ws=FAKE, wsb=BIG):
    cw = cw or _cw()
    return Q.lib().qlora_grouped_fwd(ctypes.byref(cw), e, x, m, off, a, b, r, alpha, dt, bias, y, t, ws, wsb, None)


def _bwd(cw=None, e=8, x=FAKE, m=16, off=FAKE, a=FAKE, b=FAKE, r=16, alpha=32.0, dt=1, dy=FAKE, t=None, da=FAKE,
         db=FAKE, dx=None, ws=FAKE, wsb=BIG):
    cw = cw or _cw()
    return Q.lib().qlora_grouped_bwd(ctypes.byref(cw), e, x, m, off, a, b, r, alpha, dt, dy, t, da, db, dx, ws, wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_grouped_host_validation(call):
    assert call(e=0) == 1 and call(e=513) == 1 and call(e=-1) == 1
    assert call(e=3) == 2                                  # rows do not divide
    assert call(cw=_cw(rows=8 * 252)) == 2                 # N % 8
    assert call(cw=_cw(cols=200)) == 2                     # K % 64
    assert call(cw=_cw(bs=32)) == 4 and call(cw=_cw(bs=96)) == 4 and call(cw=_cw(bs=0)) == 2
    assert call(cw=_cw(codes=None)) == 1 and call(cw=_cw(dq=0, absmax=None)) == 1
    assert call(m=-1) == 2 and call(m=(1 << 30) + 1) == 2
    assert call(off=None) == 1 and call(off=FAKE + 2) == 3
    assert call(x=None) == 1 and call(a=None) == 1 and call(b=None) == 1
    assert call(x=FAKE + 8) == 3 and call(a=FAKE + 4) == 3 and call(b=FAKE + 2) == 3
    assert call(r=4) == 1 and call(r=12) == 1 and call(r=264) == 1
    assert call(alpha=float("nan")) == 1
    assert call(dt=3) == 1 and call(dt=-1) == 1
    assert call(ws=None) == 5 and call(ws=FAKE + 8) == 5 and call(wsb=255) == 5
    assert call(t=FAKE + 2) == 3


def test_grouped_output_validation():
    assert _fwd(y=None) == 1 and _fwd(y=FAKE + 2) == 3 and _fwd(bias=FAKE + 2) == 3
    assert _fwd(m=0, x=None, y=None) == 0                  # nothing to do, nothing enqueued
    assert _fwd(m=0, x=None, y=None, off=None) == 1
    assert _bwd(dy=None) == 1 and _bwd(da=None) == 1 and _bwd(db=None) == 1
    assert _bwd(dy=FAKE + 2) == 3 and _bwd(da=FAKE + 4) == 3 and _bwd(db=FAKE + 4) == 3 and _bwd(dx=FAKE + 4) == 3


def test_int8_host_validation():
    q = lambda x=FAKE, dt=1, rows=4, cols=16, c=FAKE, s=FAKE: Q.lib().int8_quantize(x, dt, rows, cols, c, s, None)
    assert q(dt=3) == 1 and q(rows=-1) == 2 and q(cols=-1) == 2 and q(cols=1 << 31) == 2 and q(rows=1 << 31) == 2
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(x=FAKE + 2) == 3 and q(c=FAKE + 1) == 3 and q(s=FAKE + 2) == 3
    assert q(rows=0) == 0 and q(rows=0, x=None, c=None, s=None) == 0

    def lin(w=FAKE, s=FAKE, n=64, k=64, x=FAKE, xs=None, m=4, dt=1, bias=None, y=FAKE, ws=FAKE, wsb=BIG):
        return Q.lib().int8_linear_fwd(w, s, n, k, x, xs, m, dt, bias, y, ws, wsb, None)

    assert lin(w=None) == 1 and lin(s=None) == 1 and lin(x=None) == 1 and lin(y=None) == 1
    assert lin(dt=3) == 1
    assert lin(n=60) == 2 and lin(n=0) == 2 and lin(k=24) == 2 and lin(k=0) == 2 and lin(k=131088) == 2
    assert lin(m=0) == 2 and lin(m=(1 << 30) + 1) == 2
    assert lin(w=FAKE + 8) == 3 and lin(s=FAKE + 2) == 3 and lin(x=FAKE + 8) == 3 and lin(xs=FAKE + 1) == 3
    assert lin(y=FAKE + 8) == 3 and lin(bias=FAKE + 2) == 3
    assert lin(ws=None) == 5 and lin(ws=FAKE + 4) == 5 and lin(wsb=256) == 5


def test_workspace_sizes():
    w = Q.workspace_bytes
    assert w(Q.OP_GROUPED_FWD, 100, 256, 256, 16, 64, True) >= 256 + 100 * 16 * 2
    assert w(Q.OP_GROUPED_BWD, 100, 256, 256, 16, 64, True) >= 256 + 2 * 100 * 16 * 2
    assert w(Q.OP_GROUPED_FWD, 0, 256, 256, 16, 64, True) >= 256
    assert w(Q.OP_INT8_LINEAR, 33, 64, 48, 0, 0, False) >= 256 + 33 * 48 + 33 * 4


def _stack(e=4, n=64, k=128):
    import torch
    rows = e * n
    return Q.QuantizedWeight(codes=torch.zeros(rows * k // 2, dtype=torch.uint8), absmax=torch.zeros(rows * k // 64),
                             absmax_q=None, absmax_scale=None, rows=rows, cols=k, block_size=64, double_quant=False)


def test_grouped_binding_refuses():
    import torch
    bf = torch.bfloat16
    q = _stack()
    good = dict(x=torch.zeros(8, 128, dtype=bf), offsets=torch.zeros(5, dtype=torch.int32),
                A=torch.zeros(4, 16, 128, dtype=bf), B=torch.zeros(4, 64, 16, dtype=bf), alpha=32.0)
    dy = torch.zeros(8, 64, dtype=bf)
    for change in (dict(x=torch.zeros(8, 64, dtype=bf)), dict(x=torch.zeros(128, dtype=bf)),
                   dict(offsets=torch.zeros(4, dtype=torch.int32)), dict(A=torch.zeros(16, 128, dtype=bf)),
                   dict(A=torch.zeros(3, 16, 128, dtype=bf)), dict(A=torch.zeros(0, 16, 128, dtype=bf)),
                   dict(B=torch.zeros(4, 32, 16, dtype=bf)), dict(bias=torch.zeros(64, dtype=bf)),
                   dict(out=torch.zeros(8, 128, dtype=bf)), dict(t_out=torch.zeros(8, 8, dtype=bf)),
                   dict(x=torch.zeros(128, 8, dtype=bf).t())):
        with pytest.raises(ValueError):
            Q.grouped_fwd(q, **{**good, **change})
    for change in (dict(offsets=torch.zeros(5, dtype=torch.int64)), dict(x=torch.zeros(8, 128, dtype=torch.int32)),
                   dict(A=torch.zeros(4, 16, 128, dtype=torch.float16)), dict(bias=torch.zeros(4, 64))):
        with pytest.raises(TypeError):
            Q.grouped_fwd(q, **{**good, **change})
    with pytest.raises(ValueError):
        Q.grouped_bwd(q, dy=torch.zeros(8, 63, dtype=bf), **good)
    with pytest.raises(ValueError):
        Q.grouped_bwd(q, dy=dy, t=torch.zeros(8, 8, dtype=bf), **good)
    with pytest.raises(TypeError):
        Q.grouped_bwd(q, dy=dy, dA=torch.zeros(4, 16, 128, dtype=bf), **good)
    with pytest.raises(ValueError):
        Q.grouped_bwd(q, dy=dy, dB=torch.zeros(4, 16, 64), **good)


def test_int8_binding_refuses():
    import torch
    w = Q.Int8Matrix(torch.zeros(64, 32, dtype=torch.int8), torch.ones(64))
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        Q.int8_quantize(torch.zeros(4))
    with pytest.raises(TypeError):
        Q.int8_quantize(torch.zeros(4, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        Q.int8_quantize(torch.zeros(4, 8).t())
    with pytest.raises(ValueError):
        Q.int8_linear_fwd(w, x[:, :16].contiguous())
    with pytest.raises(ValueError):
        Q.int8_linear_fwd(w, x[0])
    with pytest.raises(TypeError):
        Q.int8_linear_fwd(w, x.to(torch.int32))
    with pytest.raises(TypeError):
        Q.int8_linear_fwd(w, x, out_dtype=torch.float32)
    with pytest.raises(TypeError):
        Q.int8_linear_fwd(w, x, bias=torch.zeros(64))
    with pytest.raises(ValueError):
        Q.int8_linear_fwd(Q.Int8Matrix(w.codes, torch.ones(63)), x)
    with pytest.raises(TypeError):
        Q.int8_linear_fwd(w, Q.Int8Matrix(x, torch.ones(4)))
    with pytest.raises(TypeError):
        Q.int8_linear_fwd(w, Q.Int8Matrix(x.to(torch.int8), torch.ones(4)), out_dtype=torch.float64)
