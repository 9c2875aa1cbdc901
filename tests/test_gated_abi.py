"""CPU checks of the gated entry points: every refusal is made on the host, before the GPU is touched."""
import ctypes

import pytest

from qlora_linear_layers_nf4_b200 import nf4qlora as Q

FAKE = 0x10000   # aligned, never dereferenced: every call below fails validation first, or has nothing to do
BIG = 1 << 40


def _cw(rows=256, cols=256, bs=64, dq=1, codes=FAKE, absmax=FAKE):
    return Q.CWeight(codes=codes, absmax=absmax, absmax_q=FAKE, absmax_scale=FAKE, rows=rows, cols=cols,
                     block_size=bs, double_quant=dq)


def _fwd(gate=None, up=None, x=FAKE, m=16, a=FAKE, b=FAKE, r=16, alpha=32.0, act=0, dt=1, bias=None, h=FAKE, pre=None,
         t=None, ws=FAKE, wsb=BIG):
    gate, up = gate or _cw(), up or _cw()
    return Q.lib().qlora_gated_fwd(ctypes.byref(gate), ctypes.byref(up), x, m, a, b, r, alpha, act, dt, bias, h, pre, t,
                                   ws, wsb, None)


def _bwd(gate=None, up=None, x=FAKE, m=16, a=FAKE, b=FAKE, r=16, alpha=32.0, act=0, dt=1, dh=FAKE, pre=FAKE, t=None,
         da=FAKE, db=FAKE, dx=None, ws=FAKE, wsb=BIG):
    gate, up = gate or _cw(), up or _cw()
    return Q.lib().qlora_gated_bwd(ctypes.byref(gate), ctypes.byref(up), x, m, a, b, r, alpha, act, dt, dh, pre, t, da, db,
                                   dx, ws, wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_host_validation(call):
    for bad, status in ((dict(cols=200), 2), (dict(rows=252), 2), (dict(bs=32), 4), (dict(bs=96), 4), (dict(bs=0), 2),
                        (dict(codes=None), 1), (dict(dq=0, absmax=None), 1), (dict(codes=FAKE + 8), 3)):
        assert call(gate=_cw(**bad)) == status and call(up=_cw(**bad)) == status
    assert call(up=_cw(rows=264)) == 2 and call(up=_cw(cols=320)) == 2 and call(up=_cw(bs=128)) == 2
    assert call(up=_cw(dq=0)) == 1
    assert call(m=-1) == 2 and call(m=(1 << 30) + 1) == 2
    assert call(x=None) == 1 and call(a=None) == 1 and call(b=None) == 1
    assert call(x=FAKE + 8) == 3 and call(a=FAKE + 4) == 3 and call(b=FAKE + 2) == 3
    assert call(r=4) == 1 and call(r=12) == 1 and call(r=264) == 1
    assert call(alpha=float("nan")) == 1
    assert call(act=-1) == 1 and call(act=2) == 1
    assert call(dt=3) == 1 and call(dt=-1) == 1
    assert call(ws=None) == 5 and call(ws=FAKE + 8) == 5 and call(wsb=255) == 5
    assert call(t=FAKE + 2) == 3 and call(pre=FAKE + 2) == 3


def test_output_validation():
    assert _fwd(h=None) == 1 and _fwd(h=FAKE + 2) == 3 and _fwd(bias=FAKE + 2) == 3
    assert _fwd(m=0, x=None, h=None) == 0                  # nothing to do, nothing enqueued
    assert _fwd(m=0, x=None, h=None, act=7) == 1
    assert _bwd(dh=None) == 1 and _bwd(pre=None) == 1 and _bwd(da=None) == 1 and _bwd(db=None) == 1
    assert _bwd(dh=FAKE + 2) == 3 and _bwd(da=FAKE + 4) == 3 and _bwd(db=FAKE + 4) == 3 and _bwd(dx=FAKE + 4) == 3


def test_workspace_sizes():
    w = lambda op, m=100: Q.workspace_bytes(op, m, 264, 192, 16, 64, True)
    assert w(Q.OP_GATED_FWD) >= 256 + 2 * 100 * 16 * 2
    assert w(Q.OP_GATED_BWD) >= 256 + 2 * 100 * 264 * 2 + 4 * 2 * 100 * 16 * 2
    assert w(Q.OP_GATED_FWD_F32) >= 256 + 2 * 100 * 16 * 4
    assert w(Q.OP_GATED_BWD_F32) >= 256 + 2 * 100 * 264 * 4 + 2 * 2 * 100 * 16 * 4
    for op in (Q.OP_GATED_FWD, Q.OP_GATED_BWD, Q.OP_GATED_FWD_F32, Q.OP_GATED_BWD_F32):
        assert w(op, 0) >= 256
        need = w(op)
        call = _fwd if op in (Q.OP_GATED_FWD, Q.OP_GATED_FWD_F32) else _bwd
        dt = 0 if op in (Q.OP_GATED_FWD_F32, Q.OP_GATED_BWD_F32) else 2
        cw = dict(gate=_cw(264, 192), up=_cw(264, 192), m=100)
        assert call(dt=dt, wsb=need - 1, **cw) == 5


# ---- the binding's own checks, on tensors of the CPU: each is made before the library is called


def _layer(n=64, k=128, r=8, m=3, dtype=None):
    import torch
    dt = dtype or torch.bfloat16
    q = lambda: Q.QuantizedWeight(torch.zeros(n * k // 2, dtype=torch.uint8), torch.zeros(n * k // 64), None, None, n, k, 64, False)
    return dict(gate=q(), up=q(), x=torch.zeros(m, k, dtype=dt), A=torch.zeros(2, r, k, dtype=dt), B=torch.zeros(2, n, r, dtype=dt),
                alpha=16.0)


def test_binding_refusals():
    import torch
    from dataclasses import replace
    L = _layer()
    bf = torch.bfloat16
    saved = Q.GatedSaved(torch.zeros(2, 3, 64, dtype=bf), torch.zeros(2, 3, 8, dtype=bf))
    dh = torch.zeros(3, 64, dtype=bf)
    bad = [(dict(x=torch.zeros(128, dtype=bf)), ValueError), (dict(A=torch.zeros(8, 128, dtype=bf)), ValueError),
           (dict(A=torch.zeros(1, 8, 128, dtype=bf)), ValueError), (dict(B=torch.zeros(2, 64, 16, dtype=bf)), ValueError),
           (dict(B=torch.zeros(2, 64, 8)), TypeError), (dict(x=torch.zeros(3, 128, dtype=torch.int32)), TypeError),
           (dict(x=torch.zeros(3, 256, dtype=bf)[:, ::2]), ValueError),
           (dict(activation="relu"), ValueError), (dict(up=replace(L["up"], block_size=128)), ValueError),
           (dict(up=replace(L["up"], cols=64)), ValueError), (dict(up=replace(L["up"], double_quant=True)), ValueError)]
    for change, error in bad:
        with pytest.raises(error):
            Q.gated_fwd(**{**L, **change})
        with pytest.raises(error):
            Q.gated_bwd(**{**L, **change}, dh=dh, saved=saved)
    for name, t in (("bias", torch.zeros(64, dtype=bf)), ("out", torch.zeros(3, 65, dtype=bf)),
                    ("saved", Q.GatedSaved(torch.zeros(2, 3, 64), None)), ("saved", Q.GatedSaved(saved.pre, torch.zeros(2, 3, 9, dtype=bf)))):
        with pytest.raises((ValueError, TypeError)):
            Q.gated_fwd(**L, **{name: t})
    for change in (dict(dh=dh[:2]), dict(saved=Q.GatedSaved(None, saved.t)), dict(saved=Q.GatedSaved(saved.pre[:, :2], saved.t)),
                   dict(dA=torch.zeros(2, 8, 128, dtype=bf)), dict(dB=torch.zeros(2, 8, 64)), dict(dx=torch.zeros(3, 128))):
        with pytest.raises((ValueError, TypeError)):
            Q.gated_bwd(**L, **{**dict(dh=dh, saved=saved), **change})
    with pytest.raises(ValueError, match="not the current CUDA device"):
        Q.gated_fwd(**L)
    with pytest.raises(ValueError, match="not the current CUDA device"):
        Q.gated_bwd(**L, dh=dh, saved=saved)


@pytest.mark.parametrize("op", [Q.OP_GATED_FWD, Q.OP_GATED_BWD, Q.OP_GATED_FWD_F32, Q.OP_GATED_BWD_F32])
@pytest.mark.parametrize("n,k,r", [(8, 64, 8), (2000, 512, 64), (5000, 4096, 128), (64, 20480, 16)])
def test_a_workspace_serves_smaller_batches(op, n, k, r):
    rows = [0, 1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2560, 2561, 5000, 10240, 10241, 20000]
    sizes = [Q.workspace_bytes(op, m, n, k, r, 64, True) for m in rows]
    assert sizes == sorted(sizes)
