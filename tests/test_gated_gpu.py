"""GPU parity of the gated feed-forward layer, forward and backward, against its formulas in
64 bits on the same inputs.

Bounds per element, with e = half a step of the compute type (bf16 2^-8, f16 2^-11, fp32
2^-24), f = 2^-23 per fp32 operation (the tensor core may truncate), |.| products taken with
absolute values, p a projection, y the argument of the logistic function:
  T    e |T| + Et,  Et = s (K + 2) f |x||A|
  pre  e |pre| + Ep,  Ep = (e |T| + (1 + e) Et)|B| + (K + r + 3) f (|x||W'| + |T||B| + |bias|)
  q    eq = (8 + 4 |y|) f of itself: exp (2 + 1.2 |y| units of the last place), y's own three
       operations, a sum, a quotient of two units, and 2^-125 where the quotient underflows
  h    e |h| + 1.13 Eg (|u| + Eu) + |act(g)| Eu + (eq + 3 f) |act(g)||u|   (|act'| <= 1.13)
  d    Ed: dh u (|g y'| (dp + 6 f p) + dq + f |act'|) + 3 f |dg|,  dh g dq + 3 f |du|, where
       dq = eq q, dp = dq (1 - q) + q (dq + f)
  dB   (Ed + S |d|) |T| + (M + 8) f |d||T|       S what the terms of the compute type lose:
  U    Eu = s (Ed + S |d| + (N + 8) f |d|) |B|   2^-23 (bf16, three; fp32), 2^-21 (f16, two,
  dA   (Eu + S |U|)|x| + (M + 8) f |U||x|        plus 2^-36)
  dx   e |dx| + sum_p ((e |d| + (1 + e) Ed)|W'| + (e |U| + (1 + e) Eu)|A|
                       + (2 N + 2 r + 4) f (|d||W'| + |U||A|))
"""
import math

import numpy as np
import pytest

from oracle import nf4_oracle as O

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SPLIT = {"bf16": (2.0 ** -23, 0.0), "f16": (2.0 ** -21, 2.0 ** -36), "f32": (2.0 ** -23, 0.0)}
F = 2.0 ** -23
C2 = 2 * math.sqrt(2 / math.pi)


def _Q():
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    return Q


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def logistic_parts(g, act):
    """(y, q, y') in 64 bits."""
    import torch
    y = g if act == "silu" else C2 * (g + 0.044715 * g ** 3)
    slope = torch.ones_like(g) if act == "silu" else C2 * (1 + 0.134145 * g ** 2)
    return y, torch.sigmoid(y), slope


def within(name, got, want, bound, top=math.inf):
    """top: the least size that the type rounds to infinity.  What is that large by more than the bound has to be
    infinite, with its sign; what is so by less may be."""
    import torch
    got = got.double()
    assert got.shape == want.shape, name
    if math.isfinite(top):
        over, inf = want.abs() - top, got.isinf() & (got.sign() == want.sign())
        assert inf[over > bound].all(), f"{name} should be infinite"
        got = torch.where(inf & (over >= -bound), want, got)
    assert torch.isfinite(got).all(), f"{name} is not finite"
    off = (got - want).abs() - bound
    worst = off.argmax().item() if off.numel() else 0
    assert off.numel() == 0 or off.max() <= 0, (
        f"{name}: off by {(got - want).abs().flatten()[worst]:.3e}, bound {bound.expand_as(want).flatten()[worst]:.3e}")


class Layer:
    """Two projections and a batch, on the GPU, and the same in 64 bits."""

    def __init__(self, dev, m, n, k, r, dtype="bf16", block=64, dq=True, bias=False, act="silu", seed=0):
        import torch
        Q = _Q()
        self.m, self.n, self.k, self.r, self.dtype, self.act = m, n, k, r, dtype, act
        rng = np.random.default_rng(seed + 7 * n + k + 13 * m)
        dt = _dt(dtype)
        self.q, self.W = [], []
        for _ in range(2):
            w = (rng.standard_normal((n, k)) * 0.04).astype(np.float32)
            self.q.append(Q.quantize(torch.from_numpy(w).to(dev), block, dq))
            ref = O.dequantize(O.quantize(w, block, double=dq), "f32")
            self.W.append(torch.from_numpy(np.ascontiguousarray(ref)).reshape(n, k).to(dev).to(dt).double())
        t = lambda *shape, sigma=1.0: torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(dt).to(dev)
        self.x, self.A, self.B = t(m, k), t(2, r, k, sigma=k ** -0.5), t(2, n, r, sigma=0.05)
        self.dh, self.bias = t(m, n), t(2, n) if bias else None
        self.alpha, self.s = 2.0 * r, 2.0

    def fwd(self, **kw):
        return _Q().gated_fwd(self.q[0], self.q[1], self.x, self.A, self.B, self.alpha, activation=self.act, bias=self.bias, **kw)

    def bwd(self, saved, **kw):
        return _Q().gated_bwd(self.q[0], self.q[1], self.x, self.A, self.B, self.alpha, self.dh, saved, activation=self.act, **kw)

    def check_fwd(self, h, saved, rows=slice(None)):
        e = HALF[self.dtype]
        x, A, B = self.x[rows].double(), self.A.double(), self.B.double()
        pre, err = [], []
        for p in range(2):
            tw = self.s * (x @ A[p].T)
            t_err = self.s * (self.k + 2) * F * (x.abs() @ A[p].abs().T)
            b = 0.0 if self.bias is None else self.bias[p].double()
            want = x @ self.W[p].T + tw @ B[p].T + b
            ab = 0.0 if self.bias is None else b.abs()
            bound = ((e * tw.abs() + (1 + e) * t_err) @ B[p].abs().T +
                     (self.k + self.r + 3) * F * (x.abs() @ self.W[p].abs().T + (1 + e) * tw.abs() @ B[p].abs().T + ab))
            if saved is not None:
                if saved.t is not None:
                    within("T", saved.t[p][rows], tw, e * tw.abs() + (1 + e) * t_err)
                within("pre", saved.pre[p][rows], want, e * want.abs() + (1 + e) * bound)
            pre.append(want)
            err.append(bound)
        g, u = pre
        y, q, _ = logistic_parts(g, self.act)
        a = g * q
        eq = (8 + 4 * y.abs().clamp(max=90)) * F
        bound = 1.13 * err[0] * (u.abs() + err[1]) + a.abs() * err[1] + (eq + 3 * F) * a.abs() * u.abs() + 2.0 ** -125 * (g * u).abs()
        f16 = self.dtype == "f16"   # which rounds to infinity from 65520 on, half a step above its largest, 65504
        within("h", h[rows], a * u, e * (a * u).abs() + (1 + e) * bound + (2.0 ** -25 if f16 else 0.0), 65520.0 if f16 else math.inf)

    def check_bwd(self, dA, dB, dx, saved, rows=slice(None)):
        e = HALF[self.dtype]
        S, S0 = SPLIT[self.dtype]
        x, dh, A, B = self.x[rows].double(), self.dh[rows].double(), self.A.double(), self.B.double()
        g, u, t = saved.pre[0][rows].double(), saved.pre[1][rows].double(), saved.t[:, rows].double()
        m = x.shape[0]
        y, q, slope = logistic_parts(g, self.act)
        p = q * (1 - q)
        dact = q + g * p * slope
        d = [dh * u * dact, dh * g * q]
        e_q = (8 + 4 * y.abs().clamp(max=90)) * F * q + 2.0 ** -125
        e_p = e_q * (1 - q) + q * (e_q + F)
        e_act = (g * slope).abs() * (e_p + 6 * F * p) + e_q + F * dact.abs()
        e_d = [(dh * u).abs() * e_act + 3 * F * d[0].abs(), (dh * g).abs() * e_q + 3 * F * d[1].abs()]
        want_dx, bound_dx = 0.0, 0.0
        for i in range(2):
            ad, U = d[i].abs(), self.s * (d[i] @ B[i])
            lost = e_d[i] + S * ad + S0
            within("dB", dB[i], d[i].T @ t[i], lost.T @ t[i].abs() + (m + 8) * F * (ad.T @ t[i].abs()) + 1e-30)
            e_u = self.s * ((lost + (self.n + 8) * F * ad) @ B[i].abs())
            aU = U.abs()
            within("dA", dA[i], U.T @ x, (e_u + S * aU + S0).T @ x.abs() + (m + 8) * F * (aU.T @ x.abs()) + 1e-30)
            want_dx = want_dx + d[i] @ self.W[i] + U @ A[i]
            tiny = 2.0 ** -25 if self.dtype == "f16" else 0.0   # half a step of f16's smallest values
            bound_dx = bound_dx + ((e * ad + (1 + e) * e_d[i] + tiny) @ self.W[i].abs() + (e * aU + (1 + e) * e_u + tiny) @ A[i].abs() +
                                   (2 * self.n + 2 * self.r + 4) * F * (ad @ self.W[i].abs() + aU @ A[i].abs()))
        if dx is not None:
            within("dx", dx[rows], want_dx, e * want_dx.abs() + (1 + e) * bound_dx + (2.0 ** -25 if self.dtype == "f16" else 0.0))


def ok_status():
    assert _Q().read_status() == 0


FWD = [  # m, n, k, r, dtype, block, dq, bias, act
    (1, 136, 128, 8, "bf16", 64, True, False, "silu"),
    (2, 8, 64, 16, "f16", 64, False, True, "gelu_tanh"),
    (5, 264, 1088, 24, "f16", 128, True, True, "silu"),
    (8, 1032, 192, 256, "bf16", 64, False, False, "gelu_tanh"),
    (9, 520, 4096, 64, "bf16", 64, True, False, "silu"),
    (16, 2056, 1024, 72, "bf16", 256, True, True, "silu"),
    (17, 128, 512, 136, "f16", 64, True, False, "silu"),
    (32, 256, 2048, 16, "bf16", 64, True, False, "gelu_tanh"),
    (33, 256, 256, 64, "bf16", 64, True, False, "silu"),
    (65, 120, 320, 40, "f16", 4096, False, False, "silu"),
    (255, 264, 128, 8, "bf16", 64, True, True, "silu"),
    (256, 72, 64, 128, "f16", 64, True, False, "gelu_tanh"),
    (257, 1000, 192, 24, "bf16", 64, False, False, "silu"),
    (300, 5000, 128, 64, "bf16", 64, True, False, "silu"),     # two MMAs a tile
    (513, 6008, 64, 200, "f16", 64, True, True, "gelu_tanh"),
    (1500, 3080, 320, 16, "bf16", 128, True, False, "silu"),
    (2, 64, 64, 8, "f32", 64, True, True, "silu"),
    (130, 200, 192, 24, "f32", 64, False, False, "gelu_tanh"),
]


@pytest.mark.parametrize("m,n,k,r,dtype,block,dq,bias,act", FWD)
def test_forward(cuda_device, m, n, k, r, dtype, block, dq, bias, act):
    L = Layer(cuda_device, m, n, k, r, dtype, block, dq, bias, act)
    h, saved = L.fwd()
    L.check_fwd(h, saved)
    only, none = L.fwd(want_saved=False)
    assert none is None
    L.check_fwd(only, None)
    ok_status()


BWD = [
    (1, 136, 128, 8, "bf16", 64, True, "silu"),
    (2, 8, 64, 16, "f16", 64, False, "gelu_tanh"),
    (16, 1032, 192, 256, "bf16", 64, False, "gelu_tanh"),
    (17, 128, 512, 136, "f16", 64, True, "silu"),
    (63, 264, 1088, 24, "f16", 128, True, "silu"),
    (65, 120, 320, 40, "bf16", 4096, False, "gelu_tanh"),
    (129, 72, 64, 128, "bf16", 64, True, "silu"),
    (257, 1000, 192, 24, "f16", 64, False, "gelu_tanh"),
    (300, 200, 5056, 64, "bf16", 64, True, "silu"),            # two MMAs a tile
    (1500, 3080, 320, 16, "bf16", 128, True, "silu"),
    (700, 520, 4096, 72, "f16", 64, True, "silu"),
    (2, 64, 64, 8, "f32", 64, True, "silu"),
    (130, 200, 192, 24, "f32", 64, False, "gelu_tanh"),
]


@pytest.mark.parametrize("m,n,k,r,dtype,block,dq,act", BWD)
def test_backward(cuda_device, m, n, k, r, dtype, block, dq, act):
    Q = _Q()
    L = Layer(cuda_device, m, n, k, r, dtype, block, dq, False, act)
    _, saved = L.fwd()
    dA, dB, dx = L.bwd(saved)
    L.check_bwd(dA, dB, dx, saved)
    dA2, dB2, none = L.bwd(Q.GatedSaved(saved.pre, None), want_dx=False)   # T again: the same kernel
    assert none is None and dA2.equal(dA) and dB2.equal(dB)
    ok_status()
