"""CPU checks that the gated and 8-bit floating point entry points refuse outputs which overlap an input or each other:
their kernels run beside each other and read inputs more than once, so such a call would give wrong results.  The
addresses are never dereferenced; every call here is refused on the host."""
import ctypes
import itertools

import pytest

from qlora_linear_layers_nf4_b200 import nf4qlora as Q

M, N, K, R = 48, 256, 192, 16


class Memory:
    """Made-up memory, apart from each other."""

    def __init__(self):
        self.at = 1 << 36

    def take(self, nbytes):
        here = self.at
        self.at += (nbytes + 4095) // 4096 * 4096 + 4096
        return here


def gated(backward, f32, dq):
    """(place, call, inputs, outputs) of a gated call."""
    mem, e = Memory(), 4 if f32 else 2
    op = (Q.OP_GATED_BWD_F32 if f32 else Q.OP_GATED_BWD) if backward else (Q.OP_GATED_FWD_F32 if f32 else Q.OP_GATED_FWD)
    need = Q.workspace_bytes(op, M, N, K, R, 64, dq)
    sizes = dict(gate=N * K // 2, up=N * K // 2, gate_scale=N * K // 64 * (1 if dq else 4), up_scale=N * K // 64 * (1 if dq else 4),
                 x=M * K * e, A=2 * R * K * e, B=2 * N * R * e)
    ins = list(sizes)
    if backward:
        sizes.update(dh=M * N * e, pre=2 * M * N * e, t=2 * M * R * e, dA=2 * R * K * 4, dB=2 * N * R * 4, dx=M * K * e)
        outs = ["dA", "dB", "dx"]
        ins += ["dh", "pre", "t"]
    else:
        sizes.update(bias=2 * N * e, h=M * N * e, pre=2 * M * N * e, t=2 * M * R * e)
        outs = ["h", "pre", "t"]
        ins += ["bias"]
    sizes["ws"] = need
    place = {name: mem.take(n) for name, n in sizes.items()}

    def call(p):
        w = [Q.CWeight(codes=p[i], absmax=None if dq else p[i + "_scale"], absmax_q=p[i + "_scale"] if dq else None,
                       absmax_scale=1 << 16, rows=N, cols=K, block_size=64, double_quant=int(dq)) for i in ("gate", "up")]
        first = (ctypes.byref(w[0]), ctypes.byref(w[1]), p["x"], M, p["A"], p["B"], R, 32.0, 0, 0 if f32 else 1)
        if backward:
            return Q.lib().qlora_gated_bwd(*first, p["dh"], p["pre"], p["t"], p["dA"], p["dB"], p["dx"], p["ws"], need, None)
        return Q.lib().qlora_gated_fwd(*first, p["bias"], p["h"], p["pre"], p["t"], p["ws"], need, None)

    return place, sizes, call, ins, outs + ["ws"]


def fp8(which, f32, block_rows):
    mem, e = Memory(), 4 if f32 else 2
    dt = 0 if f32 else 1
    scale = -(-M // block_rows) * -(-K // 128) * 4
    if which == "linear":
        need = Q.workspace_bytes(Q.OP_FP8_LINEAR, M, N, K, 0, 0, False)
        sizes = dict(w=N * K, w_scale=N // 128 * -(-K // 128) * 4, x=M * K * (1 if block_rows == 1 else e), bias=N * e, y=M * N * e, ws=need)
        ins, outs = ["w", "w_scale", "x", "bias"], ["y", "ws"]
        if block_rows == 1:
            sizes["x_scale"] = scale
            ins.append("x_scale")
        call = lambda p: Q.lib().fp8_linear_fwd(p["w"], p["w_scale"], N, K, p["x"], p.get("x_scale"), M, dt, p["bias"], p["y"], p["ws"], need, None)
    else:
        sizes = dict(x=M * K * e, codes=M * K, scale=scale)
        back = which == "dequantize"
        ins, outs = (["codes", "scale"], ["x"]) if back else (["x"], ["codes", "scale"])
        if back:
            call = lambda p: Q.lib().fp8_dequantize(p["codes"], p["scale"], M, K, block_rows, dt, p["x"], None)
        else:
            call = lambda p: Q.lib().fp8_quantize(p["x"], dt, M, K, block_rows, p["codes"], p["scale"], None)
    return {name: mem.take(n) for name, n in sizes.items()}, sizes, call, ins, outs


CALLS = [lambda b=b, f=f, d=d: gated(b, f, d) for b, f, d in itertools.product((False, True), (False, True), (False, True))]
CALLS += [lambda w=w, f=f, r=r: fp8(w, f, r) for w, f, r in itertools.product(("quantize", "dequantize", "linear"), (False, True), (1, 128))]


@pytest.mark.parametrize("make", CALLS)
def test_overlaps_are_refused(make):
    import torch
    place, sizes, call, ins, outs = make()
    if not torch.cuda.is_available():     # made-up memory: only where nothing can be launched
        assert call(place) == 6           # NF4_ERR_CUDA: past every check
    pairs = [(o, i) for o in outs for i in ins] + list(itertools.combinations(outs, 2))
    for out, other in pairs:
        # at the same place; with the first bytes on the other's last ones; with the last on its first
        for at in (place[other], place[other] + (sizes[other] - 1) // 16 * 16, place[other] - (sizes[out] - 1) // 16 * 16):
            assert call({**place, out: at}) == 1, (out, other)
