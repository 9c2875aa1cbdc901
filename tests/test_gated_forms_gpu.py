"""The gated layer in the forms that full-size layers take and small ones do not: the work splits of the streaming
forward, few tokens by the GEMM, tiles of two MMAs, several rounds of split tiles, long sums over tokens.  That each
size takes its form is checked without a GPU, in test_plans.py.  Bounds as in test_gated_gpu.py."""
import pytest

from tests.test_gated_gpu import Layer, ok_status

pytestmark = pytest.mark.gpu

# m, n, k, r, dtype, act, and what the split has to be like: whole tiles a CTA; of the others none, CTAs of their own, or
# shares that straddle tiles
DECODE = [
    (1, 11008, 1088, 16, "bf16", "silu", 1, "own"),          # the shares are one unit, an odd number
    (2, 9600, 1600, 72, "f16", "gelu_tanh", 1, "own"),
    (20, 5000, 1088, 24, "bf16", "silu", 1, "own"),          # two groups of tokens
    (20, 5000, 1088, 24, "f16", "gelu_tanh", 1, "own"),
    (3, 20008, 320, 8, "bf16", "gelu_tanh", 2, "own"),
    (11, 20008, 320, 40, "f16", "silu", 2, "own"),
    (5, 9472, 256, 8, "bf16", "silu", 1, "none"),
    (16, 6400, 1088, 64, "bf16", "silu", 0, "straddle"),
    (8, 6400, 2048, 16, "f16", "silu", 0, "straddle"),
    (1, 5000, 64, 16, "bf16", "gelu_tanh", 0, "straddle"),   # one unit a tile: a share is whole tiles after all
    (12, 14584, 576, 40, "bf16", "silu", 1, "straddle"),
    (4, 14584, 1344, 128, "f16", "gelu_tanh", 1, "straddle"),
    (13, 24008, 448, 8, "bf16", "silu", 2, "straddle"),
]


@pytest.mark.parametrize("m,n,k,r,dtype,act,whole,rest", DECODE)
def test_work_splits_of_few_tokens(cuda_device, m, n, k, r, dtype, act, whole, rest):
    L = Layer(cuda_device, m, n, k, r, dtype, bias=True, act=act)
    h, saved = L.fwd()
    L.check_fwd(h, saved)
    for _ in range(5):                       # joins happen in whatever order; the bits are the same
        again, s = L.fwd()
        assert again.equal(h) and s.pre.equal(saved.pre) and s.t.equal(saved.t)
    assert L.fwd(want_saved=False)[0].equal(h)
    ok_status()


# m, n, k, r, dtype: few tokens that the GEMM takes, as shares of the streaming kernel would straddle tiles
FEW_BY_GEMM = [(17, 4096, 512, 16, "bf16"), (32, 4096, 512, 72, "f16"), (24, 2560, 2560, 24, "bf16"), (31, 8200, 1024, 8, "f16")]


@pytest.mark.parametrize("m,n,k,r,dtype", FEW_BY_GEMM)
def test_few_tokens_by_the_gemm(cuda_device, m, n, k, r, dtype):
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    import torch
    L = Layer(cuda_device, m, n, k, r, dtype, bias=True)
    big = torch.full((m + 3, n), 7.0, dtype=L.x.dtype, device=cuda_device)
    h, saved = L.fwd(out=big[:m])
    L.check_fwd(h, saved)
    assert (big[m:] == 7).all() and L.fwd(want_saved=False)[0].equal(h)
    grads = L.bwd(saved)
    L.check_bwd(*grads, saved)
    assert all(a.equal(b) for a, b in zip(grads, L.bwd(Q.GatedSaved(saved.pre, None))))   # T again: the same bits
    ok_status()


# m, n, k, r, dtype, block, dq, act: forwards of two MMAs a weight tile
TWO_MMAS_FWD = [
    (300, 9600, 128, 64, "bf16", 64, True, "silu"),
    (300, 9480, 192, 24, "f16", 128, False, "gelu_tanh"),      # a short last tile of outputs
    (520, 6008, 320, 72, "f16", 64, True, "silu"),             # the last token tile has one part
]


@pytest.mark.parametrize("m,n,k,r,dtype,block,dq,act", TWO_MMAS_FWD)
def test_forward_of_two_mmas_a_tile(cuda_device, m, n, k, r, dtype, block, dq, act):
    L = Layer(cuda_device, m, n, k, r, dtype, block, dq, True, act)
    h, saved = L.fwd()
    L.check_fwd(h, saved)
    assert L.fwd(want_saved=False)[0].equal(h)
    ok_status()


# the same of dx: training batches
TWO_MMAS_DX = [
    (1500, 200, 4096, 24, "bf16", 64, True, "silu"),
    (1500, 200, 4032, 24, "f16", 64, False, "gelu_tanh"),      # a short last tile of columns
    (520, 72, 9728, 16, "bf16", 128, False, "gelu_tanh"),      # the last token tile has one part
    (520, 136, 9728, 8, "f16", 64, True, "silu"),
    (800, 1096, 6400, 72, "bf16", 64, True, "gelu_tanh"),      # more steps than stages and code slots, several rounds
    (1300, 520, 4160, 200, "f16", 256, True, "silu"),
]


@pytest.mark.parametrize("m,n,k,r,dtype,block,dq,act", TWO_MMAS_DX)
def test_backward_of_two_mmas_a_tile(cuda_device, m, n, k, r, dtype, block, dq, act):
    L = Layer(cuda_device, m, n, k, r, dtype, block, dq, False, act)
    _, saved = L.fwd()
    dA, dB, dx = L.bwd(saved)
    L.check_bwd(dA, dB, dx, saved)
    for _ in range(3):
        assert all(a.equal(b) for a, b in zip((dA, dB, dx), L.bwd(saved)))
    ok_status()


# m, n, k, r, dtype: forwards whose splits are more tiles than the CTA pairs take at once
ROUNDS_OF_SPLITS = [(33, 9608, 2560, 16, "bf16"), (64, 9608, 2560, 24, "f16"), (40, 10400, 3008, 72, "bf16")]


@pytest.mark.parametrize("m,n,k,r,dtype", ROUNDS_OF_SPLITS)
def test_rounds_of_split_tiles(cuda_device, m, n, k, r, dtype):
    L = Layer(cuda_device, m, n, k, r, dtype, bias=True)
    h, saved = L.fwd()
    L.check_fwd(h, saved)
    for _ in range(3):
        again, s = L.fwd()
        assert again.equal(h) and s.pre.equal(saved.pre)
    ok_status()


# m, n, k, r: long sums over tokens with enough tiles that a CTA has about seventy of their steps of 64: of U (over n)
# and dB, and of dA
LONG_SUMS = [(9000, 8200, 128, 16), (9000, 136, 8256, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k,r", LONG_SUMS)
def test_sums_brought_to_fp32_in_time(cuda_device, m, n, k, r, dtype):
    """dA and dB of many tokens, every row nonzero, relative to 64 bits in norm.  The tensor core loses up to 2^-25 of an
    accumulator at an instruction (towards zero, so the losses add up), and no more than 16 go into one before it is added
    to an fp32 total: 16 * 2^-25 of a sum; dA has that of U and of its own.  The activation's fp32 values and the terms'
    24 (22) bits are within 2^-22.  Seventy steps are 140 instructions into each accumulator: left there they would lose
    about 140 * 2^-26 * 2 / 3 = 1.4e-6 in each sum."""
    L = Layer(cuda_device, m, n, k, r, dtype)
    _, saved = L.fwd()
    dA, dB, dx = L.bwd(saved)
    d = [v.double() for v in (L.dh, saved.pre[0], saved.pre[1])]
    sig = d[1].sigmoid()
    d = (d[0] * d[2] * (sig + d[1] * sig * (1 - sig)), d[0] * d[1] * sig)
    window = 16 * 2.0 ** -25
    for i in range(2):
        want = d[i].T @ saved.t[i].double()
        off = (dB[i].double() - want).norm() / want.norm()
        assert off <= window + 2.0 ** -22, f"dB: {off:.2e}"
        want = (L.s * (d[i] @ L.B[i].double())).T @ L.x.double()
        off = (dA[i].double() - want).norm() / want.norm()
        assert off <= 2 * window + 2.0 ** -22, f"dA: {off:.2e}"
    ok_status()
