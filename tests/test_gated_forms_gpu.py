"""The gated layer in the forms that full-size layers take and small ones do not: the work splits of the streaming
forward.  That each size takes its form is
checked without a GPU, in test_plans.py.  Bounds as in test_gated_gpu.py."""
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
