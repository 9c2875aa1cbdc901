"""The 8-bit floating point linear of few tokens with more weight rows than its CTAs take at once, which is what layers
of a full size have.  That each size takes this form is checked without a GPU, in test_plans.py.  Bounds as in
test_fp8_gpu.py."""
import pytest

from tests.test_fp8_gpu import Lin, _Q, _dt

pytestmark = pytest.mark.gpu

# m, n, k, dtype, bias, rounds of the CTAs over the rows
STREAMED = [
    (1, 4744, 144, "bf16", False, 2),
    (1, 11008, 2064, "f16", True, 3),
    (3, 9480, 272, "f32", True, 3),
    (8, 12000, 1040, "f16", False, 3),
    (7, 5000, 6160, "bf16", True, 2),
    (2, 20008, 2064, "bf16", True, 5),
]


@pytest.mark.parametrize("m,n,k,dtype,bias,rounds", STREAMED)
def test_rounds_of_weight_rows(cuda_device, m, n, k, dtype, bias, rounds):
    import torch
    Q = _Q()
    L = Lin(cuda_device, m, n, k, dtype, bias)
    big = torch.full((m + 5, n), 7.0, dtype=_dt(dtype), device=cuda_device)
    y = Q.fp8_linear_fwd(L.w, L.x, bias=L.bias, out=big[:m])
    L.check(y)
    assert (big[m:] == 7).all()
    given = Q.fp8_linear_fwd(L.w, Q.fp8_quantize(L.x), bias=L.bias, out_dtype=_dt(dtype))
    assert given.equal(y)
    for _ in range(3):
        assert Q.fp8_linear_fwd(L.w, L.x, bias=L.bias).equal(y)
    assert Q.read_status() == 0
