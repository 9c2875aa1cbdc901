"""int8_quantize at its longest rows: columns whose successor lies past 32-bit signed indexes."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 8])
def test_longest_rows(cuda_device, cols):
    """Off the vector width (scalar loops) and on it.  The last column holds the largest value, 254: the scale is 2,
    so a code is x / 2 to the nearest, ties to even, which torch gives exactly."""
    import torch
    from qlora_linear_layers_nf4_b200 import nf4qlora as Q
    x = torch.empty(cols, dtype=torch.bfloat16, device=cuda_device)
    step = 251 << 20
    ramp = ((torch.arange(step, device=cuda_device) % 251) - 125).to(torch.bfloat16)
    for at in range(0, cols, step):
        part = x[at:at + step]
        part.copy_(ramp[:part.numel()])
    x[-1] = 254.0
    m = Q.int8_quantize(x.view(1, cols))
    assert float(m.scale[0]) == 2.0
    for at in range(0, cols, step):
        want = (x[at:at + step].float() / 2).round().to(torch.int8)
        assert torch.equal(m.codes[0, at:at + step], want), at
