"""The 8-bit norm at the ends of fp32: scales that are subnormal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    import bit_quantized_linear_q8_gb300 as B
    return B


@pytest.mark.parametrize("k", [256, 1001])
@pytest.mark.parametrize("units", [128, 150, 180, 190])
def test_codes_of_subnormal_scales_saturate(B, k, units):
    # y = `units` times 2^-149: the scale rounds to one unit, and the codes stop at 127
    big = 1000.0
    w = torch.full((k,), 2.0 ** -133, dtype=torch.bfloat16)
    w[0] = 0
    x = torch.full((1, k), units * 2.0 ** -16 * big / k ** 0.5).bfloat16()
    x[0, ::2] *= -1
    x[0, 0] = big
    x, w = x.cuda(), w.cuda()
    sign = torch.ones(k, dtype=torch.int8)
    sign[::2] = -1
    codes, scales, _ = B.rms_norm_int8(x, w)
    assert 2.0 ** -149 <= scales.item() <= 2.0 ** -148
    c = codes.cpu()[0, 1:]
    assert (c * sign[1:] > 60).all(), c
    act, _ = B.rms_norm_q8_1(x, w)
    c = act.cpu()[1:k].view(torch.int8)
    assert (c * sign[1:] > 60).all(), c
