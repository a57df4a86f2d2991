"""The 8-bit norm at the ends of fp32: sums of squares that overflow, scales that are subnormal."""
import numpy as np
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


@pytest.mark.parametrize("k", [256, 1001, 40000])
@pytest.mark.parametrize("residual", [False, True])
def test_sum_of_squares_past_fp32(B, k, residual):
    # finite values whose squares leave fp32: the row reads as NaN, its neighbours are not touched
    x = torch.randn((3, k), generator=torch.Generator().manual_seed(k))
    x[1] *= 1e25
    x, w = x.bfloat16().cuda(), torch.ones(k, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(x) if residual else None
    y = torch.empty_like(x)
    codes, scales, h = B.rms_norm_int8(x, w, residual=r, y_out=y)
    s = scales.cpu().numpy()
    assert not np.isfinite(s[1]) and not codes[1].any()
    assert B.dequant_int8_to_bf16(codes, scales)[1].isnan().all() and y[1].isnan().all()
    if residual:
        assert torch.equal(h, x)
    assert np.isfinite(s[[0, 2]]).all() and codes[0].any() and codes[2].any()
    act, _ = B.rms_norm_q8_1(x, w, residual=r)
    kp = (k + 255) // 256 * 256
    raw = act.cpu().numpy()
    d = raw[3 * kp:].view(np.float32).reshape(3, kp // 32, 2)
    assert not np.isfinite(d[1, :k // 32]).any() and np.isfinite(d[[0, 2]]).all()
    assert not raw[: 3 * kp].reshape(3, kp)[1].any()


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
