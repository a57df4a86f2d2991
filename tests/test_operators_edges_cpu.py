"""Argument checks, without a GPU, that keep a kernel from a misaligned or a racing access: none of these calls
launches a kernel."""
import ctypes

import pytest

P = ctypes.c_void_p
X = 0x1000000


@pytest.fixture(scope="module")
def L():
    from bit_quantized_linear_q8_gb300 import build, _abi
    build.build()
    return _abi.lib()


def refused(L, status, text):
    from bit_quantized_linear_q8_gb300 import _abi
    assert status == _abi.BQ_ERR_INVALID, status
    assert text in L.bq_last_error(), L.bq_last_error()


def delta(L, which, g=(X * 6, 4, 1), beta=(X * 7, 4, 1), idx=0, cu=X * 9):
    from bit_quantized_linear_q8_gb300 import _abi
    d = [_abi.HeadsDesc(*h) for h in ((X * 2, 256, 128), (X * 3, 256, 128), (X * 4, 512, 128), g, beta)]
    args = [ctypes.byref(x) for x in d]
    if which == "decode":
        return L.gated_delta_decode(*args, P(X * 16), P(idx), P(X * 64), 2, 2, 2, 4, 128, 2, 1.0, 0, P(0))
    # (scratch NULL: the last check, so that no call gets as far as a launch)
    return L.gated_delta_prefill(*args, P(X * 16), P(cu), P(idx), P(X * 64), P(0), 2, 4, 2, 4, 128, 2, 1.0, 0, P(0))


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_gates_and_indices(L, which):
    refused(L, delta(L, which, g=(X * 6 + 2, 4, 1)), b"g must be non-NULL and 4-byte aligned")
    refused(L, delta(L, which, beta=(X * 7 + 1, 4, 1)), b"beta must be non-NULL and 4-byte aligned")
    refused(L, delta(L, which, g=(0, 4, 1)), b"g must be")
    refused(L, delta(L, which, g=(X * 6, -4, 1)), b"strides of g")
    refused(L, delta(L, which, beta=(X * 7, 4, -1)), b"strides of beta")
    refused(L, delta(L, which, idx=X + 2), b"state_idx")


def test_prefill_bounds_pointer(L):
    refused(L, delta(L, "prefill", cu=X + 1), b"cu_seqlens")
    refused(L, delta(L, "prefill"), b"scratch")


def test_norm_overlaps(L):
    # 4 x 64: x, residual, y and residual_out 512 bytes, weight 128, codes 256 (q8_1: 1024 and 256), scales 16
    def norm(x=X, residual=2 * X, weight=3 * X, h=4 * X, y=5 * X, codes=6 * X, scales=7 * X, eps=-1.0):
        return L.rms_norm_int8(P(x), P(residual), P(weight), eps, P(h), P(y), P(codes), P(scales), 4, 64, P(0))

    for kw in (dict(codes=X + 496), dict(codes=2 * X + 16), dict(codes=3 * X + 112), dict(scales=X), dict(scales=3 * X + 112),
               dict(codes=5 * X), dict(codes=4 * X + 256), dict(scales=6 * X + 240), dict(h=3 * X), dict(y=3 * X + 16),
               dict(codes=X - 240), dict(h=X + 16), dict(h=5 * X)):
        refused(L, norm(**kw), b"overlap")
    # neighbours that only touch are no overlap: the call goes on to the next check
    for kw in (dict(codes=X + 512), dict(codes=X - 256), dict(h=X), dict(h=2 * X), dict(scales=6 * X + 256)):
        refused(L, norm(**kw), b"eps")
    q8 = lambda act: L.rms_norm_q8_1(P(X), P(0), P(3 * X), 1e-6, P(0), P(0), P(act), 4, 64, P(0))  # noqa: E731
    refused(L, q8(X + 16), b"overlap")
    refused(L, q8(X - 1024 - 16), b"overlap")  # the scales behind the codes
    refused(L, L.quantize_int8(P(X), P(X), P(7 * X), 4, 64, P(0)), b"overlap")
    refused(L, L.quantize_int8(P(X), P(6 * X), P(6 * X), 4, 64, P(0)), b"overlap")
    refused(L, L.dequant_int8_to_bf16(P(X), P(3 * X), P(X - 16), 4, 64, P(0)), b"overlap")
    refused(L, L.dequant_int8_to_bf16(P(X), P(3 * X), P(3 * X - 16), 4, 64, P(0)), b"overlap")
