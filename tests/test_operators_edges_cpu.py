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
