"""The gated delta rule at the ends of its range: queries that are stored keys."""
import numpy as np
import pytest
import torch

from helpers import bf16_half_ulp

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    import bit_quantized_linear_q8_gb300 as B
    return B


def test_queries_that_are_stored_keys(B):
    # S = k v^T and q = k: all 128 terms of S^T q have one sign, so a rounding that leans one way does not
    # cancel.  The prefill takes S^T q from one FP16 term of S, rounded to nearest: each term is off by at most
    # 2^-11, and their mean by far less.  400 000 outputs: the BF16 store's own errors average to 2^-18.
    tokens, heads = 64, 48
    g = torch.Generator("cpu").manual_seed(5)
    k = torch.randn((heads, D), generator=g)
    k = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    v = torch.randn((heads, D), generator=g)
    state = (k.float()[:, :, None] * v[:, None, :])[None].cuda()
    # every token asks for a multiple of the key, so that the mantissas of all of them differ
    m = 1 + torch.rand((tokens, 1, 1), generator=g)
    q = (m * k.float()).bfloat16().cuda()
    zeros = torch.zeros((tokens, heads), device="cuda")
    ref = torch.einsum("hkv,thk->thv", state[0].double(), q.double()).cpu().numpy()
    for what in ("prefill", "decode"):
        s = state.clone()
        if what == "prefill":
            out = B.gated_delta_prefill(q, q, torch.zeros_like(q), zeros, zeros, s, scale=1.0)
        else:
            out = B.gated_delta_decode(q, q, torch.zeros_like(q), zeros, zeros, s, tokens=tokens, scale=1.0)
        assert torch.equal(s, state), what
        err = out.cpu().double().numpy() - ref
        assert np.all(np.abs(err) <= bf16_half_ulp(ref) * (1 + 2.0 ** -7) + 2.0 ** -11 * np.abs(ref)), what
        mean = (err * np.sign(ref)).sum() / np.abs(ref).sum()
        assert abs(mean) <= 2.0 ** -14, (what, np.log2(abs(mean)))
