"""Lengths at which 32-bit counts would wrap: one sequence of 2^27 tokens, rows of almost 2^32 codes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    import bit_quantized_linear_q8_gb300 as B
    return B


@pytest.fixture(autouse=True)
def free_after():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def all_equal(t, value, step=1 << 30):
    flat = t.view(-1)
    return all(bool((flat[i:i + step] == value).all()) for i in range(0, flat.numel(), step))


@pytest.mark.parametrize("tokens", [2 ** 27 - 8, 2 ** 27 + 100])
def test_skipped_sequence_of_many_tokens(B, tokens):
    # a sequence without a state: zeros in all of its rows, none in the rows behind it (34 GB of outputs; the
    # rows of q, k and v overlap, as nothing reads them)
    total = tokens + 3
    q, k, v = (torch.ones(8 * total + D, dtype=torch.bfloat16, device="cuda").as_strided((total, 1, D), (8, D, 1))
               for _ in range(3))
    g, beta = (torch.zeros((total, 1), device="cuda") for _ in range(2))
    out = torch.full((total, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    state = torch.ones((1, 1, D, D), device="cuda")
    B.gated_delta_prefill(q, k, v, g, beta, state, cu_seqlens=torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                          state_idx=torch.tensor([-1], dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert B.lib().bq_device_status() == 0
    assert all_equal(out[:tokens], 0.0) and (out[tokens:] == 7).all() and (state == 1).all()


def test_dequant_int8_rows_of_almost_2_32(B):
    k = 2 ** 32 - 8
    codes = torch.ones((2, k), dtype=torch.int8, device="cuda")
    out = B.dequant_int8_to_bf16(codes, torch.tensor([0.5, 2.0], device="cuda"))
    assert all_equal(out[0], 0.5) and all_equal(out[1], 2.0)
