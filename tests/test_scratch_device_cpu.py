"""A caller's scratch has to lie on the GPU of the call's tensors; without a GPU, on stand-ins that answer what
the binding asks (none of these calls reaches the library's launch)."""
import pytest
import torch

CUDA0, CUDA1 = torch.device("cuda:0"), torch.device("cuda:1")


class Fake(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    is_cuda = True
    device = CUDA0

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        return super().__torch_function__(func, types, args, kwargs or {})


def fake(dtype, *shape, device=CUDA0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Fake)
    t.device = device
    return t


@pytest.fixture(scope="module")
def B():
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    import bit_quantized_linear_q8_gb300 as B
    return B


def test_int8_gemm(B):
    m, n, k = 200, 8, 64
    a, w = fake(torch.int8, m, k), fake(torch.int8, n, k)
    sa, sw, out = fake(torch.float32, m), fake(torch.float32, n), fake(torch.bfloat16, m, n)
    scratch = fake(torch.uint8, B.int8_gemm_scratch_bytes(m, n, k), device=CUDA1)
    with pytest.raises(ValueError, match="cuda:1"):
        B.int8_gemm(a, sa, w, sw, out=out, scratch=scratch)


def test_gated_delta_prefill(B):
    q, k, v, o = (fake(torch.bfloat16, 5, 1, 128) for _ in range(4))
    g, beta, state = fake(torch.float32, 5, 1), fake(torch.float32, 5, 1), fake(torch.float32, 1, 1, 128, 128)
    scratch = fake(torch.uint8, B.gated_delta_prefill_scratch_bytes(1, 5, 1, 1), device=CUDA1)
    with pytest.raises(ValueError, match="cuda:1"):
        B.gated_delta_prefill(q, k, v, g, beta, state, out=o, scratch=scratch)
