"""Outputs of the layer of examples/linear_attention.py: single tokens against prompts, and the whole layer
against its definition in 64 bits.

Bounds.  A BF16 store is off by at most 2^-8 of the value, by 2^-8 / sqrt(3) in the mean square, so two
stores of the same value differ by 2^-8 sqrt(2 / 3) in the mean square; the prompts' one-term products add about 2^-12.
Together below 2^-8.  Behind the second quantiser (codes of step s) either side's codes carry errors of s / sqrt(12), so
the two differ by at most s / sqrt(6) in the mean square, beside the 2^-8 of the rule's outputs and of the gate's store."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def example():
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import linear_attention
    return linear_attention


@pytest.mark.parametrize("prompts", [(1,), (63, 1, 130), (64, 200)])
def test_single_tokens_give_the_outputs_of_prompts(example, prompts):
    out_err, _ = example.run(hidden=512, heads_k=2, heads_v=6, prompts=prompts, steps=4)
    assert out_err <= 2.0 ** -8


def quantised(y):
    s = y.abs().amax(1, keepdim=True) / 127
    t = y / s
    return torch.copysign((t.abs() + 0.5).floor(), t) * s, s


def definition(layer, x, r, lens):
    """(rule's outputs, layer's outputs, step of the second quantiser over its values) in 64 bits; the BF16 stores in
    between are kept, as the next step reads them."""
    bf = lambda t: t.float().bfloat16().double()  # noqa: E731
    cpu = lambda t: t.cpu().double()  # noqa: E731
    hk, hv = layer.hk, layer.hv
    h = cpu(x) + cpu(r)
    y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * cpu(layer.norm)
    p = bf(quantised(y)[0] @ (cpu(layer.w_in) * cpu(layer.s_in)[:, None]).T)
    q, k, v, z, a, b, _ = p.split((hk * D, hk * D, hv * D, hv * D, hv, hv, p.shape[1] - (2 * hk + 2 * hv) * D - 2 * hv), 1)
    q, k = (t.unflatten(1, (hk, D)) for t in (q, k))
    q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(hv // hk, 1) for t in (q, k))
    v = v.unflatten(1, (hv, D))
    g, beta = cpu(layer.decay) * torch.nn.functional.softplus(a), torch.sigmoid(b)
    o = torch.zeros_like(v)
    t = 0
    for n in lens:
        S = torch.zeros(hv, D, D, dtype=torch.float64)
        for _ in range(n):
            S = S * g[t].exp()[:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            o[t] = torch.einsum("hkv,hk->hv", S, q[t]) * D ** -0.5
            t += 1
    gated = bf(z * torch.sigmoid(z) * bf(o).flatten(1))
    values, s = quantised(gated)
    return o, values @ (cpu(layer.w_out) * cpu(layer.s_out)[:, None]).T, \
        float((s.square().mean() / gated.square().mean()).sqrt())


def test_layer_against_its_definition(example):
    lens = (63, 1, 70)
    layer = example.LinearAttention(512, 2, 6, slots=3, seed=3)
    g = torch.Generator("cuda").manual_seed(4)
    x, r = (torch.randn(sum(lens), 512, generator=g, device="cuda").bfloat16() for _ in range(2))
    cu = torch.tensor([0, 63, 64, 134], dtype=torch.int32, device="cuda")
    y, h = layer.prefill(x, r, cu, torch.arange(3, dtype=torch.int32, device="cuda"))
    o64, y64, step = definition(layer, x, r, lens)
    rms = lambda a, b: float(((a.cpu().double() - b).square().sum() / b.square().sum()).sqrt())  # noqa: E731
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    assert rms(layer.heads_out, o64) <= 2.0 ** -8
    assert rms(y, y64) <= step / 6 ** 0.5 + 2 * 2.0 ** -8
