"""The gated delta rule at the ends of its range: very large states, chunks that write nothing, keys and
queries that underflow, queries that are stored keys.  Bounds as in test_gated_delta_gpu.py unless a
test derives its own."""
import numpy as np
import pytest
import torch

from helpers import bf16_half_ulp
from test_gated_delta_gpu import check, make, reference

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_quantized_linear_q8_gb300 import build
    build.build()
    import bit_quantized_linear_q8_gb300 as B
    return B


def both_forms(B, args, state, tokens, **kw):
    """(name, out, new state) of the prefill and of single-token calls."""
    s = state.clone()
    yield "prefill", B.gated_delta_prefill(*args, s, **kw), s
    s = state.clone()
    out = [B.gated_delta_decode(*(a[t:t + 1] for a in args), s, **kw) for t in range(tokens)]
    yield "decode", torch.cat(out), s


@pytest.mark.parametrize("size", [1e5, 1e6, 1e20, 1e35])
@pytest.mark.parametrize("tokens", [1, 64, 65, 130])
def test_large_state_that_nothing_writes(B, size, tokens):
    # beta = 0 everywhere: the state decays by e^(sum g) and nothing else happens
    q, k, v, g, beta, state = make(tokens, tokens, 1, 2, 1, decay=0.01)
    beta.zero_()
    g[:, 0] = 0
    state *= 10 * size
    state[0, :, :, 5] = 0  # a column of zeros beside the large ones
    ref = reference(q, k, v, g, beta, state, [tokens])
    for what, out, s in both_forms(B, (q, k, v, g, beta), state, tokens):
        assert torch.equal(s[0, 0], state[0, 0]), what
        check(out, s, ref, what)


@pytest.mark.parametrize("size", [1e5, 1e20, 1e35])
@pytest.mark.parametrize("tokens", [1, 64, 65, 130])
@pytest.mark.parametrize("forget", [float("-inf"), -500.0])
def test_large_state_is_forgotten(B, size, tokens, forget):
    # the first token forgets the state: the rest is as from a state of zeros, also where nothing is
    # written (v = 0 in a few columns, beta = 0 in one head)
    q, k, v, g, beta, state = make(tokens + 1, tokens, 1, 2, 1)
    v = v.clone()
    v[:, :, 3:9] = 0
    beta[:, 1] = 0
    g[0] = forget
    state *= 10 * size
    ref = reference(q, k, v, g, beta, torch.zeros_like(state), [tokens])
    for what, out, s in both_forms(B, (q, k, v, g, beta), state, tokens):
        check(out, s, ref, what)
        assert not s[0, 1].any() and not s[0, 0, :, 3:9].any(), what


@pytest.mark.parametrize("tokens", [1, 65])
def test_largest_state_is_forgotten(B, tokens):
    # Products with such a state leave fp32, and nothing of them may stay: what comes out is what comes from a
    # state of zeros.  Scales by powers of two do not change how terms are rounded, so the states agree as
    # closely as fp32 sums do and the outputs to a BF16 neighbour.
    q, k, v, g, beta, state = make(tokens + 2, tokens, 1, 2, 1)
    q, k = q.abs(), k.abs()
    g[0] = float("-inf")
    state.fill_(3e38)
    zeros = torch.zeros_like(state)
    mag = reference(q, k, v, g, beta, zeros, [tokens])[2].cuda()
    args = (q, k, v, g, beta)
    for (what, out, s), (_, out0, s0) in zip(both_forms(B, args, state, tokens), both_forms(B, args, zeros, tokens)):
        assert bool(((s - s0).abs() <= 2.0 ** -17 * mag[:, None, None]).all()), what
        limit = 2.0 ** -7 * out0.float().abs() + 2.0 ** -17 * mag[:, None]
        assert bool(((out.float() - out0.float()).abs() <= limit).all()), what


def test_large_state_forgotten_in_mid_prompt(B):
    # a chunk that writes nothing, then one that forgets, then ordinary ones; compared with a start from zeros there
    q, k, v, g, beta, state = make(9, 300, 1, 2, 1)
    state *= 1e21
    beta[:64] = 0
    g[:64] = 0
    g[64] = float("-inf")
    zero = torch.zeros_like(state)
    rest = (q[64:], k[64:], v[64:], g[64:], beta[64:])
    ref = reference(*rest, zero, [236])
    for what, out, s in both_forms(B, (q, k, v, g, beta), state, 300):
        check(out[64:], s, ref, what)
        assert torch.isfinite(out[:64]).all(), what


@pytest.mark.parametrize("tokens", [1, 70])
def test_normalised_rows_that_underflow(B, tokens):
    # sums of squares that are subnormal or zero in fp32: x / sqrt(0 + 1e-6) is tiny, not NaN
    q, k, v, g, beta, state = make(21, tokens, 2, 4, 1, normed=False)
    sizes = torch.tensor([1e-18, 1e-20, 1e-22, 3e-24, 1e-25, 1e-28, 1e-33, 1e-37, 2e-39, 0.0])
    for t in range(tokens):
        k[t, t % 2] *= sizes[t % 10].item()
        q[t, (t + 1) % 2] *= sizes[(t + 4) % 10].item()
    ref = reference(q, k, v, g, beta, state, [tokens], l2norm=True)
    for what, out, s in both_forms(B, (q, k, v, g, beta), state, tokens, l2norm=True):
        check(out, s, ref, what)


def test_one_tiny_row_keeps_its_digits(B):
    # with a key of 1e-25 and no normalisation of the query, the output is that of the scaled key
    q, k, v, g, beta, state = make(22, 1, 1, 1, 1, normed=False)
    k *= 1e-25
    q *= 1e-25
    ref = reference(q, k, v, g, beta, state, [1], l2norm=True)
    for what, out, s in both_forms(B, (q, k, v, g, beta), state, 1, l2norm=True):
        o = ref[0].numpy()
        # a query of 1e-22 after the norm: 2^-10 of sum |S q|, which random signs keep below 128 x the mean
        lim = bf16_half_ulp(o) * (1 + 2.0 ** -7) + 2.0 ** -10 * (state.double().abs().amax() * q.double().abs().sum() * 1e3).item() * D ** -0.5
        assert np.all(np.abs(out.cpu().double().numpy() - o) <= lim), what
        assert np.abs(out.cpu().double().numpy()).max() > 0, what


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


def out_of_order(cu, total):
    """The sequences that a list of bounds gives: bounds that are negative, past the end or below an
    earlier one make theirs empty."""
    spans, most = [], cu[0]
    for a, b in zip(cu[:-1], cu[1:]):
        good = 0 <= a <= b <= total and a >= most
        spans.append((a, b) if good else (0, 0))
        most = max(most, a, b)
    return spans


# one head: chunks prepared beside the recurrence; many heads, and more sequences than are ordered: before it
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 32)])
@pytest.mark.parametrize("cu", [[0, 200, 100, 300], [0, 130, 60, 190, 150, 300, 300], [0, 64, 500, 100, 300],
                                [-5, 40, 20, 90, 300], [300, 0, 100, 300]])
def test_bounds_out_of_order(B, cu, hk, hv):
    total, n = 300, len(cu) - 1
    a = make(31 + n, total, hk, hv, n)
    spans = out_of_order(cu, total)
    state, out = a[5].clone(), torch.full((total, hv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    B.gated_delta_prefill(*a[:5], state, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
    torch.cuda.synchronize()
    assert B.lib().bq_device_status() == 0
    rest = torch.ones(total, dtype=torch.bool)
    for s, (i, j) in enumerate(spans):
        if i == j:
            assert torch.equal(state[s], a[5][s]), s
            continue
        rest[i:j] = False
        ref = reference(*(t[i:j] for t in a[:5]), a[5][s:s + 1], [j - i])
        check(out[i:j], state[s:s + 1], ref, (cu, s))
    assert (out.cpu()[rest] == 7).all()


def test_bounds_out_of_order_among_many(B):
    # 600 sequences, two of them with a bound that belongs elsewhere
    lens = [1 + (i * 7) % 5 for i in range(600)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    total = cu[-1]
    cu[100], cu[500] = cu[100] - 40, cu[500] + 150
    a = make(33, total, 1, 1, 600)
    state, out = a[5].clone(), torch.full((total, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    B.gated_delta_prefill(*a[:5], state, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
    spans = out_of_order(cu, total)
    assert 0 < sum(i == j for i, j in spans) < 300
    rest = torch.ones(total, dtype=torch.bool)
    for s, (i, j) in enumerate(spans):
        if i == j:
            assert torch.equal(state[s], a[5][s]), s
            continue
        rest[i:j] = False
        ref = reference(*(t[i:j] for t in a[:5]), a[5][s:s + 1], [j - i])
        check(out[i:j], state[s:s + 1], ref, s)
    assert (out.cpu()[rest] == 7).all()
