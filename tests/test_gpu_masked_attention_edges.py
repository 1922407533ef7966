"""Masked attention at the ends of its arguments' ranges.  Tolerances as in the forward and backward tests, or equal
bits."""
import numpy as np
import pytest
import torch

import patch_attention_b200 as pa
from tests._bounds import within
from tests._oracle_util import f64
from tests.test_gpu_masked_attention import BF, E, check, documents, inputs, slopes
from tests.test_gpu_masked_attention_bwd import check as check_bwd

pytestmark = pytest.mark.gpu


def forward_and_backward(q, k, v, rule, seed=100):
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(q.shape, device="cuda", generator=g).to(BF)
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True)
    return (o, lse) + pa.masked_attention_backward(do, q, k, v, o, lse, rule)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("prefix", [-2 ** 31, -2 ** 31 + 1, -1, 0])
@pytest.mark.parametrize("nq,nk", [(1, 500), (300, 300), (260, 700)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_prefix_below_zero_is_none(prefix, nq, nk, d):
    q, k, v = inputs(2, nq, nk, 4, 2, d, seed=nq)
    # the other batch element has a prefix
    p = torch.tensor([prefix, nk // 2], device="cuda", dtype=torch.int32)
    rule = pa.ScoreRule(causal=True, prefix=p)
    check(q, k, v, rule)
    check_bwd(q, k, v, rule)
    first = [t[:1].contiguous() for t in (q, k, v)]
    got = forward_and_backward(*first, pa.ScoreRule(causal=True, prefix=p[:1].contiguous()))
    assert same(got, forward_and_backward(*first, pa.ScoreRule(causal=True)))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (2, 2, 72), (6, 2, 128)])
def test_a_nan_or_infinite_score_shows_where_keys_are_split(value, hq, hk, d):
    # one query against nine key tiles: the keys are split over a cluster (tests/test_masked_plan_host.py)
    q, k, v = inputs(1, 1, 1100, hq, hk, d, seed=21)
    want = forward_and_backward(q, k, v, None)
    q[0, 0, hq - 1, 3] = value  # keys of either sign there: scores of +inf and -inf, or NaN
    o, lse, dq, dk, dv = forward_and_backward(q, k, v, None)
    assert torch.isnan(o[0, 0, hq - 1]).all() and torch.isnan(lse[0, hq - 1]).all()
    assert torch.isnan(dq[0, 0, hq - 1]).all()
    assert torch.isnan(dk[:, :, hk - 1]).all() and torch.isnan(dv[:, :, hk - 1]).all()
    # the other heads are untouched
    assert torch.equal(o[:, :, :hq - 1], want[0][:, :, :hq - 1]) and torch.equal(lse[:, :hq - 1], want[1][:, :hq - 1])
    assert torch.equal(dq[:, :, :hq - 1], want[2][:, :, :hq - 1])
    assert torch.equal(dk[:, :, :hk - 1], want[3][:, :, :hk - 1])


@pytest.mark.parametrize("at", [0, 700, 1099])
def test_a_nan_key_shows_where_keys_are_split(at):
    q, k, v = inputs(1, 1, 1100, 2, 2, 64, seed=22)
    k[0, at, 1, 5] = float("nan")
    o, lse = pa.masked_attention(q, k, v, want_lse=True)
    assert torch.isfinite(o[:, :, 0]).all() and torch.isnan(o[:, :, 1]).all() and torch.isnan(lse[:, 1]).all()


def test_parts_of_split_keys_that_see_nothing():
    # documents of a single key tile: the other parts of the cluster hold nothing and say so
    q, k, v = inputs(1, 1, 1100, 2, 2, 64, seed=23)
    doc_k = torch.full((1, 1100), 3, device="cuda", dtype=torch.int32)
    doc_k[0, 600:640] = 0
    check(q, k, v, pa.ScoreRule(doc_q=torch.zeros(1, 1, device="cuda", dtype=torch.int32), doc_k=doc_k))
    q[0, 0, 1, 0] = float("nan")
    o, lse = pa.masked_attention(q, k, v, pa.ScoreRule(doc_q=torch.zeros(1, 1, device="cuda", dtype=torch.int32),
                                                       doc_k=doc_k), want_lse=True)
    assert torch.isfinite(o[:, :, 0]).all() and torch.isnan(o[:, :, 1]).all() and torch.isnan(lse[:, 1]).all()
    o, lse = pa.masked_attention(q, k, v, pa.ScoreRule(doc_q=torch.ones(1, 1, device="cuda", dtype=torch.int32),
                                                       doc_k=doc_k), want_lse=True)
    assert not o.any() and torch.isneginf(lse).all()  # it sees no key, whatever it holds


@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_a_capped_row_does_not_depend_on_its_neighbours(d, bias):
    # the cap's two forms are chosen element by element: rows beyond half the cap change no other row's bits
    q, k, v = inputs(1, 200, 300, 2, 2, d, seed=24)
    rule = pa.ScoreRule(softcap=20.0, slopes=slopes(2) if bias else None)
    want = forward_and_backward(q, k, v, rule)
    q2 = q.clone()
    q2[:, 40:60] *= 30
    got = forward_and_backward(q2, k, v, rule)
    keep = [i for i in range(200) if not 40 <= i < 60]
    assert torch.equal(got[0][:, keep], want[0][:, keep]) and torch.equal(got[1][:, :, keep], want[1][:, :, keep])
    assert torch.equal(got[2][:, keep], want[2][:, keep])
    assert not torch.equal(got[0][:, 40:60], want[0][:, 40:60])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e4])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_unseen_keys_under_a_cap_may_hold_anything(value, d):
    q, k, v = inputs(1, 300, 300, 2, 1, d, seed=25)
    doc = documents(1, 300, seed=5)
    dk = doc.clone()
    dk[0, 130:140] = 4
    doc[doc == 4] = 5
    for causal in (False, True):
        rule = pa.ScoreRule(softcap=20.0, slopes=slopes(2), causal=causal, doc_q=doc, doc_k=dk)
        want = forward_and_backward(q, k, v, rule)
        unseen = (dk < 0) | (dk == 4)
        k2, v2 = k.clone(), v.clone()
        k2[unseen] = value
        v2[unseen] = value
        assert same(forward_and_backward(q, k2, v2, rule), want)


@pytest.mark.parametrize("hq,d", [(3, 64), (5, 64), (3, 72), (7, 128)])
def test_a_capped_tile_with_unwritten_rows_repeats_its_bits(hq, d):
    # heads that share a key head and do not divide 128 leave the last rows of a query tile unwritten; the calls in
    # between leave large and small numbers in shared memory there
    q, k, v = inputs(1, 200, 300, hq, 1, d, seed=26)
    rule = pa.ScoreRule(softcap=20.0)
    f = inputs(1, 128, 128, 160, 160, d, seed=27)
    got = []
    for size in (0.0, 1e3):
        pa.masked_attention((f[0].float() * size).to(BF), f[1], f[2], rule)
        got.append(pa.masked_attention(q, k, v, rule, want_lse=True))
    check(q, k, v, rule)
    assert same(*got)


@pytest.mark.parametrize("cap", [1.0, 30.0, 1e4, 1e6])
@pytest.mark.parametrize("mixed", [False, True])
def test_the_cap_is_exact_far_below_it(cap, mixed):
    """With one key and one non-zero column the score is a product of two bf16 numbers, exact in fp32, and lse is the
    capped score w.  With y = s / cap: the polynomial (|y| <= 1/2) is within 9.3 E (5.6e-7) of tanh relative to it,
    scale / cap, y, y^2, three steps, the last product, the factor and its log2(e) round once each (10 E), the
    reference and lse twice more (3 E): 24 E |w|.  Beyond, 1 - 2 / (1 + exp(2 y)): the argument rounds three times
    (relative 3 E of 2 y: 6 E y exp(2 y) in exp(2 y), at most 1.4 E after division), the exponential and the
    reciprocal are approximate by 4 E each, the difference and the factor as above: 16 E cap + 6 E |w|."""
    g = torch.Generator(device="cuda").manual_seed(28)
    n = 256
    frac = torch.rand(n, device="cuda", generator=g) * 0.49 * torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)
    frac[::3] *= 1e-3
    frac[::7] *= 1e-5
    if mixed:  # every fifth row beyond half the cap
        frac[::5] = 0.6 + 3.0 * torch.rand(frac[::5].shape, device="cuda", generator=g)
    q = torch.zeros(1, n, 1, 64, device="cuda", dtype=BF)
    q[0, :, 0, 0] = (frac * cap).to(BF)
    k = torch.zeros(1, 1, 1, 64, device="cuda", dtype=BF)
    k[..., 0] = 1.0
    v = torch.ones_like(k)
    o, lse = pa.masked_attention(q, k, v, pa.ScoreRule(softcap=cap, softmax_scale=1.0), want_lse=True)
    s = f64(q[0, :, 0, 0])
    w = cap * np.tanh(s / cap)
    bound = np.where(np.abs(s) <= 0.5 * cap, 24 * E * np.abs(w), 16 * E * cap + 6 * E * np.abs(w))
    within(f64(lse[0, 0]), w, bound, "lse")
    assert (o == 1.0).all()
