"""Attention over capped, biased and masked scores against the fp64 oracle.

Tolerances.  u = 2^-8 is half a step of bf16, e = 2^-24 of fp32.
  A score is off by at most ds: the d products of q.k add up in fp32 (2 d e times scale sum |q_x k_x|, counting a
  truncated alignment as two roundings), a cap's exponential, reciprocal and products 16 e cap, a bias 4 e slope
  |distance|, scaling 4 e |score|.
  o: the output rounds once (u |o|); each probability rounds to bf16 once before it meets v (u sum p |v|) and is off by
  ds and the exponential's 8 e relative, as is the row sum.  So u |o| + (u + 2 ds + 32 e) sum p |v|.
  lse: ds + 16 e (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import patch_attention_b200 as pa
from oracle import block
from tests._bounds import within
from tests._oracle_util import f64

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24
BF = torch.bfloat16


def inputs(b, nq, nk, hq, hk, d, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return (scale * r(b, nq, hq, d)).to(BF), r(b, nk, hk, d).to(BF), r(b, nk, hk, d).to(BF)


def score_error(q, k, rule, scale):
    """Largest error ds of a score, over the whole problem."""
    Q, K = np.abs(f64(q)), np.abs(f64(k))
    if K.size == 0 or Q.size == 0:
        return 0.0
    d = Q.shape[-1]
    # |q|.|k| of the largest rows by Cauchy-Schwarz
    top = scale * np.sqrt((Q ** 2).sum(-1).max() * (K ** 2).sum(-1).max())
    ds = (2 * d + 4) * E * top
    if rule.softcap:
        ds += 16 * E * rule.softcap
    if rule.slopes is not None:
        ds += 4 * E * float(rule.slopes.abs().max()) * max(Q.shape[1], K.shape[1])
    return ds


def oracle_args(rule, d):
    n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    scale = rule.softmax_scale or d ** -0.5
    return scale, dict(softcap=rule.softcap, slopes=n(rule.slopes), causal=rule.causal, prefix=n(rule.prefix),
                       doc_q=n(rule.doc_q), doc_k=n(rule.doc_k))


def clean(t):
    """A copy without NaN and infinities, for error bounds."""
    return torch.nan_to_num(t.float(), 0.0, 0.0, 0.0)


def check(q, k, v, rule=None, **kw):
    rule = rule or pa.ScoreRule()
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True, **kw)
    torch.cuda.synchronize()
    pa.pf_device_status()
    assert torch.equal(o, pa.masked_attention(q, k, v, rule, **kw))  # with and without lse
    scale, args = oracle_args(rule, q.shape[-1])
    ro, rl = block.masked_attention(f64(q), f64(k), f64(v), scale, **args)
    ra, _ = block.masked_attention(f64(q), f64(k), np.abs(f64(clean(v))), scale, **args)
    ds = score_error(clean(q), clean(k), rule, scale)
    within(f64(o), ro, U * np.abs(ro) + (U + 2 * ds + 32 * E) * ra, "o")
    got = f64(lse)
    none = np.isneginf(rl)
    assert np.array_equal(none, np.isneginf(got))
    within(got[~none], rl[~none], ds + 16 * E * (1 + np.abs(rl[~none])), "lse")
    assert not f64(o)[np.moveaxis(none, 1, 2)].any()  # a query that sees nothing gives 0
    return o, lse


def slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def documents(b, n, seed=0, most=200, pad=True):
    """Ragged runs of ids in any order, with padding between and after them."""
    rng = np.random.default_rng(seed)
    out = np.full((b, n), -1, dtype=np.int32)
    for i in range(b):
        at = 0
        while at < n:
            run = int(rng.integers(1, most))
            out[i, at:at + run] = -3 if pad and rng.random() < 0.2 else int(rng.integers(0, 9))
            at += run
    return torch.from_numpy(out).cuda()


# ends inside tiles and halves, one and two query tiles per CTA, split and unsplit keys
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 63), (1, 64), (1, 65), (1, 129), (2, 3), (64, 64), (127, 200), (128, 128),
                                   (129, 300), (200, 1000), (257, 257), (384, 640)])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_sizes(nq, nk, d):
    check(*inputs(2, nq, nk, 2, 2, d, seed=nq + nk))


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 500), (3, 500), (100, 100), (129, 130), (300, 300), (300, 17), (260, 700)])
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("prefix", [False, True])
def test_causal_and_prefix(nq, nk, d, prefix):
    q, k, v = inputs(3, nq, nk, 2, 1, d, seed=nq)
    p = torch.tensor([0, nk // 2 + 1, nk + 5], device="cuda", dtype=torch.int32) if prefix else None
    check(q, k, v, pa.ScoreRule(causal=True, prefix=p))


@pytest.mark.parametrize("b,hq,hk,nq,nk", [(1, 3, 1, 1, 700), (2, 24, 8, 1, 300), (1, 5, 1, 7, 260), (1, 8, 2, 40, 200),
                                           (1, 6, 2, 200, 333), (1, 130, 1, 1, 64), (2, 40, 20, 130, 150), (40, 4, 4, 1, 129),
                                           (1, 128, 1, 2, 90)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_heads_and_split_keys(b, hq, hk, nq, nk, d):
    check(*inputs(b, nq, nk, hq, hk, d, seed=hq), pa.ScoreRule(causal=True))


@pytest.mark.parametrize("cap", [0.0, 5.0, 50.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("nq,nk", [(1, 400), (250, 250), (140, 300)])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_cap_and_bias(cap, bias, nq, nk, d):
    q, k, v = inputs(1, nq, nk, 4, 2, d, seed=3, scale=3.0)
    check(q, k, v, pa.ScoreRule(softcap=cap, slopes=slopes(4) if bias else None))
    check(q, k, v, pa.ScoreRule(softcap=cap, slopes=slopes(4) if bias else None, causal=True, softmax_scale=0.2))


@pytest.mark.parametrize("n", [5, 128, 300, 515, 1100])
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_documents(n, d, causal):
    q, k, v = inputs(2, n, n, 2, 2, d, seed=n)
    doc = documents(2, n, seed=n)
    check(q, k, v, pa.ScoreRule(causal=causal, doc_q=doc, doc_k=doc))


def test_documents_of_other_lengths_and_everything_at_once():
    q, k, v = inputs(2, 300, 520, 6, 2, 64, seed=8)
    rule = pa.ScoreRule(softcap=20.0, slopes=slopes(6), causal=True,
                        prefix=torch.tensor([100, 400], device="cuda", dtype=torch.int32),
                        doc_q=documents(2, 300, 1), doc_k=documents(2, 520, 2))
    check(q, k, v, rule)
    # ids of one row each, in a shuffled order: every row of a warp in a document of its own
    perm = torch.stack([torch.randperm(256), torch.randperm(256)]).to("cuda", torch.int32)
    q, k, v = inputs(2, 256, 256, 2, 2, 64, seed=9)
    o, _ = check(q, k, v, pa.ScoreRule(doc_q=perm, doc_k=perm.roll(3, 1).contiguous()))
    assert torch.equal(o, v.roll(-3, 1))  # each query copies the one value it sees


def test_any_negative_id_is_padding():
    q, k, v = inputs(1, 128, 128, 1, 1, 64, seed=14)
    doc = torch.zeros(1, 128, device="cuda", dtype=torch.int32)
    doc[0, 5], doc[0, 77], doc[0, 127] = -2 ** 31, -1, -7
    check(q, k, v, pa.ScoreRule(doc_q=doc, doc_k=doc))


def test_scores_beyond_half_the_cap_and_within():
    # some rows of a warp take the exponential form of the cap, others alone would not
    q, k, v = inputs(1, 200, 300, 2, 2, 64, seed=15)
    for cap in (1.0, 2.0, 8.0, 100.0):
        check(q, k, v, pa.ScoreRule(softcap=cap))
    q[:, 40:60] *= 30
    check(q, k, v, pa.ScoreRule(softcap=8.0, slopes=slopes(2)))


def test_no_keys_no_queries():
    q, k, v = inputs(2, 5, 0, 2, 2, 64)
    o, lse = check(q, k, v)
    assert not o.any() and torch.isneginf(lse).all()
    q, k, v = inputs(2, 0, 5, 2, 2, 64)
    assert pa.masked_attention(q, k, v).shape == q.shape
    doc = torch.full((2, 7), -1, device="cuda", dtype=torch.int32)
    q, k, v = inputs(2, 7, 7, 2, 2, 64)
    o, lse = check(q, k, v, pa.ScoreRule(doc_q=doc, doc_k=doc))
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_unseen_places_may_hold_anything(value, d):
    # padding keys and queries between documents, and a document of keys that no query has
    q, k, v = inputs(1, 300, 300, 2, 2, d, seed=4)
    doc = documents(1, 300, seed=5)
    dk = doc.clone()
    dk[0, 130:140] = 4
    doc[doc == 4] = 5
    rule = pa.ScoreRule(doc_q=doc, doc_k=dk)
    want, wl = check(q, k, v, rule)
    unseen = (dk < 0) | (dk == 4)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[doc < 0] = value
    k2[unseen] = value
    v2[unseen] = value
    got, gl = pa.masked_attention(q2, k2, v2, rule, want_lse=True)
    assert torch.equal(want, got) and torch.equal(wl, gl)
    # keys behind the last position that the queries see, split over CTAs too
    for nq, cut in ((1, 200), (150, 170)):
        q, k, v = inputs(1, nq, 300, 2, 2, d, seed=6)
        pre = torch.tensor([0], device="cuda", dtype=torch.int32)
        big = pa.masked_attention(q, k[:, :cut].contiguous(), v[:, :cut].contiguous(), pa.ScoreRule(causal=True, prefix=pre))
        doc_k = torch.zeros(1, 300, device="cuda", dtype=torch.int32)
        doc_k[:, cut:] = -1
        k[:, cut:], v[:, cut:] = value, value
        o = pa.masked_attention(q, k, v, pa.ScoreRule(doc_q=torch.zeros(1, nq, device="cuda", dtype=torch.int32), doc_k=doc_k))
        assert torch.isfinite(o).all()
        if nq == 1:
            assert (o.float() - big.float()).abs().max() <= 2 * U * big.float().abs().max()


def test_a_seen_nan_shows_and_infinite_scores():
    q, k, v = inputs(1, 200, 200, 1, 1, 64, seed=7)
    k[0, 77, 0, 3] = float("nan")
    o = pa.masked_attention(q, k, v, pa.ScoreRule(causal=True))
    assert torch.isfinite(o[0, :77]).all() and torch.isnan(o[0, 77:]).all()
    # a score of -inf is a key that weighs nothing
    q, k, v = inputs(1, 3, 50, 1, 1, 64, seed=7)
    q[..., 0], k[..., 0] = 1.0, 0.0
    k[0, 9, 0, 0] = float("-inf")
    keep = [i for i in range(50) if i != 9]
    a, b = pa.masked_attention(q, k, v), pa.masked_attention(q, k[:, keep].contiguous(), v[:, keep].contiguous())
    assert (a.float() - b.float()).abs().max() <= 2 * U * b.float().abs().max()


@pytest.mark.parametrize("nq", [1, 200])
def test_large_scores_and_growing_maxima(nq):
    # scores in the hundreds whose maximum keeps rising: O is rescaled tile after tile
    q, k, v = inputs(1, nq, 900, 2, 2, 128, seed=10, scale=4.0)
    k = (k.float() * torch.linspace(0.1, 6.0, 900, device="cuda")[None, :, None, None]).to(BF)
    check(q, k, v)
    check(q, k.flip(1).contiguous(), v)


def test_strided_views():
    qkv = torch.randn(2, 150, 3, 4, 72, device="cuda").to(BF)
    q, k, v = qkv.unbind(2)
    want = pa.masked_attention(q.contiguous(), k.contiguous(), v.contiguous(), pa.ScoreRule(causal=True))
    assert torch.equal(pa.masked_attention(q, k, v, pa.ScoreRule(causal=True)), want)
    # heads before tokens, and a window of a longer cache
    cache = torch.full((2, 4, 400, 72), float("nan"), device="cuda", dtype=BF)
    cache[:, :, 100:250] = k.transpose(1, 2)
    win = cache.transpose(1, 2)[:, 100:250]
    assert torch.equal(pa.masked_attention(q, win, v, pa.ScoreRule(causal=True)), want)
    o = pa.masked_attention(q[:, -1:], win, v, pa.ScoreRule(causal=True))
    assert (o.float() - want[:, -1:].float()).abs().max() <= 4 * U * want.float().abs().max()


def test_rows_behind_the_last_query_are_left_alone():
    q, k, v = inputs(1, 130, 200, 3, 3, 64, seed=11)
    for nq in (1, 3, 130):
        buf = torch.full((nq * 3 * 64 + 4096,), 7.0, device="cuda", dtype=BF)
        pa.pf_masked_attn(q[:, :nq].contiguous(), k, v, buf[:nq * 3 * 64].view(1, nq, 3, 64))
        assert (buf[nq * 3 * 64:] == 7.0).all()


def test_repeated_bits_side_stream_and_graphs():
    q, k, v = inputs(2, 300, 700, 4, 2, 64, seed=12)
    q1 = q[:, :1].contiguous()
    doc_q, doc_k = documents(2, 300, 3), documents(2, 700, 4)
    rules = [pa.ScoreRule(causal=True), pa.ScoreRule(doc_q=doc_q, doc_k=doc_k, softcap=10.0)]

    def both(**kw):
        return [pa.masked_attention(q, k, v, r, want_lse=True, **kw) for r in rules] + [
            pa.masked_attention(q1, k, v, rules[0], want_lse=True, **kw)]

    want = both()
    same = lambda got: all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))  # noqa: E731
    assert same(both())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = both(stream=side), both()  # two streams at once
    torch.cuda.synchronize()
    assert same(a) and same(b)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = both()
        graphs.append((g, got))
    for g, got in graphs + graphs:
        g.replay()
        torch.cuda.synchronize()
        assert same(got)


def test_after_and_before_the_patch_attention():
    # the patch kernels release their dependents early: a masked call between two of them still sees
    # finished inputs, and they its outputs
    pat = pa.PatchAttention(1, 4, 64, 1024, 4, 0, 1)
    x = torch.randn(1, 1024, 4, 64, device="cuda").to(BF)
    pat.init_layer(0, x, x)
    p = [x[:, i * 256:(i + 1) * 256].contiguous() for i in range(4)]
    try:
        outs = []
        for rep in range(2):
            if rep:
                torch.cuda.synchronize()
            o0 = pat.step(0, 0, p[0], p[0], p[0])
            m = pa.masked_attention(o0, o0, o0, pa.ScoreRule(causal=True))
            if rep:
                torch.cuda.synchronize()
            o1 = pat.step(0, 1, m, m, m)
            outs.append((o0, m, o1))
            torch.cuda.synchronize()
            pat.check()
            pat.init_layer(0, x, x)
        assert all(torch.equal(a, b) for a, b in zip(*outs))
    finally:
        pat.close()
