"""Masked attention in calls large enough for two query tiles per CTA, forward and backward, against the fp64
oracle.  Heads are independent but for shared keys, so a few groups of heads stand for all in the comparison; the tolerances
are those of the other tests, over these heads."""
import numpy as np
import pytest
import torch

import patch_attention_b200 as pa
from oracle import block
from tests._bounds import within
from tests._oracle_util import f64
from tests._two_tiles import HEAD_BY_HEAD, TWO_TILES
from tests.test_gpu_masked_attention import BF, E, U, clean, documents, inputs, oracle_args, score_error, slopes
from tests.test_gpu_masked_attention_bwd import bounds

pytestmark = pytest.mark.gpu


def rule_of(b, nq, nk, hq, letters, seed=0):
    """k: cap, b: bias, c: causal, p: prefix, d: documents."""
    doc = {}
    if "d" in letters:
        every = documents(b, max(nq, nk), seed)
        doc = dict(doc_q=every[:, -nq:].contiguous(), doc_k=every[:, :nk].contiguous())
    prefix = torch.tensor([(37 + 200 * i) % (nk + 50) for i in range(b)], device="cuda", dtype=torch.int32)
    return pa.ScoreRule(softcap=20.0 if "k" in letters else 0.0, slopes=slopes(hq) if "b" in letters else None,
                        causal="c" in letters, prefix=prefix if "p" in letters else None, **doc)


def check_heads(q, k, v, rule, groups, batches):
    """The whole call, compared in some batch elements and the query heads of some key heads."""
    g = torch.Generator(device="cuda").manual_seed(100)
    do = torch.randn(q.shape, device="cuda", generator=g).to(BF)
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True)
    grads = pa.masked_attention_backward(do, q, k, v, o, lse, rule)
    torch.cuda.synchronize()
    pa.pf_device_status()
    assert torch.equal(o, pa.masked_attention(q, k, v, rule))
    share = q.shape[2] // k.shape[2]
    heads = [h for x in groups for h in range(x * share, x * share + share)]
    cut = lambda t, at: None if t is None else t[at].contiguous()  # noqa: E731
    part = pa.ScoreRule(rule.softmax_scale, rule.softcap, cut(rule.slopes, heads), rule.causal, cut(rule.prefix, batches),
                        cut(rule.doc_q, batches), cut(rule.doc_k, batches))
    few = lambda t, at: t[batches][:, :, at].contiguous()  # noqa: E731
    q, do, o, dq = (few(t, heads) for t in (q, do, o, grads[0]))
    k, v, dk, dv = (few(t, groups) for t in (k, v, *grads[1:]))
    scale, args = oracle_args(part, q.shape[-1])
    ro, rl, *rg = block.masked_attention(f64(q), f64(k), f64(v), scale, do=f64(do), **args)
    ra, _ = block.masked_attention(f64(q), f64(k), np.abs(f64(v)), scale, **args)
    ds = score_error(clean(q), clean(k), part, scale)
    within(f64(o), ro, U * np.abs(ro) + (U + 2 * ds + 32 * E) * ra, "o")
    got, none = f64(lse[batches][:, heads]), np.isneginf(rl)
    assert np.array_equal(none, np.isneginf(got))
    within(got[~none], rl[~none], ds + 16 * E * (1 + np.abs(rl[~none])), "lse")
    for name, x, w, b in zip(("dq", "dk", "dv"), (dq, dk, dv), rg, bounds(q, k, v, do, part)):
        within(f64(x), w, U * np.abs(w) + b + 1e-30, name)


@pytest.mark.parametrize("name", TWO_TILES)
def test_two_query_tiles(name):
    b, nq, nk, hq, hk, d, letters = TWO_TILES[name]
    q, k, v = inputs(b, nq, nk, hq, hk, d, seed=len(name))
    check_heads(q, k, v, rule_of(b, nq, nk, hq, letters, seed=nq), sorted({0, hk // 2, hk - 1}), sorted({0, b - 1}))


@pytest.mark.parametrize("name", HEAD_BY_HEAD)
def test_head_by_head(name):
    b, nq, nk, hq, hk, d, letters = HEAD_BY_HEAD[name]
    q, k, v = inputs(b, nq, nk, hq, hk, d, seed=len(name))
    check_heads(q, k, v, rule_of(b, nq, nk, hq, letters), [0, hk - 1], [0])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_unseen_places_may_hold_anything(value, d, cap):
    # padding keys and queries between documents, and a document of keys that no query has
    q, k, v = inputs(1, 390, 390, 52, 26, d, seed=4)
    doc = documents(1, 390, seed=5)
    dk = doc.clone()
    dk[0, 130:140] = 4
    doc[doc == 4] = 5
    rule = pa.ScoreRule(softcap=cap, doc_q=doc, doc_k=dk)
    want, wl = pa.masked_attention(q, k, v, rule, want_lse=True)
    unseen = (dk < 0) | (dk == 4)
    q[doc < 0], k[unseen], v[unseen] = value, value, value
    got, gl = pa.masked_attention(q, k, v, rule, want_lse=True)
    assert torch.equal(want, got) and torch.equal(wl, gl)


def test_repeated_bits_side_stream_and_graphs():
    b, nq, nk, hq, hk, d, letters = TWO_TILES["cap_bias_prefix_documents"]
    q, k, v = inputs(b, nq, nk, hq, hk, d, seed=12)
    rule = rule_of(b, nq, nk, hq, letters)
    run = lambda **kw: pa.masked_attention(q, k, v, rule, want_lse=True, **kw)  # noqa: E731
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [run(), run(stream=side), run()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got.append(run())
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))
