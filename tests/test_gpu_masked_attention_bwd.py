"""Gradients of masked attention against the fp64 oracle.

Tolerances (u, e and the score error ds as in the forward tests).
  p recomputed from lse is off by a relative r = 2 ds + 64 e (score, lse, exponential); do.v by dd = (2 d + 4) e |do| |v|;
  delta by u sum |o do| (o is bf16) + dd; the cap's 1 - tanh^2 by 16 e.  ds rounds to bf16 once:
    |err ds| <= u |ds| + p ((r + 16 e) (|do.v| + |delta|) + 2 dd + u sum |o do|)
  dq, dk: u |g| + scale sum |err ds| |k or q|, and the fp32 sums 2 n e of the same terms' sizes, n of them
  dv:     u |dv| + sum (u + r) p |do|, and the same for its sums
"""
import numpy as np
import pytest
import torch

import patch_attention_b200 as pa
from oracle import block
from tests._bounds import within
from tests._oracle_util import f64
from tests.test_gpu_masked_attention import BF, E, U, clean, documents, inputs, oracle_args, score_error, slopes

pytestmark = pytest.mark.gpu


def bounds(q, k, v, do, rule):
    """(dq, dk, dv) error bounds from the formulas above."""
    scale, a = oracle_args(rule, q.shape[-1])
    ds_err = score_error(clean(q), clean(k), rule, scale)
    r = 2 * ds_err + 64 * E
    Q, K, V, DO = (f64(clean(t)) for t in (q, k, v, do))
    B, nq, H, d = Q.shape
    nk, hk = K.shape[1], K.shape[2]
    bq, bk, bv = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V)
    dist = np.abs(np.arange(nq)[:, None] + (nk - nq) - np.arange(nk)[None])
    for b in range(B):
        ok = block.visible(nq, nk, a["causal"], None if a["prefix"] is None else int(a["prefix"][b]),
                           None if a["doc_q"] is None else a["doc_q"][b], None if a["doc_k"] is None else a["doc_k"][b])
        for h in range(H):
            g = h * hk // H
            s = scale * (Q[b, :, h] @ K[b, :, g].T)
            t = np.tanh(s / a["softcap"]) if a["softcap"] else np.zeros_like(s)
            s = a["softcap"] * t if a["softcap"] else s
            if a["slopes"] is not None:
                s = s - float(a["slopes"][h]) * dist
            s = np.where(ok, s, -np.inf)
            m = np.where(ok.any(1), s.max(1, initial=-np.inf), 0.0)
            p = np.exp(s - m[:, None])
            p /= np.where(ok.any(1), p.sum(1), 1.0)[:, None]
            o = p @ V[b, :, g]
            dp = DO[b, :, h] @ V[b, :, g].T
            delta = (o * DO[b, :, h]).sum(1, keepdims=True)
            od = np.abs(o * DO[b, :, h]).sum(1, keepdims=True)
            dd = (2 * d + 4) * E * np.sqrt((DO[b, :, h] ** 2).sum(1)[:, None] * (V[b, :, g] ** 2).sum(1)[None])
            ds = np.abs(p * (dp - delta) * (1 - t * t))
            err = U * ds + p * ((r + 16 * E) * (np.abs(dp) + np.abs(delta)) + 2 * dd + U * od)
            bq[b, :, h] += scale * ((err + 2 * nk * E * ds) @ np.abs(K[b, :, g]))
            bk[b, :, g] += scale * ((err + 2 * nq * H * E * ds).T @ np.abs(Q[b, :, h]))
            bv[b, :, g] += ((U + r + 2 * nq * H * E) * p).T @ np.abs(DO[b, :, h])
    return bq, bk, bv


def check(q, k, v, rule=None, seed=100, **kw):
    rule = rule or pa.ScoreRule()
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(q.shape, device="cuda", generator=g).to(BF)
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True)
    got = pa.masked_attention_backward(do, q, k, v, o, lse, rule, **kw)
    torch.cuda.synchronize()
    pa.pf_device_status()
    scale, args = oracle_args(rule, q.shape[-1])
    want = block.masked_attention(f64(q), f64(k), f64(v), scale, do=f64(do), **args)[2:]
    for name, x, w, b in zip(("dq", "dk", "dv"), got, want, bounds(q, k, v, do, rule)):
        within(f64(x), w, U * np.abs(w) + b + 1e-30, name)
    return do, o, lse, got


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 65), (2, 3), (64, 64), (127, 200), (128, 128), (129, 300), (257, 257), (384, 640)])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_sizes(nq, nk, d):
    check(*inputs(2, nq, nk, 2, 2, d, seed=nq + nk))


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 500), (100, 100), (129, 130), (300, 300), (300, 17), (260, 500)])
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("prefix", [False, True])
def test_causal_and_prefix(nq, nk, d, prefix):
    q, k, v = inputs(3, nq, nk, 2, 1, d, seed=nq)
    p = torch.tensor([0, nk // 2 + 1, nk + 5], device="cuda", dtype=torch.int32) if prefix else None
    check(q, k, v, pa.ScoreRule(causal=True, prefix=p))


@pytest.mark.parametrize("b,hq,hk,nq,nk", [(1, 3, 1, 200, 200), (2, 8, 2, 130, 140), (1, 6, 2, 300, 333), (1, 130, 1, 1, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_heads(b, hq, hk, nq, nk, d):
    check(*inputs(b, nq, nk, hq, hk, d, seed=hq), pa.ScoreRule(causal=True))


@pytest.mark.parametrize("cap", [0.0, 5.0, 50.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("nq,nk", [(250, 250), (140, 300)])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_cap_and_bias(cap, bias, nq, nk, d):
    q, k, v = inputs(1, nq, nk, 4, 2, d, seed=3, scale=3.0)
    check(q, k, v, pa.ScoreRule(softcap=cap, slopes=slopes(4) if bias else None))
    check(q, k, v, pa.ScoreRule(softcap=cap, slopes=slopes(4) if bias else None, causal=True, softmax_scale=0.2))


@pytest.mark.parametrize("n", [5, 128, 300, 515])
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_documents(n, d, causal):
    q, k, v = inputs(2, n, n, 2, 2, d, seed=n)
    doc = documents(2, n, seed=n)
    check(q, k, v, pa.ScoreRule(causal=causal, doc_q=doc, doc_k=doc))


def test_everything_at_once():
    q, k, v = inputs(2, 300, 520, 6, 2, 64, seed=8)
    check(q, k, v, pa.ScoreRule(softcap=20.0, slopes=slopes(6), causal=True,
                                prefix=torch.tensor([100, 400], device="cuda", dtype=torch.int32),
                                doc_q=documents(2, 300, 1), doc_k=documents(2, 520, 2)))


def test_no_keys_no_queries():
    for nq, nk in ((5, 0), (0, 5)):
        q, k, v = inputs(2, nq, nk, 2, 2, 64)
        o, lse = pa.masked_attention(q, k, v, want_lse=True)
        dq, dk, dv = pa.masked_attention_backward(torch.ones_like(o), q, k, v, o, lse)
        assert not dq.any() and not dk.any() and not dv.any() and dk.shape == k.shape
    doc = torch.full((2, 200), -1, device="cuda", dtype=torch.int32)
    q, k, v = inputs(2, 200, 200, 2, 2, 64)
    _, _, _, got = check(q, k, v, pa.ScoreRule(doc_q=doc, doc_k=doc))
    assert not any(g.any() for g in got)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_unseen_places_may_hold_anything(value, d):
    q, k, v = inputs(1, 300, 300, 2, 1, d, seed=4)
    doc = documents(1, 300, seed=5)
    dk_ = doc.clone()
    dk_[0, 130:140] = 4
    doc[doc == 4] = 5
    rule = pa.ScoreRule(doc_q=doc, doc_k=dk_, causal=True)
    do, o, lse, want = check(q, k, v, rule)
    unseen_k, unseen_q = (dk_ < 0) | (dk_ == 4), torch.isneginf(lse[:, 0])
    assert unseen_q.any() and unseen_k.any()
    for t, where in ((q, unseen_q), (do, unseen_q), (o, unseen_q), (k, unseen_k), (v, unseen_k)):
        t[where] = value
    got = pa.masked_attention_backward(do, q, k, v, o, lse, rule)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not got[0][unseen_q].any() and not got[1][unseen_k].any() and not got[2][unseen_k].any()


def test_strided_views_and_guards():
    qkv = torch.randn(2, 150, 3, 4, 72, device="cuda").to(BF)
    q, k, v = qkv.unbind(2)
    rule = pa.ScoreRule(causal=True)
    do, o, lse, want = check(q.contiguous(), k.contiguous(), v.contiguous(), rule)
    got = pa.masked_attention_backward(do, q, k, v, o, lse, rule)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    n = q.numel()
    bufs = [torch.full((n + 4096,), 7.0, device="cuda", dtype=BF) for _ in range(3)]
    ws = torch.full((2 * 150 * 4 * 4 + 256,), 7, device="cuda", dtype=torch.uint8)
    outs = [b[:n].view(2, 150, 4, 72) for b in bufs]
    pa.pf_masked_attn_bwd(do, q, k, v, o, lse, *outs, ws[:2 * 150 * 4 * 4], rule)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all((b[n:] == 7.0).all() for b in bufs) and (ws[2 * 150 * 4 * 4:] == 7).all()


def test_repeated_bits_side_stream_and_graphs():
    q, k, v = inputs(2, 300, 400, 4, 2, 64, seed=12)
    rule = pa.ScoreRule(doc_q=documents(2, 300, 3), doc_k=documents(2, 400, 4), softcap=10.0)
    do = torch.randn_like(q)

    def both(**kw):
        o, lse = pa.masked_attention(q, k, v, rule, want_lse=True, **kw)
        return (o,) + pa.masked_attention_backward(do, q, k, v, o, lse, rule, **kw)

    want = both()
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))  # noqa: E731
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


def test_gradients_against_differences():
    # the loss sum(o do) along random directions: differences of the 64-bit forward
    rng = np.random.default_rng(13)
    q, k, v = inputs(1, 70, 90, 2, 1, 64, seed=13)
    rule = pa.ScoreRule(softcap=4.0, slopes=slopes(2), causal=True)
    do, _, _, got = check(q, k, v, rule)
    scale, args = oracle_args(rule, 64)
    base = [f64(t) for t in (q, k, v)]
    f = lambda x: (block.masked_attention(*x, scale, **args)[0] * f64(do)).sum()  # noqa: E731
    for at, (grad, bound) in enumerate(zip(got, bounds(q, k, v, do, rule))):
        w = rng.standard_normal(grad.shape)
        h = 1e-5
        x0, x1 = list(base), list(base)
        x0[at], x1[at] = base[at] - h * w, base[at] + h * w
        d = (f(x1) - f(x0)) / (2 * h)
        G = f64(grad)
        assert abs(d - (G * w).sum()) <= ((U * np.abs(G) + bound) * np.abs(w)).sum() + 1e-6 * np.abs(G * w).sum()
