"""The fp64 oracle of the block operators: gradients against central differences, and closed forms."""
import numpy as np
import pytest

from oracle import block

H = 1e-5
# central differences in float64: truncation h^2 = 1e-10 times a third derivative of order 10,
# rounding 1e-16 / h = 1e-11 times values of order 10
TOL = 1e-7


def _directional(f, x, rng):
    """(sum of f's central differences along a random direction, the direction)."""
    v = rng.standard_normal(x.shape)
    return (f(x + H * v) - f(x - H * v)) / (2 * H), v


@pytest.mark.parametrize("grouped", [False, True])
def test_layernorm_gradients(grouped):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 5, 12)) + 0.5, rng.standard_normal((3, 5, 12))
    shape = (3, 12) if grouped else (12,)
    w, b = rng.standard_normal(shape), rng.standard_normal(shape)
    dx, dw, db = block.layernorm_backward(dy, x, w, 1.0, grouped=grouped)
    loss = lambda x, w, b: float((block.layernorm(x, w, b, 1.0)[0] * dy).sum())  # noqa: E731
    for at, grad in ((x, dx), (w, dw), (b, db)):
        f = {id(x): lambda a: loss(a, w, b), id(w): lambda a: loss(x, a, b), id(b): lambda a: loss(x, w, a)}[id(at)]
        d, v = _directional(f, at, rng)
        assert abs(d - (grad * v).sum()) <= TOL * (1 + np.abs(grad * v).sum())


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("eps", [None, 1e-6])
def test_norm_rope_gradients(interleaved, eps):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 3, 2, 16)), rng.standard_normal((2, 3, 2, 16))
    pos, dims, theta = rng.uniform(-9, 9, (3, 2)), (4, 8), (100.0, 10000.0)
    gain = 1 + rng.standard_normal(16) if eps else None
    dx, dg = block.norm_rope_backward(dy, x, pos, dims, theta, interleaved, gain, eps)
    f = lambda a, g: float((block.norm_rope(a, pos, dims, theta, interleaved, g, eps) * dy).sum())  # noqa: E731
    d, v = _directional(lambda a: f(a, gain), x, rng)
    assert abs(d - (dx * v).sum()) <= TOL * (1 + np.abs(dx * v).sum())
    if eps:
        d, v = _directional(lambda g: f(x, g), gain, rng)
        assert abs(d - (dg * v).sum()) <= TOL * (1 + np.abs(dg * v).sum())


def test_rotation_is_orthogonal_and_relative():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 1, 24)), rng.standard_normal((1, 1, 1, 24))
    rot = lambda z, p: block.rotate(z, [[p, 2 * p]], (8, 12), (50.0, 10000.0), False)  # noqa: E731
    assert np.allclose(np.linalg.norm(rot(q, 3.7)), np.linalg.norm(q), rtol=1e-14)
    assert np.allclose(rot(q, 3.7)[..., 20:], q[..., 20:])
    a, b = (rot(q, 5.0) * rot(k, 2.0)).sum(), (rot(q, 105.0) * rot(k, 102.0)).sum()
    assert abs(a - b) <= 1e-10


@pytest.mark.parametrize("kw", [
    dict(), dict(causal=True), dict(causal=True, prefix=[3, 0]), dict(softcap=2.0),
    dict(slopes=[0.5, 0.25, 0.1, 0.0]),
    dict(softcap=3.0, slopes=[0.5, 0.25, 0.1, 0.0], causal=True, prefix=[1, 5]),
    dict(docs=True), dict(docs=True, causal=True, softcap=4.0),
])
def test_masked_attention_gradients(kw):
    rng = np.random.default_rng(4)
    kw = dict(kw)
    nq, nk = 6, 7
    if kw.pop("docs", False):
        kw["doc_q"] = [[0, 0, 1, -1, 2, 5], [3, 1, 1, 1, 1, -1]]
        kw["doc_k"] = [[0, 1, 1, 0, -1, 2, 2], [1, 1, -1, 4, 1, 1, -1]]
    q, k, v = (rng.standard_normal(s) for s in ((2, nq, 4, 5), (2, nk, 2, 5), (2, nk, 2, 5)))
    do = rng.standard_normal(q.shape)
    o, lse, dq, dk, dv = block.masked_attention(q, k, v, 0.6, do=do, **kw)
    f = lambda q, k, v: float((block.masked_attention(q, k, v, 0.6, **kw)[0] * do).sum())  # noqa: E731
    for fn, at, grad in ((lambda a: f(a, k, v), q, dq), (lambda a: f(q, a, v), k, dk), (lambda a: f(q, k, a), v, dv)):
        d, w = _directional(fn, at, rng)
        assert abs(d - (grad * w).sum()) <= TOL * (1 + np.abs(grad * w).sum())


def test_masked_attention_closed_forms():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((1, 3, 1, 4)), rng.standard_normal((1, 5, 1, 4)), rng.standard_normal((1, 5, 1, 4))
    # no mask: ordinary softmax attention
    s = 0.5 * q[0, :, 0] @ k[0, :, 0].T
    p = np.exp(s) / np.exp(s).sum(1, keepdims=True)
    o, lse = block.masked_attention(q, k, v, 0.5)
    assert np.allclose(o[0, :, 0], p @ v[0, :, 0]) and np.allclose(lse[0, 0], np.log(np.exp(s).sum(1)))
    # a query alone with one key of its document copies that key's value; without any key it gives zero
    o, lse = block.masked_attention(q, k, v, 0.5, doc_q=[[7, 9, -1]], doc_k=[[1, 7, -1, -1, 2]])
    assert np.allclose(o[0, 0, 0], v[0, 1, 0]) and not o[0, 1:].any() and np.isneginf(lse[0, 0, 1:]).all()
    # causal with fewer queries than keys: the queries are the last positions
    assert block.visible(2, 5, causal=True).tolist() == [[True] * 4 + [False], [True] * 5]
    assert block.visible(3, 2, causal=True).sum(1).tolist() == [0, 1, 2]
