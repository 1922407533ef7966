"""QK norm + rotary embedding, forward and backward, against the fp64 oracle.

Tolerances.  u is half a step of the type, e = 2^-24.
  forward: the mean square has at most 8 terms per lane and 5 tree levels (13 e, half of it in the root), rsqrtf
      2 e, gain and angle products 3 e, cosine and sine 2 e absolute each, their angle 2 pi 2^-25 (the fraction of
      a turn rounded to 32 bits) = 3.2 e: |error| <= u |y| + 24 e (|z0| + |z1|) for the pair's normalised elements.
  dx: the same over the turned gradient, and the mean of a x^ (13 e of the mean size):
      u |dx| + 40 e r (|a0| + |a1| + |x^| mean|a x^|), with a over the pair.
  dgain: chains of at most 512 additions: u |dg| + 600 e sum(|dz0| + |dz1|) |x^|.
"""
import numpy as np
import pytest
import torch

import patch_attention_b200 as pa
from oracle import block
from tests._oracle_util import f64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def _partner(z, dims, interleaved):
    """|z0| + |z1| of every element's pair (the element alone past the axes)."""
    out = np.abs(z).copy()
    for e, f, _, _ in block.rope_pairs(z.shape[-1], dims, interleaved):
        out[..., e] = out[..., f] = np.abs(z[..., e]) + np.abs(z[..., f])
    return out


def _inputs(b, n, hq, hk, d, dtype, na, seed=0, far=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    t = lambda h: r(b, n, h, d).to(dtype) if h else None  # noqa: E731
    pos = (torch.randint(0, 500, (n, na), device="cuda", generator=g) * far).float()
    gains = [(1 + 0.3 * r(d)).to(dtype) if h else None for h in (hq, hk)]
    return t(hq), t(hk), t(hq), t(hk), pos, gains


def _check(q, k, dq, dk, pos, axes, gq, gk, eps):
    out = pa.qk_norm_rope(q, k, pos, axes, gain_q=gq, gain_k=gk, eps=eps)
    grads = pa.qk_norm_rope_backward(dq, dk, q if eps else None, k if eps else None, pos, axes, gain_q=gq, gain_k=gk,
                                     eps=eps)
    P = f64(pos)
    for x, y, dy, dx, gain, dg in ((q, out[0], dq, grads[0], gq, grads[2]), (k, out[1], dk, grads[1], gk, grads[3])):
        if x is None:
            assert y is None and dx is None and dg is None
            continue
        X, DY, G = f64(x), f64(dy), None if gain is None else f64(gain)
        u = torch.finfo(x.dtype).eps / 2
        tiny = float(torch.finfo(x.dtype).smallest_normal) * u * 2
        ref = block.norm_rope(X, P, axes.dims, axes.theta, axes.interleaved, G, eps)
        z = block.norm_rope(X, P * 0, axes.dims, axes.theta, axes.interleaved, G, eps)
        assert np.all(np.abs(f64(y) - ref) <= u * np.abs(ref) + 24 * E * _partner(z, axes.dims, axes.interleaved) + tiny)
        rdx, rdg = block.norm_rope_backward(DY, X, P, axes.dims, axes.theta, axes.interleaved, G, eps)
        dz = _partner(block.rotate(DY, P, axes.dims, axes.theta, axes.interleaved, -1.0), axes.dims, axes.interleaved)
        if eps is None:
            assert np.all(np.abs(f64(dx) - rdx) <= u * np.abs(rdx) + 24 * E * dz + tiny)
            continue
        r = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
        a = dz if G is None else dz * np.abs(G).max()
        size = r * (a + np.abs(X * r) * (a * np.abs(X * r)).mean(-1, keepdims=True))
        assert np.all(np.abs(f64(dx) - rdx) <= u * np.abs(rdx) + 40 * E * size + tiny)
        if gain is not None:
            size = (dz * np.abs(X * r)).sum((0, 1, 2))
            assert np.all(np.abs(f64(dg) - rdg) <= u * np.abs(rdg) + 600 * E * size + tiny)
    return out, grads


# head_dim, sections; half-split sections with halves that are multiples of 4, of 2 and odd
@pytest.mark.parametrize("d,dims", [(8, (8,)), (8, (2,)), (24, (6, 10)), (64, (16, 24, 24)), (72, (36, 36)),
                                    (72, (64,)), (128, (16, 56, 56)), (128, (44, 42, 42)), (128, (128,)),
                                    (256, (64, 64, 64, 64)), (200, (40, 80, 80))])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_sections_and_types(d, dims, interleaved, dtype):
    axes = pa.RopeAxes(dims, theta=10000.0, interleaved=interleaved)
    q, k, dq, dk, pos, (gq, gk) = _inputs(2, 5, 3, 1, d, dtype, len(dims), seed=d)
    _check(q, k, dq, dk, pos, axes, gq, gk, 1e-6)
    _check(q, k, dq, dk, pos, axes, None, None, None)


@pytest.mark.parametrize("b,n,hq,hk", [(1, 1, 1, 0), (1, 1, 0, 1), (2, 1, 24, 24), (1, 3, 24, 8), (3, 130, 5, 2),
                                       (1, 2500, 2, 2), (1, 4097, 1, 1)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_tokens_and_heads(b, n, hq, hk, interleaved):
    axes = pa.RopeAxes((16, 24, 24), interleaved=interleaved)
    q, k, dq, dk, pos, (gq, gk) = _inputs(b, n, hq, hk, 64, BF, 3, seed=n)
    _check(q, k, dq, dk, pos, axes, gq, gk, 1e-6)


def test_norm_without_gains_and_one_gain():
    axes = pa.RopeAxes((32, 32))
    q, k, dq, dk, pos, (gq, gk) = _inputs(2, 9, 4, 2, 64, BF, 2, seed=1)
    _check(q, k, dq, dk, pos, axes, None, None, 1e-6)
    _check(q, k, dq, dk, pos, axes, gq, None, 1e-6)


@pytest.mark.parametrize("far", [1000.0, 30000.25, -70000.5])
def test_far_and_fractional_positions(far):
    axes = pa.RopeAxes((16, 24, 24), theta=(10000.0, 500.0, 1e6), interleaved=False)
    q, k, dq, dk, pos, (gq, gk) = _inputs(1, 33, 2, 2, 64, FF, 3, seed=2, far=far)
    _check(q, k, dq, dk, pos, axes, gq, gk, 1e-6)


def test_positions_per_batch_element():
    axes = pa.RopeAxes((32, 32))
    q, k, dq, dk, _, (gq, gk) = _inputs(3, 7, 2, 2, 64, BF, 2, seed=3)
    pos = torch.randint(0, 99, (3, 7, 2), device="cuda").float()
    out, _ = _check(q, k, dq, dk, pos, axes, gq, gk, 1e-6)
    one = pa.qk_norm_rope(q[1:2], k[1:2], pos[1], axes, gain_q=gq, gain_k=gk, eps=1e-6)
    assert torch.equal(out[0][1:2], one[0]) and torch.equal(out[1][1:2], one[1])


def test_norm_agrees_with_the_separate_norm():
    # position 0 turns nothing: the norm alone, within one rounding of pf_qk_rmsnorm's own
    q, k, _, _, pos, (gq, gk) = _inputs(1, 50, 4, 4, 128, BF, 1, seed=4)
    y, _ = pa.qk_norm_rope(q, k, pos * 0, pa.RopeAxes((128,)), gain_q=gq, gain_k=gk, eps=1e-6)
    x = q.clone()
    pa.pf_qk_rmsnorm(x, gq, 1e-6)
    assert ((x.float() - y.float()).abs() <= 2.0 ** -7 * x.float().abs()).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_packed_projection_in_place_and_transposed(interleaved):
    axes = pa.RopeAxes((16, 24, 24), interleaved=interleaved)
    qkv = torch.randn(2, 37, 3, 6, 64, device="cuda").to(BF)
    pos = torch.randint(0, 64, (37, 3), device="cuda").float()
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    want = pa.qk_norm_rope(q.contiguous(), k.contiguous(), pos, axes, eps=1e-6)
    got = pa.qk_norm_rope(q, k, pos, axes, eps=1e-6)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # [batch, heads, tokens, head_dim] storage
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(pa.qk_norm_rope(qt, None, pos, axes, eps=1e-6)[0], want[0])
    # gradients through strided views
    d = torch.randn_like(qkv)
    gw = pa.qk_norm_rope_backward(d[:, :, 0].contiguous(), d[:, :, 1].contiguous(), q, k, pos, axes, eps=1e-6)
    gs = pa.qk_norm_rope_backward(d[:, :, 0], d[:, :, 1], q, k, pos, axes, eps=1e-6)
    assert torch.equal(gw[0], gs[0]) and torch.equal(gw[1], gs[1])
    # in place, values untouched
    v = qkv[:, :, 2].clone()
    pa.pf_qk_norm_rope(q, k, pos, axes, q, k, eps=1e-6)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 2], v)


def test_unturned_tail_is_copied_bit_for_bit():
    q = torch.randn(1, 4, 2, 72, device="cuda").to(BF)
    q[0, 1, 0, 66] = float("inf")
    pos = torch.randint(1, 9, (4, 1), device="cuda").float()
    for inter in (True, False):
        y, _ = pa.qk_norm_rope(q, None, pos, pa.RopeAxes((64,), interleaved=inter))
        assert torch.equal(y[..., 64:].view(torch.int16), q[..., 64:].view(torch.int16))


def test_no_tokens():
    axes = pa.RopeAxes((32, 32))
    for shape in ((2, 0, 3, 64), (0, 5, 3, 64)):
        q = torch.empty(shape, device="cuda", dtype=BF)
        pos = torch.zeros(shape[1], 2, device="cuda")
        gain = torch.ones(64, device="cuda", dtype=BF)
        y, _ = pa.qk_norm_rope(q, None, pos, axes, gain_q=gain, eps=1e-6)
        dq, _, dg, _ = pa.qk_norm_rope_backward(q, None, q, None, pos, axes, gain_q=gain, eps=1e-6)
        assert y.shape == q.shape and dq.shape == q.shape and not dg.any()


def test_repeated_bits_side_stream_and_graph():
    axes = pa.RopeAxes((16, 56, 56))
    q, k, dq, dk, pos, (gq, gk) = _inputs(1, 700, 24, 8, 128, BF, 3, seed=5)

    def both(**kw):
        out = pa.qk_norm_rope(q, k, pos, axes, gain_q=gq, gain_k=gk, eps=1e-6, **kw)
        return out + pa.qk_norm_rope_backward(dq, dk, q, k, pos, axes, gain_q=gq, gain_k=gk, eps=1e-6, **kw)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("interleaved", [True, False])
def test_gradient_against_differences(interleaved):
    rng = np.random.default_rng(6)
    axes = pa.RopeAxes((16, 24), theta=100.0, interleaved=interleaved)
    q, _, dq, _, pos, (gq, _) = _inputs(1, 6, 2, 0, 48, FF, 2, seed=6)
    dx, _, dg, _ = pa.qk_norm_rope_backward(dq, None, q, None, pos, axes, gain_q=gq, eps=1e-6)
    X, DY, P, G = f64(q), f64(dq), f64(pos), f64(gq)
    f = lambda x, g: (block.norm_rope(x, P, axes.dims, axes.theta, interleaved, g, 1e-6) * DY).sum()  # noqa: E731
    h = 1e-5
    for grad, at in ((dx, lambda v: f(X + h * v, G) - f(X - h * v, G)), (dg, lambda v: f(X, G + h * v) - f(X, G - h * v))):
        v = rng.standard_normal(grad.shape)
        # the gradient's own error (at most 600 e = 3.6e-5 of its terms' sizes) and 1e-7 of the differences
        assert abs(at(v) / (2 * h) - (f64(grad) * v).sum()) <= 4e-5 * (np.abs(f64(grad) * v).sum() + 1)
