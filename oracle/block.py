"""Operators of the transformer block around the patch attention, fp64: layer norm, QK norm with
a rotary embedding over several position axes, attention over masked scores, and their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Every gradient is written from its formula and pinned against central differences of the
forward function in ``tests/test_oracle_block.py``.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


# ------------------------------------------------------------------ layer norm


def layernorm(x, weight=None, bias=None, weight_offset=0.0, eps=1e-6):
    """x: [..., C]; weight, bias: [C] or [x.shape[0], C].  Returns (y, mean, rstd)."""
    x, w, b = _f(x), _f(weight), _f(bias)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * (_per_row(w, x) + weight_offset)
    if b is not None:
        y = y + _per_row(b, x)
    return y, mean, rstd


def _per_row(p, x):
    """[C] or [G, C] parameters shaped to broadcast over x [G, ..., C]."""
    return p if p.ndim == 1 else p.reshape((p.shape[0],) + (1,) * (x.ndim - 2) + (p.shape[-1],))


def layernorm_backward(dy, x, weight=None, weight_offset=0.0, eps=1e-6, grouped=False):
    """(dx, dweight, dbias); the sums are [x.shape[0], C] if grouped, else [C]."""
    dy, x, w = _f(dy), _f(x), _f(weight)
    xh, _, rstd = layernorm(x, eps=eps)
    a = dy if w is None else dy * (_per_row(w, x) + weight_offset)
    dx = rstd[..., None] * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    over = tuple(range(1 if grouped else 0, x.ndim - 1))
    return dx, (dy * xh).sum(over), dy.sum(over)


# ------------------------------------------------------------------ QK norm + rotary


def rope_pairs(head_dim, dims, interleaved):
    """[(first element, second element, axis, exponent 2i/w)] of the rotated pairs."""
    out, base = [], 0
    for a, w in enumerate(dims):
        for i in range(w // 2):
            first = base + (2 * i if interleaved else i)
            out.append((first, first + (1 if interleaved else w // 2), a, 2.0 * i / w))
        base += w
    assert base <= head_dim
    return out


def rotate(z, pos, dims, theta, interleaved, sign=1.0):
    """z: [B, N, H, d]; pos: [N, axes] or [B, N, axes]; sign -1 turns back."""
    z, pos = _f(z), _f(pos)
    pos = pos if pos.ndim == 3 else pos[None]
    y = z.copy()
    for e, f, a, ex in rope_pairs(z.shape[-1], dims, interleaved):
        phi = (sign * pos[..., a] * theta[a] ** -ex)[..., None]
        y[..., e] = z[..., e] * np.cos(phi) - z[..., f] * np.sin(phi)
        y[..., f] = z[..., e] * np.sin(phi) + z[..., f] * np.cos(phi)
    return y


def norm_rope(x, pos, dims, theta, interleaved, gain=None, eps=None):
    x = _f(x)
    z = x
    if eps is not None:
        z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if gain is not None:
            z = z * _f(gain)
    return rotate(z, pos, dims, theta, interleaved)


def norm_rope_backward(dy, x, pos, dims, theta, interleaved, gain=None, eps=None):
    """(dx, dgain); dgain is None without a norm."""
    dz = rotate(dy, pos, dims, theta, interleaved, -1.0)
    if eps is None:
        return dz, None
    x = _f(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    a = dz if gain is None else dz * _f(gain)
    dx = r * (a - xh * (a * xh).mean(-1, keepdims=True))
    return dx, (dz * xh).sum(tuple(range(x.ndim - 1)))


# ------------------------------------------------------------------ attention over masked scores


def visible(n_q, n_k, causal=False, prefix=None, doc_q=None, doc_k=None):
    """[n_q, n_k] truth values of one batch element: query i stands at position i + n_k - n_q."""
    i = np.arange(n_q)[:, None] + (n_k - n_q)
    j = np.arange(n_k)[None]
    ok = np.ones((n_q, n_k), dtype=bool)
    if causal:
        ok = j <= i
        if prefix is not None:
            ok = ok | (j < prefix)
    if doc_q is not None:
        dq, dk = np.asarray(doc_q)[:, None], np.asarray(doc_k)[None]
        ok = ok & (dq == dk) & (dq >= 0)
    return ok


def masked_attention(q, k, v, scale, softcap=0.0, slopes=None, causal=False, prefix=None, doc_q=None, doc_k=None,
                     do=None):
    """q: [B, Nq, H, d]; k, v: [B, Nk, Hkv, d]; slopes [H]; prefix [B]; doc_q [B, Nq], doc_k [B, Nk].
    Returns (o, lse [B, H, Nq]) or, with do, (o, lse, dq, dk, dv).  A query that sees no key gives 0, lse -inf."""
    q, k, v, do = _f(q), _f(k), _f(v), _f(do)
    B, nq, H, d = q.shape
    nk, hk = k.shape[1], k.shape[2]
    o, lse = np.zeros_like(q), np.full((B, H, nq), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dist = np.abs(np.arange(nq)[:, None] + (nk - nq) - np.arange(nk)[None])
    for b in range(B):
        ok = visible(nq, nk, causal, None if prefix is None else int(prefix[b]),
                     None if doc_q is None else doc_q[b], None if doc_k is None else doc_k[b])
        some = ok.any(1)
        seen = ok.any(0)
        for h in range(H):
            g = h * hk // H
            # keys and values that no query sees do not matter, whatever they hold
            kk, vv = np.where(seen[:, None], k[b, :, g], 0.0), np.where(seen[:, None], v[b, :, g], 0.0)
            qq = np.where(some[:, None], q[b, :, h], 0.0)
            s = scale * (qq @ kk.T)
            t = np.zeros_like(s)
            if softcap:
                t = np.tanh(s / softcap)
                s = softcap * t
            if slopes is not None:
                s = s - float(slopes[h]) * dist
            s = np.where(ok, s, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - m[:, None])
            z = e.sum(1)
            p = e / np.where(some, z, 1.0)[:, None]
            o[b, :, h] = p @ vv
            lse[b, h] = np.where(some, m + np.log(np.where(some, z, 1.0)), -np.inf)
            if do is not None:
                dd = np.where(some[:, None], do[b, :, h], 0.0)
                dp = dd @ vv.T
                ds = p * (dp - (p * dp).sum(1, keepdims=True)) * (1 - t * t) * scale
                dq[b, :, h] = ds @ kk
                dk[b, :, g] += ds.T @ qq
                dv[b, :, g] += p.T @ dd
    return (o, lse) if do is None else (o, lse, dq, dk, dv)
