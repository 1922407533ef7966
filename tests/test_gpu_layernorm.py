"""Layer norm, forward and backward, against the fp64 oracle.

Tolerances.  u is half a step of the output type; e = 2^-24 that of fp32, in which everything before the
last rounding is computed.
  y:  |error| <= u |y| + e (64 r |w'| mean|x| + 80 |x^ w'| + 4 |b|).  A lane adds at most 48 terms and a tree of
      at most 9 levels follows, so the mean is off by at most 57 e mean|x| (and x - mean by one e more), the
      variance by about 60 e relative, its root by half of that and rsqrtf by 2 e; three products round.
  dx: |error| <= u |dx| + 256 e r (|a| + mean|a| + |x^| mean|a x^|) (1 + r mean|x|): the same sums over a and a x^,
      with x^ itself off by 64 e (1 + r mean|x|).
  dw, db: fp32 chains of at most 512 additions (a block's rows, then the blocks): 512 e times the sum of the
      terms' sizes, where a term dy x^ also carries x^'s error 64 e |dy| r mean|x|; and u for the last rounding.
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


def _half_step(t):
    return torch.finfo(t).eps / 2


def _inputs(shape, dtype, grouped, wide, seed=0, offset=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    c = shape[-1]
    x = (r(*shape) * (0.5 + r(c).abs()) + offset * r(c)).to(dtype)
    dy = r(*shape).to(dtype)
    p = (0.3 * r(*((shape[0],) if grouped else ()), 3, c)).to(FF if wide else dtype)
    return x, dy, p[..., 1, :], p[..., 0, :]  # views with a row stride of 3 C when grouped


def _check(x, dy, w, b, w0, eps=1e-6):
    """Runs both directions and holds every output against the oracle."""
    grouped = w is not None and w.dim() == 2
    y, mean, rstd = pa.layernorm(x, w, b, weight_offset=w0, eps=eps, want_stats=True)
    assert torch.equal(y, pa.layernorm(x, w, b, weight_offset=w0, eps=eps))
    X, DY, W, B = f64(x), f64(dy), None if w is None else f64(w), None if b is None else f64(b)
    ref, rm, rr = block.layernorm(X, W, B, w0, eps)
    wf = 1.0 if w is None else np.abs(block._per_row(W, X) + w0)
    bf = 0.0 if b is None else np.abs(block._per_row(B, X))
    xh = np.abs(X - rm[..., None]) * rr[..., None]
    ma = np.abs(X).mean(-1, keepdims=True) * rr[..., None]
    u = _half_step(x.dtype)
    tiny = float(torch.finfo(x.dtype).smallest_normal) * u * 2  # spacing of subnormal values
    assert np.all(np.abs(f64(y) - ref) <= u * np.abs(ref) + E * (64 * wf * ma + 80 * xh * wf + 4 * bf) + tiny)
    assert np.all(np.abs(f64(mean) - rm) <= 64 * E * np.abs(X).mean(-1) + 1e-45)
    assert np.all(np.abs(f64(rstd) - rr) <= 64 * E * rr * (1 + ma[..., 0]))

    dx, dw, db = pa.layernorm_backward(dy, x, w, mean, rstd, weight_offset=w0, bias_like=b)
    rdx, rdw, rdb = block.layernorm_backward(DY, X, W, w0, eps, grouped)
    a = np.abs(DY * (1.0 if w is None else block._per_row(W, X) + w0))
    r = rr[..., None]
    size = r * (a + a.mean(-1, keepdims=True) + xh * (a * xh).mean(-1, keepdims=True)) * (1 + ma)
    assert np.all(np.abs(f64(dx) - rdx) <= u * np.abs(rdx) + 256 * E * size + tiny)
    over = tuple(range(1 if grouped else 0, x.dim() - 1))
    if w is not None:
        uw = _half_step(w.dtype)
        size = (np.abs(DY) * (512 * xh + 64 * (ma + xh))).sum(over)
        assert dw.shape == w.shape and dw.dtype == w.dtype
        assert np.all(np.abs(f64(dw) - rdw) <= uw * np.abs(rdw) + E * size + tiny)
    if b is not None:
        ub = _half_step(b.dtype)
        assert db.shape == b.shape and db.dtype == b.dtype
        assert np.all(np.abs(f64(db) - rdb) <= ub * np.abs(rdb) + 512 * E * np.abs(DY).sum(over) + tiny)
    return y, dx, dw, db


# every team width (a warp, 128 and 512 threads), its full and ragged ends, and both access widths
@pytest.mark.parametrize("c", [1, 2, 7, 8, 255, 256, 264, 512, 1000, 1024, 1031, 1536, 1537, 1544, 2048, 4096, 4097,
                               8192, 8200, 16384])
@pytest.mark.parametrize("dtype", [BF, FF])
def test_widths(c, dtype):
    x, dy, w, b = _inputs((5, c), dtype, False, False, seed=c)
    _check(x, dy, w, b, 1.0)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 1184, 1185, 4999])
@pytest.mark.parametrize("dtype,wide", [(BF, False), (BF, True), (HF, False), (HF, True), (FF, False)])
def test_rows_and_types(rows, dtype, wide):
    x, dy, w, b = _inputs((rows, 160), dtype, False, wide, seed=rows)
    _check(x, dy, w, b, 0.0)


@pytest.mark.parametrize("shape", [(1, 1, 64), (3, 1, 64), (4, 77, 136), (2, 600, 1152), (7, 3, 5, 33), (700, 2, 24)])
@pytest.mark.parametrize("dtype,wide", [(BF, False), (HF, True), (FF, False)])
def test_modulation_per_sample(shape, dtype, wide):
    x, dy, w, b = _inputs(shape, dtype, True, wide, seed=9)
    if shape[0] > 1:
        assert not w.is_contiguous()
    _check(x, dy, w, b, 1.0)


def test_parameters_left_out():
    x, dy, w, b = _inputs((9, 136), BF, False, False, seed=3)
    y, _, dw, db = _check(x, dy, None, None, 1.0)  # the offset goes with a weight
    assert dw is None and db is None
    _, _, dw, db = _check(x, dy, None, b, 0.0)
    assert dw is None and db is not None
    _check(x, dy, w, None, 0.0)


def test_rows_off_a_16_byte_boundary():
    # an offset of one element moves every row and parameter off 16 bytes: element accesses
    x, dy, w, b = _inputs((6, 160), BF, False, False, seed=4)
    shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    y0, y1 = pa.layernorm(x, w, b), pa.layernorm(shift(x), shift(w), shift(b))
    assert shift(x).data_ptr() % 16 and (y0.float() - y1.float()).abs().max() <= 2 ** -7 * y0.float().abs().max()
    _check(shift(x), shift(dy), shift(w), shift(b), 0.0)


def test_far_mean_and_constant_rows():
    # 32 bits around the mean: a row 1000 deviations away keeps its variance
    x = (torch.randn(4, 512, device="cuda") + 1000).to(FF)
    _check(x, torch.randn_like(x), None, None, 0.0)
    # a constant row: variance 0, so x^ = 0 (eps in the root) and y = b
    x = torch.full((3, 256), 2.5, device="cuda", dtype=BF)
    b = torch.randn(256, device="cuda").to(BF)
    assert torch.equal(pa.layernorm(x, None, b), b.expand(3, -1))


def test_nonfinite_rows_stay_in_their_rows():
    x, dy, w, b = _inputs((8, 256), BF, False, False, seed=6)
    bad = x.clone()
    bad[3, 17], bad[5, 0] = float("nan"), float("inf")
    y0, y1 = pa.layernorm(x, w, b), pa.layernorm(bad, w, b)
    keep = [0, 1, 2, 4, 6, 7]
    assert torch.equal(y0[keep], y1[keep]) and y1[3].isnan().all() and y1[5].isnan().any()


def test_empty_rows():
    w = torch.ones(64, device="cuda", dtype=BF)
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    y, mean, rstd = pa.layernorm(x, w, w, want_stats=True)
    assert y.shape == x.shape and mean.numel() == 0
    dx, dw, db = pa.layernorm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    x = torch.empty(3, 0, 64, device="cuda", dtype=BF)
    g = torch.ones(3, 64, device="cuda", dtype=BF)
    _, mean, rstd = pa.layernorm(x, g, g, want_stats=True)
    _, dw, db = pa.layernorm_backward(x, x, g, mean, rstd)
    assert dw.shape == (3, 64) and not dw.any() and not db.any()


def test_in_place_and_repeated_bits():
    x, dy, w, b = _inputs((700, 1152), BF, False, False, seed=7)
    y, mean, rstd = pa.layernorm(x, w, b, want_stats=True)
    first = pa.layernorm_backward(dy, x, w, mean, rstd)
    again = pa.layernorm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    buf = x.clone()
    pa.pf_layernorm(buf, buf, w, b)
    assert torch.equal(buf, y)
    for over in (dy.clone(), x.clone()):  # dx over dy, dx over x
        d_, x_ = (over, x) if torch.equal(over, dy) else (dy, over)
        ws = torch.empty(pa.pf_layernorm_bwd_workspace_bytes(1, 700, 1152), dtype=torch.uint8, device="cuda")
        dw, db = torch.empty_like(w), torch.empty_like(w)
        pa.pf_layernorm_bwd(d_, x_, w, 0.0, mean, rstd, over, dw, db, ws)
        assert torch.equal(over, first[0]) and torch.equal(dw, first[1]) and torch.equal(db, first[2])


def test_rows_past_the_end_are_left_alone():
    x, dy, w, b = _inputs((33, 96), BF, False, False, seed=8)
    guard = torch.full((40, 96), 7.0, device="cuda", dtype=BF)
    pa.pf_layernorm(x, guard[:33], w, b)
    assert (guard[33:] == 7.0).all()


def test_side_stream_and_graph():
    x, dy, w, b = _inputs((300, 1152), BF, False, False, seed=10)
    y, mean, rstd = pa.layernorm(x, w, b, want_stats=True)
    want = (y,) + pa.layernorm_backward(dy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, m2, r2 = pa.layernorm(x, w, b, want_stats=True, stream=side)
    got = (y2,) + pa.layernorm_backward(dy, x, w, m2, r2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    xs = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y3, m3, r3 = pa.layernorm(xs, w, b, want_stats=True)
        got = (y3,) + pa.layernorm_backward(dy, xs, w, m3, r3)
    xs.copy_(x)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_gradient_against_differences():
    # the loss sum(y dy) along a random direction: differences of the 64-bit forward
    rng = np.random.default_rng(11)
    x, dy, w, b = _inputs((6, 64), FF, False, False, seed=11)
    _, mean, rstd = pa.layernorm(x, w, b, want_stats=True)
    dx, dw, db = pa.layernorm_backward(dy, x, w, mean, rstd)
    X, DY, W, B = (f64(t) for t in (x, dy, w, b))
    h = 1e-5
    for grad, f in ((dx, lambda v: block.layernorm(X + h * v, W, B)[0] - block.layernorm(X - h * v, W, B)[0]),
                    (dw, lambda v: block.layernorm(X, W + h * v, B)[0] - block.layernorm(X, W - h * v, B)[0]),
                    (db, lambda v: block.layernorm(X, W, B + h * v)[0] - block.layernorm(X, W, B - h * v)[0])):
        v = rng.standard_normal(grad.shape)
        d = (f(v) * DY).sum() / (2 * h)
        # the gradient's own error (1e-5 relative, see above) times the terms, and 1e-7 of the differences
        assert abs(d - (f64(grad) * v).sum()) <= 1.1e-5 * (np.abs(f64(grad) * v).sum() + 1)
