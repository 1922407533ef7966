"""Tensors whose elements lie more than 2^32 apart, and calls of many rows.

A strided view and its contiguous copy hold the same numbers and take the same kernels, so their results must be equal
bit for bit.
"""
import pytest
import torch

import patch_attention_b200 as pa
from tests.test_gpu_layernorm import BF, FF, HF, _check, _inputs

pytestmark = pytest.mark.gpu

FAR = 2 ** 32 + 2 ** 20


@pytest.fixture(scope="module")
def buffer():
    return torch.empty(FAR, device="cuda", dtype=BF)


def _spread(buffer, t, at):
    """A copy of t [1, n, h, d] whose tokens are spread over the buffer, from element `at` on."""
    _, n, h, d = t.shape
    step = (FAR - 2 ** 16) // (n - 1) // 8 * 8
    v = buffer[at:].as_strided((1, n, h, d), (FAR // 8 * 8, step, d, 1))
    v.copy_(t)
    assert (n - 1) * step > 2 ** 32
    return v


@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("nq", [1, 300])
def test_attention_over_a_far_cache(buffer, d, nq):
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v, do = (torch.randn(1, n, h, d, device="cuda", generator=g).to(BF)
                   for n, h in ((nq, 4), (300, 2), (300, 2), (nq, 4)))
    rule = pa.ScoreRule(causal=True)
    fk, fv = _spread(buffer, k, 0), _spread(buffer, v, 8192)
    assert torch.equal(fk, k) and torch.equal(fv, v)
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True)
    fo, flse = pa.masked_attention(q, fk, fv, rule, want_lse=True)
    assert torch.equal(o, fo) and torch.equal(lse, flse)
    for a, b in zip(pa.masked_attention_backward(do, q, k, v, o, lse, rule),
                    pa.masked_attention_backward(do, q, fk, fv, o, lse, rule)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    pa.pf_device_status()


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_of_far_tokens(buffer, interleaved):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, dy = (torch.randn(1, 300, 4, 64, device="cuda", generator=g).to(BF) for _ in range(2))
    gain = torch.randn(64, device="cuda", generator=g).to(BF)
    pos = torch.arange(300, device="cuda", dtype=torch.float32)[:, None]
    axes = pa.RopeAxes((64,), interleaved=interleaved)
    want, _ = pa.qk_norm_rope(q, None, pos, axes, gain_q=gain, eps=1e-6)
    far = _spread(buffer, q, 0)
    got, _ = pa.qk_norm_rope(far, None, pos, axes, gain_q=gain, eps=1e-6)
    assert torch.equal(got, want)
    a = pa.qk_norm_rope_backward(dy, None, q, None, pos, axes, gain_q=gain, eps=1e-6)
    b = pa.qk_norm_rope_backward(dy, None, far, None, pos, axes, gain_q=gain, eps=1e-6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    pa.pf_qk_norm_rope(far, None, pos, axes, far, None, gain, None, 1e-6)  # in place
    assert torch.equal(far, want)


def test_layernorm_past_32_bits(buffer):
    """The last rows of a tensor of more than 2^32 elements against a call on them alone: both are within half a step
    of the value, plus fp32's part (2^-16 of it at these sizes)."""
    c = 2048
    x = buffer[:FAR // c * c].view(-1, c)
    x[-5:] = torch.randn(5, c, device="cuda").to(BF)
    want = pa.layernorm(x[-5:].clone())
    y = x  # in place: the rest of the rows is whatever the buffer holds
    pa.pf_layernorm(x, y)
    assert torch.allclose(y[-5:].float(), want.float(), rtol=2 ** -7 * 1.01, atol=1e-5)


@pytest.mark.parametrize("shape,grouped", [((1, 6001, 264), False), ((3, 8000, 256), True), ((1, 24001, 40), False),
                                           ((2, 12001, 264), True), ((1, 6001, 33), False), ((40, 600, 128), True)])
@pytest.mark.parametrize("dtype,wide", [(BF, False), (HF, False), (BF, True), (FF, False)])
def test_layernorm_of_many_rows(shape, grouped, dtype, wide):
    """Enough rows that blocks walk over them, in one round and in several."""
    x, dy, w, b = _inputs(shape, dtype, grouped, wide, seed=shape[1])
    if grouped:
        _check(x, dy, w, b, 1.0)
    else:
        _check(x, dy, w, b, 0.0)
        if dtype == BF and not wide:
            _check(x, dy, w, None, 1.0)
            _check(x, dy, None, None, 0.0)
