"""Masked attention at the ends of its arguments' ranges.  Tolerances as in the forward and backward tests, or equal
bits."""
import pytest
import torch

import patch_attention_b200 as pa
from tests.test_gpu_masked_attention import BF, check, inputs
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
