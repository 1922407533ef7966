"""Host side of the block operators at the ends of their arguments' ranges; no GPU is needed."""
import pytest
import torch

import patch_attention_b200 as pa
from patch_attention_b200 import block
from tests.test_block_args import _attn, _attn_bwd, _attn_cfg


@pytest.mark.parametrize("cap,scale", [(1e30, 0.0), (3e38, 0.0), (1e25, 1e-6), (1e30, 0.9), (100.0, 1e-29)])
def test_a_cap_beyond_what_32_bits_divide_by_is_refused(cap, scale):
    # scale / cap below 1e-30: q.k times that would fall among the denormal numbers, and the scores to 0
    cfg = _attn_cfg(softcap=cap, softmax_scale=scale)
    assert _attn(cfg) == pa.PF_ERR_INVALID_ARG and _attn_bwd(cfg) == pa.PF_ERR_INVALID_ARG
    assert pa.pf_masked_attn_bwd_workspace_bytes(cfg) == 0


@pytest.mark.parametrize("cap,scale", [(1e28, 0.0), (1e29, 1.0), (1.0, 1e-25), (1e-10, 1e-20)])
def test_large_and_small_caps_are_taken(cap, scale):
    assert pa.pf_masked_attn_bwd_workspace_bytes(_attn_cfg(softcap=cap, softmax_scale=scale)) > 0
    assert _attn(_attn_cfg(softcap=cap, softmax_scale=scale, n_q=0), q=None, o=None) == pa.PF_OK


def test_a_number_that_is_zero_in_32_bits_is_not_taken_for_none():
    # 0 stands for no norm, no cap and the default scale in the C structures
    q, pos = torch.zeros(1, 2, 3, 64), torch.zeros(2, 1)
    for eps in (1e-46, 1e-300):
        with pytest.raises(ValueError):
            block._rope_config(q, None, pos, pa.RopeAxes((64,)), eps)
    assert block._rope_config(q, None, pos, pa.RopeAxes((64,)), 1e-44).eps > 0
    assert block._rope_config(q, None, pos, pa.RopeAxes((64,)), None).eps == 0
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for scale, cap in ((1e-46, 0.0), (0.0, 1e-46), (-1e-60, 0.0), (0.0, -1e-60)):
        with pytest.raises(ValueError):
            block._masked_config(q, q, q, scale, cap, False)
    block._masked_config(q, q, q, 0.0, 0.0, False)
