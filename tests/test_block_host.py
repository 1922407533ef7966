"""Host side of the block operators at the ends of their arguments' ranges; no GPU is needed."""
import contextlib
import sys
import threading
import types

import pytest
import torch

import patch_attention_b200 as pa
from patch_attention_b200 import block
from tests.test_block_args import _attn, _attn_bwd, _attn_cfg, _rope_cfg


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


@pytest.mark.parametrize("less", [0, 1, 2, 3, 4, 5000, 9471, 9472, 20000])
@pytest.mark.parametrize("head_dim", [64, 256])
def test_rotary_sizes_up_to_the_most_tokens(less, head_dim):
    # as many partial rows as for any long call: what is resident at once
    axes = dict(head_dim=head_dim, n_axes=1, axis_dim=(head_dim,), theta=(1e4,))
    want = pa.pf_qk_norm_rope_bwd_workspace_bytes(_rope_cfg(tokens=1 << 20, **axes))
    assert want > 0
    assert pa.pf_qk_norm_rope_bwd_workspace_bytes(_rope_cfg(tokens=2 ** 31 - 1 - less, **axes)) == want


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


@pytest.fixture
def two_devices(monkeypatch):
    """Two fake devices with a status word each; pf_device_status reads and clears the current one's."""
    at = types.SimpleNamespace(current=0, words=[0, 0], synchronised=[])

    class Stream:
        def __init__(self, index, handle):
            self.device, self.cuda_stream = torch.device("cuda", index), handle

    @contextlib.contextmanager
    def device(d):
        before = at.current
        if d is not None:
            at.current = d if isinstance(d, int) else torch.device(d).index
        try:
            yield
        finally:
            at.current = before

    class Lib:
        @staticmethod
        def pf_device_status(raw):
            at.synchronised.append(raw)
            word, at.words[at.current] = at.words[at.current], 0
            return pa.PF_ERR_TIMEOUT if word else pa.PF_OK

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(at.current, 100 + at.current))
    monkeypatch.setattr(block, "_lib", lambda: Lib)
    at.stream = Stream
    return at


def test_the_device_status_is_that_of_the_streams_device(two_devices):
    at = two_devices
    at.words[1] = 4
    block.pf_device_status()  # device 0 has nothing to report, and device 1's report stays
    block.pf_device_status(at.stream(0, 7))
    assert at.words == [0, 4] and at.synchronised == [100, 7]
    with pytest.raises(pa.PatchAttnError) as e:
        block.pf_device_status(at.stream(1, 8))
    assert e.value.status == pa.PF_ERR_TIMEOUT and at.current == 0 and at.words == [0, 0]
    block.pf_device_status(at.stream(1, 8))  # the report is cleared
    assert at.synchronised == [100, 7, 8, 8]


def test_the_device_status_of_a_named_device(two_devices):
    at = two_devices
    for stream, raw in ((None, 101), (9, 9), (0, 0)):
        at.words = [0, 2]
        block.pf_device_status(stream)
        with pytest.raises(pa.PatchAttnError):
            block.pf_device_status(stream, device=1)
        assert at.synchronised[-1] == raw and at.current == 0 and at.words == [0, 0]
    with pytest.raises(ValueError):
        block.pf_device_status(at.stream(1, 8), device="cuda:0")


def test_many_threads_with_layouts_of_their_own(monkeypatch):
    monkeypatch.setattr(block, "_MOST_LAYOUTS", 8)
    plans, errors = {}, []

    def work(t):
        try:
            for i in range(3000):
                key = (t, i) if i % 3 else i % 5  # own layouts and shared ones
                assert block._kept(plans, key, lambda: ("plan", key)) == ("plan", key)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(t,)) for t in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    assert not errors and len(plans) == 8
