"""Refusals of the block operators, on the host: nothing is enqueued, so no GPU is needed."""
import ctypes

import pytest
import torch

import patch_attention_b200 as pa

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced on these paths


def _ln(**kw):
    a = dict(x=FAKE, y=FAKE, groups=2, rpg=3, c=64, w=FAKE, ws=64, b=FAKE, bs=64, w0=0.0, eps=1e-6, dtype=pa.PF_BF16,
             wdtype=pa.PF_BF16, mean=None, rstd=None)
    a.update(kw)
    return pa._lib().pf_layernorm(a["x"], a["y"], a["groups"], a["rpg"], a["c"], a["w"], a["ws"], a["b"], a["bs"],
                                  a["w0"], a["eps"], a["dtype"], a["wdtype"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), pa.PF_ERR_SHAPE), (dict(rpg=-1), pa.PF_ERR_SHAPE), (dict(c=0), pa.PF_ERR_SHAPE),
    (dict(c=16385, ws=16385, bs=16385), pa.PF_ERR_SHAPE), (dict(groups=1 << 20, rpg=1 << 20), pa.PF_ERR_SHAPE),
    (dict(groups=1 << 40, rpg=1 << 40), pa.PF_ERR_SHAPE),
    (dict(dtype=3), pa.PF_ERR_UNSUPPORTED), (dict(wdtype=pa.PF_F16), pa.PF_ERR_UNSUPPORTED),
    (dict(dtype=pa.PF_F32), pa.PF_ERR_UNSUPPORTED),
    (dict(x=None), pa.PF_ERR_INVALID_ARG), (dict(y=None), pa.PF_ERR_INVALID_ARG),
    (dict(ws=63), pa.PF_ERR_INVALID_ARG), (dict(bs=0), pa.PF_ERR_INVALID_ARG), (dict(ws=-64), pa.PF_ERR_INVALID_ARG),
    (dict(eps=0.0), pa.PF_ERR_INVALID_ARG), (dict(eps=float("nan")), pa.PF_ERR_INVALID_ARG),
    (dict(eps=float("inf")), pa.PF_ERR_INVALID_ARG), (dict(w0=float("inf")), pa.PF_ERR_INVALID_ARG),
    (dict(x=FAKE + 1), pa.PF_ERR_ALIGN), (dict(w=FAKE + 2, wdtype=pa.PF_F32), pa.PF_ERR_ALIGN),
    (dict(mean=FAKE + 2), pa.PF_ERR_ALIGN),
    (dict(rpg=0, x=None, y=None), pa.PF_OK),
])
def test_layernorm(kw, status):
    assert _ln(**kw) == status


def _ln_bwd(**kw):
    need = pa.pf_layernorm_bwd_workspace_bytes(2, 300, 64)
    a = dict(dy=FAKE, x=FAKE, groups=2, rpg=300, c=64, w=FAKE, ws=64, w0=0.0, dtype=pa.PF_BF16, wdtype=pa.PF_BF16,
             mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE, work=FAKE, bytes=need)
    a.update(kw)
    return pa._lib().pf_layernorm_bwd(a["dy"], a["x"], a["groups"], a["rpg"], a["c"], a["w"], a["ws"], a["w0"], a["dtype"],
                                      a["wdtype"], a["mean"], a["rstd"], a["dx"], a["dw"], a["db"], a["work"], a["bytes"],
                                      None)


def test_layernorm_backward():
    need = pa.pf_layernorm_bwd_workspace_bytes(2, 300, 64)
    assert need >= 2 * 2 * 64 * 4
    assert pa.pf_layernorm_bwd_workspace_bytes(2, 0, 64) == 0 and pa.pf_layernorm_bwd_workspace_bytes(0, 1, 64) == 0
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert _ln_bwd(**{name: None}) == pa.PF_ERR_INVALID_ARG, name
    assert _ln_bwd(bytes=need - 1) == pa.PF_ERR_INVALID_ARG
    assert _ln_bwd(work=None) == pa.PF_ERR_INVALID_ARG
    assert _ln_bwd(work=FAKE + 8) == pa.PF_ERR_ALIGN
    assert _ln_bwd(dw=FAKE + 1) == pa.PF_ERR_ALIGN
    assert _ln_bwd(c=0) == pa.PF_ERR_SHAPE


def _rope_cfg(**kw):
    a = dict(batch=1, tokens=4, heads_q=2, heads_k=2, head_dim=64, n_axes=3, axis_dim=(16, 24, 24), theta=(1e4,) * 3,
             interleaved=1, dtype=pa.PF_BF16, eps=1e-6, pos_batch_stride=0)
    a.update(kw)
    pad = lambda t: tuple(t) + (0,) * (4 - len(t))  # noqa: E731
    return pa.pf_rope_config(a["batch"], a["tokens"], a["heads_q"], a["heads_k"], a["head_dim"], a["n_axes"],
                             (ctypes.c_int * 4)(*pad(a["axis_dim"])), (ctypes.c_double * 4)(*pad(a["theta"])),
                             a["interleaved"], a["dtype"], a["eps"], a["pos_batch_stride"])


def _rope(cfg, st=(512, 128, 64), **kw):
    a = dict(pos=FAKE, q=FAKE, k=FAKE, gq=None, gk=None, qo=FAKE, ko=FAKE, st=st and pa.pf_strides(*st))
    a.update(kw)
    s = a["st"]
    return pa._lib().pf_qk_norm_rope(cfg, a["pos"], a["q"], s, a["k"], s, a["gq"], a["gk"], a["qo"], s, a["ko"], s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=60), pa.PF_ERR_SHAPE), (dict(head_dim=264), pa.PF_ERR_SHAPE), (dict(head_dim=0), pa.PF_ERR_SHAPE),
    (dict(n_axes=0), pa.PF_ERR_SHAPE), (dict(n_axes=5), pa.PF_ERR_SHAPE), (dict(axis_dim=(16, 24, 26)), pa.PF_ERR_SHAPE),
    (dict(axis_dim=(15, 24, 24)), pa.PF_ERR_SHAPE), (dict(axis_dim=(0, 24, 24)), pa.PF_ERR_SHAPE),
    (dict(axis_dim=(-2, 24, 24)), pa.PF_ERR_SHAPE), (dict(batch=-1), pa.PF_ERR_SHAPE), (dict(tokens=-1), pa.PF_ERR_SHAPE),
    (dict(heads_q=0, heads_k=0), pa.PF_ERR_SHAPE), (dict(heads_q=-1), pa.PF_ERR_SHAPE),
    (dict(batch=1 << 20, tokens=1 << 20), pa.PF_ERR_SHAPE),
    (dict(dtype=7), pa.PF_ERR_UNSUPPORTED), (dict(eps=-1.0), pa.PF_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pa.PF_ERR_INVALID_ARG), (dict(theta=(1e4, 0.0, 1e4)), pa.PF_ERR_INVALID_ARG),
    (dict(theta=(1e4, float("inf"), 1e4)), pa.PF_ERR_INVALID_ARG), (dict(pos_batch_stride=-1), pa.PF_ERR_INVALID_ARG),
    (dict(tokens=0), pa.PF_OK), (dict(batch=0), pa.PF_OK),
])
def test_rope_config(kw, status):
    cfg = _rope_cfg(**kw)
    assert _rope(cfg) == status
    if status != pa.PF_OK:
        assert pa.pf_qk_norm_rope_bwd_workspace_bytes(cfg) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(pos=None), pa.PF_ERR_INVALID_ARG), (dict(q=None), pa.PF_ERR_INVALID_ARG), (dict(ko=None), pa.PF_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), pa.PF_ERR_ALIGN), (dict(qo=FAKE + 2), pa.PF_ERR_ALIGN), (dict(gk=FAKE + 8), pa.PF_ERR_ALIGN),
    (dict(pos=FAKE + 2), pa.PF_ERR_ALIGN), (dict(st=(512, 132, 64)), pa.PF_ERR_ALIGN),
    (dict(st=(512, 128, 68)), pa.PF_ERR_ALIGN), (dict(st=None), pa.PF_ERR_INVALID_ARG),
])
def test_rope_operands(kw, status):
    assert _rope(_rope_cfg(), **kw) == status


def test_rope_gains_need_a_norm_and_heads():
    assert _rope(_rope_cfg(eps=0.0), gq=FAKE) == pa.PF_ERR_INVALID_ARG
    cfg = _rope_cfg(heads_k=0)
    assert _rope(cfg, k=None, ko=None, gk=FAKE) == pa.PF_ERR_INVALID_ARG
    assert _rope(cfg) == pa.PF_ERR_INVALID_ARG  # keys given without heads


def test_rope_backward():
    cfg = _rope_cfg()
    need = pa.pf_qk_norm_rope_bwd_workspace_bytes(cfg)
    assert need >= 2 * 64 * 4

    def call(c=cfg, **kw):
        st = pa.pf_strides(512, 128, 64)
        a = dict(pos=FAKE, dqo=FAKE, dko=FAKE, q=FAKE, k=FAKE, gq=None, gk=None, dq=FAKE, dk=FAKE, dgq=FAKE, dgk=FAKE,
                 work=FAKE, bytes=need)
        a.update(kw)
        return pa._lib().pf_qk_norm_rope_bwd(c, a["pos"], a["dqo"], st, a["dko"], st, a["q"], st, a["k"], st, a["gq"],
                                             a["gk"], a["dq"], st, a["dk"], st, a["dgq"], a["dgk"], a["work"], a["bytes"],
                                             None)

    for name in ("pos", "dqo", "dko", "q", "k", "dq", "dk", "work"):
        assert call(**{name: None}) == pa.PF_ERR_INVALID_ARG, name
    assert call(bytes=need - 1) == pa.PF_ERR_INVALID_ARG
    assert call(work=FAKE + 8) == pa.PF_ERR_ALIGN
    assert call(dgq=FAKE + 1) == pa.PF_ERR_ALIGN
    assert call(_rope_cfg(eps=0.0)) == pa.PF_ERR_INVALID_ARG  # gain gradients without a norm


def _attn_cfg(**kw):
    a = dict(batch=2, heads_q=4, heads_kv=2, head_dim=64, n_q=10, n_k=20, softmax_scale=0.0, softcap=0.0, causal=1,
             q=(2560, 256, 64), k=(2560, 128, 64), v=(2560, 128, 64))
    a.update(kw)
    return pa.pf_masked_attn_config(a["batch"], a["heads_q"], a["heads_kv"], a["head_dim"], a["n_q"], a["n_k"],
                                    a["softmax_scale"], a["softcap"], a["causal"], pa.pf_strides(*a["q"]),
                                    pa.pf_strides(*a["k"]), pa.pf_strides(*a["v"]))


def _attn(cfg, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, slopes=None, prefix=None, doc_q=None, doc_k=None, o=FAKE, lse=None)
    a.update(kw)
    return pa._lib().pf_masked_attn(cfg, *a.values(), None)


def _attn_bwd(cfg, **kw):
    a = dict(dout=FAKE, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, slopes=None, prefix=None, doc_q=None, doc_k=None,
             dq=FAKE, dk=FAKE, dv=FAKE, work=FAKE, bytes=1 << 20)
    a.update(kw)
    return pa._lib().pf_masked_attn_bwd(cfg, *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), pa.PF_ERR_SHAPE), (dict(heads_q=5), pa.PF_ERR_SHAPE), (dict(heads_kv=0), pa.PF_ERR_SHAPE),
    (dict(heads_q=0), pa.PF_ERR_SHAPE), (dict(n_q=-1), pa.PF_ERR_SHAPE), (dict(n_k=-1), pa.PF_ERR_SHAPE),
    (dict(n_k=(1 << 30) + 1), pa.PF_ERR_SHAPE), (dict(batch=1 << 16, heads_q=1 << 10, n_q=1 << 20), pa.PF_ERR_SHAPE),
    (dict(head_dim=96), pa.PF_ERR_UNSUPPORTED), (dict(softmax_scale=-1.0), pa.PF_ERR_INVALID_ARG),
    (dict(softmax_scale=float("nan")), pa.PF_ERR_INVALID_ARG), (dict(softcap=-1.0), pa.PF_ERR_INVALID_ARG),
    (dict(softcap=float("inf")), pa.PF_ERR_INVALID_ARG), (dict(softcap=1e-38, softmax_scale=1e30), pa.PF_ERR_INVALID_ARG),
    (dict(q=(2560, 260, 64)), pa.PF_ERR_ALIGN), (dict(k=(2560, 0, 64)), pa.PF_ERR_INVALID_ARG),
    (dict(v=(2560, -128, 64)), pa.PF_ERR_INVALID_ARG), (dict(v=(1 << 39, 128, 64)), pa.PF_ERR_INVALID_ARG),
])
def test_masked_attention_config(kw, status):
    cfg = _attn_cfg(**kw)
    assert _attn(cfg) == status and _attn_bwd(cfg) == status
    assert pa.pf_masked_attn_bwd_workspace_bytes(cfg) == 0


def test_masked_attention_operands():
    cfg = _attn_cfg()
    for name in ("q", "k", "v", "o"):
        assert _attn(cfg, **{name: None}) == pa.PF_ERR_INVALID_ARG
        assert _attn(cfg, **{name: FAKE + 8}) == pa.PF_ERR_ALIGN
    for name in ("dout", "q", "k", "v", "o", "dq", "dk", "dv", "work"):
        assert _attn_bwd(cfg, **{name: None}) == pa.PF_ERR_INVALID_ARG
        assert _attn_bwd(cfg, **{name: FAKE + 8}) == pa.PF_ERR_ALIGN
    assert _attn_bwd(cfg, lse=None) == pa.PF_ERR_INVALID_ARG and _attn_bwd(cfg, lse=FAKE + 2) == pa.PF_ERR_ALIGN
    assert _attn(cfg, lse=FAKE + 2) == pa.PF_ERR_ALIGN
    need = pa.pf_masked_attn_bwd_workspace_bytes(cfg)
    assert need == 2 * 4 * 10 * 4 and _attn_bwd(cfg, bytes=need - 1) == pa.PF_ERR_INVALID_ARG
    # masks: a prefix without a causal mask, one side's documents, too many keys for documents
    assert _attn(_attn_cfg(causal=0), prefix=FAKE) == pa.PF_ERR_INVALID_ARG
    assert _attn(cfg, doc_q=FAKE) == pa.PF_ERR_INVALID_ARG and _attn(cfg, doc_k=FAKE) == pa.PF_ERR_INVALID_ARG
    assert _attn(cfg, doc_q=FAKE + 2, doc_k=FAKE) == pa.PF_ERR_ALIGN
    assert _attn(_attn_cfg(n_k=(1 << 20) + 1), doc_q=FAKE, doc_k=FAKE) == pa.PF_ERR_SHAPE
    assert _attn_bwd(_attn_cfg(n_q=(1 << 20) + 1), doc_q=FAKE, doc_k=FAKE) == pa.PF_ERR_SHAPE
    assert _attn(None) == pa.PF_ERR_INVALID_ARG and _attn_bwd(None) == pa.PF_ERR_INVALID_ARG
    assert _attn(_attn_cfg(n_q=0), q=None, o=None) == pa.PF_OK


def test_score_rule():
    t = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.ScoreRule(prefix=t)
    with pytest.raises(ValueError):
        pa.ScoreRule(doc_q=t)
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.masked_attention(q, q, q)  # not on a GPU


def test_python_refuses_cpu_tensors_and_bad_layouts():
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        pa.layernorm(x)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(torch.zeros(1, 2, 3, 64), None, torch.zeros(2, 1), pa.RopeAxes((64,)))
    with pytest.raises(ValueError):
        pa.qk_norm_rope(None, None, torch.zeros(2, 1), pa.RopeAxes((64,)))
    with pytest.raises(ValueError):
        pa.RopeAxes((2, 2, 2, 2, 2))
    with pytest.raises(ValueError):
        pa.RopeAxes((2, 2), theta=(1.0,))


def test_bias_needs_a_scale_to_divide_by():
    slopes = FAKE
    for scale, status in ((1e-21, pa.PF_ERR_INVALID_ARG), (1e-30, pa.PF_ERR_INVALID_ARG)):
        cfg = _attn_cfg(softmax_scale=scale)
        assert _attn(cfg, slopes=slopes) == status
        assert _attn_bwd(cfg, slopes=slopes) == status
