"""Operators of a diffusion transformer's block around the patch attention: layer norm with an
affine or a per-sample modulation, QK norm with a rotary embedding over several position axes,
and attention over capped, biased and masked scores, each with its gradients.

The ``pf_*`` functions carry the C ABI's names (``include/patchattn.h``) and fill tensors that
the caller allocated; the others allocate their outputs with torch.  All tensors of a call are on
one device, which need not be the current one; ``stream`` (a ``torch.cuda.Stream`` of that device or
a raw handle; default: the device's current stream) is where the call is enqueued and where its
outputs and workspace are allocated.  Nothing here is differentiated by autograd: the backward
functions are called by the program.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import PF_BF16, PF_F16, PF_F32, _check, _lib, pf_masked_attn_config, pf_rope_config, pf_strides

_DTYPES = {torch.bfloat16: PF_BF16, torch.float16: PF_F16, torch.float32: PF_F32}
_HERE = contextlib.nullcontext()


def _device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> torch.device:
    """The one CUDA device of a call's tensors (None is skipped)."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: one device per call")
    return dev


def _on(dev: torch.device, stream):
    """Context in which `dev` is the current device and `stream` its current stream."""
    if stream is None:
        return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    return torch.cuda.stream(stream)


def _raw_stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype_of(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _whole(t: Optional[torch.Tensor], dtype, shape, name: str) -> Optional[int]:
    """Pointer of a contiguous tensor of that type and shape (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ------------------------------------------------------------------ layer norm


def _ln_layout(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor]):
    """(groups, rows per group, channels, parameter type, weight row stride, bias row stride)."""
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least one channel")
    c = x.shape[-1]
    groups, wdtype, strides = None, x.dtype, [0, 0]
    for at, (t, name) in enumerate(((weight, "weight"), (bias, "bias"))):
        if t is None:
            continue
        if t.dtype != x.dtype and t.dtype != torch.float32:
            raise ValueError(f"{name} must be {x.dtype} or float32, got {t.dtype}")
        if t.dim() == 1:
            g = 1
        elif t.dim() == 2 and x.dim() >= 2 and t.shape[0] == x.shape[0]:
            g = t.shape[0]
        else:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({c},) or ({x.shape[0]}, {c})")
        if t.shape[-1] != c or t.stride(-1) != 1 and c > 1:
            raise ValueError(f"{name} needs {c} contiguous channels")
        if groups is not None and (g, wdtype) != (groups, t.dtype):
            raise ValueError("weight and bias must have one type and number of rows")
        groups, wdtype = g, t.dtype
        strides[at] = t.stride(0) if t.dim() == 2 else 0
        if t.dim() == 2 and g > 1 and strides[at] < c:
            raise ValueError(f"{name}'s rows overlap (an expanded tensor?)")
    groups = 1 if groups is None else groups
    rows = x.numel() // c
    if groups == 0:  # a modulation of no samples
        groups, rows = 1, 0
    return groups, rows // groups, c, wdtype, strides[0], strides[1]


def pf_layernorm(x: torch.Tensor, y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, weight_offset: float = 0.0, eps: float = 1e-6,
                 mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None) -> None:
    dev = _device(x, y, weight, bias, mean, rstd)
    code = _dtype_of(x, "x")
    groups, rpg, c, wdtype, ws, bs = _ln_layout(x, weight, bias)
    xp, yp = _whole(x, x.dtype, x.shape, "x"), _whole(y, x.dtype, x.shape, "y")
    stats = x.shape[:-1]
    mp, rp = _whole(mean, torch.float32, stats, "mean"), _whole(rstd, torch.float32, stats, "rstd")
    with _on(dev, stream):
        _check(_lib().pf_layernorm(xp, yp, groups, rpg, c, None if weight is None else weight.data_ptr(), ws,
                                   None if bias is None else bias.data_ptr(), bs, weight_offset, eps, code,
                                   _DTYPES[wdtype], mp, rp, _raw_stream(dev)), "pf_layernorm")


def pf_layernorm_bwd_workspace_bytes(groups: int, rows_per_group: int, channels: int) -> int:
    return int(_lib().pf_layernorm_bwd_workspace_bytes(groups, rows_per_group, channels))


def pf_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], weight_offset: float,
                     mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                     dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dweight and dbias are [C] or [x.shape[0], C] as the forward call's parameters were (weight's own shape
    when there is one) and share their type."""
    dev = _device(x, dy, weight, mean, rstd, dx, dweight, dbias, workspace)
    code = _dtype_of(x, "x")
    lead = weight if weight is not None else dweight if dweight is not None else dbias
    groups, rpg, c, wdtype, ws, _ = _ln_layout(x, lead, None)
    xp, dyp, dxp = (_whole(t, x.dtype, x.shape, n) for t, n in ((x, "x"), (dy, "dy"), (dx, "dx")))
    mp, rp = (_whole(t, torch.float32, x.shape[:-1], n) for t, n in ((mean, "mean"), (rstd, "rstd")))
    shape = None if lead is None else lead.shape
    dwp, dbp = _whole(dweight, wdtype, shape, "dweight"), _whole(dbias, wdtype, shape, "dbias")
    wp = None if workspace is None else _whole(workspace, torch.uint8, workspace.shape, "workspace")
    with _on(dev, stream):
        _check(_lib().pf_layernorm_bwd(dyp, xp, groups, rpg, c, None if weight is None else weight.data_ptr(), ws,
                                       weight_offset, code, _DTYPES[wdtype], mp, rp, dxp, dwp, dbp, wp,
                                       0 if workspace is None else workspace.numel(), _raw_stream(dev)),
               "pf_layernorm_bwd")


def layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
              weight_offset: float = 0.0, eps: float = 1e-6, want_stats: bool = False, stream=None):
    """Layer norm over the last dimension of the contiguous x.

    weight and bias are [C], or [x.shape[0], C] (rows may be views into a wider modulation tensor) for one
    modulation per sample, then usually with ``weight_offset=1``.  They have x's type or float32.  Returns y,
    or (y, mean, rstd) with the fp32 statistics that ``layernorm_backward`` takes."""
    with _on(_device(x), stream):
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        mean = rstd = None
        if want_stats:
            mean, rstd = torch.empty((2,) + tuple(x.shape[:-1]), dtype=torch.float32, device=x.device)
        pf_layernorm(x, y, weight, bias, weight_offset, eps, mean, rstd)
    return (y, mean, rstd) if want_stats else y


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                       rstd: torch.Tensor, *, weight_offset: float = 0.0, want_dweight: bool = True,
                       want_dbias: bool = True, bias_like: Optional[torch.Tensor] = None, stream=None):
    """(dx, dweight, dbias) of ``layernorm``; a gradient that is not wanted is None.  The sums have the shape and
    type of weight, or of ``bias_like`` (the bias) for a norm without a weight, which then has no dweight."""
    like = weight if weight is not None else bias_like
    with _on(_device(x), stream):
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        new = lambda want: torch.empty(like.shape, dtype=like.dtype, device=x.device) if want else None  # noqa: E731
        dw, db = new(want_dweight and weight is not None), new(want_dbias and like is not None)
        ws = None
        if dw is not None or db is not None:
            groups, rpg, c = _ln_layout(x, like, None)[:3]
            ws = torch.empty(pf_layernorm_bwd_workspace_bytes(groups, rpg, c), dtype=torch.uint8, device=x.device)
        pf_layernorm_bwd(dy, x, weight, weight_offset, mean, rstd, dx, dw, db, ws)
    return dx, dw, db


# ------------------------------------------------------------------ QK norm + rotary


class RopeAxes:
    """How a head vector is cut into rotary sections: ``dims[a]`` elements turn with position axis a (even; the
    elements past them do not turn), at frequencies theta^(-2i/dims[a]).  ``interleaved`` pairs elements
    (2i, 2i + 1) of a section, otherwise (i, i + dims[a]/2)."""

    def __init__(self, dims: Sequence[int], theta=10000.0, interleaved: bool = True):
        self.dims: Tuple[int, ...] = tuple(int(d) for d in dims)
        if not 1 <= len(self.dims) <= 4:
            raise ValueError("one to four axes")
        self.theta = tuple(float(t) for t in theta) if isinstance(theta, (tuple, list)) else (float(theta),) * len(self.dims)
        if len(self.theta) != len(self.dims):
            raise ValueError("one theta, or one per axis")
        self.interleaved = bool(interleaved)


def _heads_view(t: Optional[torch.Tensor], like: Optional[torch.Tensor], name: str):
    """Pointer and strides of a [batch, tokens, heads, head_dim] tensor with contiguous head vectors."""
    if t is None:
        return None, None
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, tokens, heads, head_dim], got {tuple(t.shape)}")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {like.dtype} {tuple(like.shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"{name}'s head vectors must be contiguous")
    # the stride of a dimension of one element is never used: any multiple of 16 bytes will do
    b, n, h = (t.stride(i) if t.shape[i] > 1 else 0 for i in range(3))
    return t.data_ptr(), pf_strides(b, n, h)


def _no_overlap(t: Optional[torch.Tensor], name: str) -> None:
    """An output must not be an expanded tensor."""
    if t is not None and any(t.stride(i) == 0 and t.shape[i] > 1 for i in range(t.dim())):
        raise ValueError(f"{name} has overlapping elements")


def _rope_config(q, k, pos, axes: RopeAxes, eps) -> pf_rope_config:
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is needed")
    if lead.dim() != 4:
        raise ValueError(f"expected [batch, tokens, heads, head_dim], got {tuple(lead.shape)}")
    b, n, _, d = lead.shape
    if k is not None and (k.dim() != 4 or (k.shape[0], k.shape[1], k.shape[3]) != (b, n, d) or k.dtype != lead.dtype):
        raise ValueError("q and k must agree but for their heads")
    na = len(axes.dims)
    if pos.dtype != torch.float32 or tuple(pos.shape) not in ((n, na), (b, n, na)):
        raise ValueError(f"pos must be float32 of shape ({n}, {na}) or ({b}, {n}, {na}), got {pos.dtype} {tuple(pos.shape)}")
    if not pos.is_contiguous():
        raise ValueError("pos must be contiguous")
    if eps is not None and not eps > 0:
        raise ValueError("eps must be positive (None: no norm)")
    pad = (0,) * (4 - na)
    return pf_rope_config(b, n, 0 if q is None else q.shape[2], 0 if k is None else k.shape[2], d, na,
                          (ctypes.c_int * 4)(*(axes.dims + pad)), (ctypes.c_double * 4)(*(axes.theta + pad)),
                          int(axes.interleaved), _dtype_of(lead, "q"), 0.0 if eps is None else eps,
                          n * na if pos.dim() == 3 else 0)


def pf_qk_norm_rope(q, k, pos, axes: RopeAxes, q_out, k_out, gain_q=None, gain_k=None, eps: Optional[float] = None,
                    stream=None) -> None:
    lead = q if q is not None else k
    cfg = _rope_config(q, k, pos, axes, eps)
    dev = _device(lead, k, pos, q_out, k_out, gain_q, gain_k)
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("an output for each input")
    _no_overlap(q_out, "q_out")
    _no_overlap(k_out, "k_out")
    d = (lead.shape[3],)
    args = _heads_view(q, None, "q") + _heads_view(k, None, "k") + (
        _whole(gain_q, lead.dtype, d, "gain_q"), _whole(gain_k, lead.dtype, d, "gain_k"))
    outs = _heads_view(q_out, q, "q_out") + _heads_view(k_out, k, "k_out")
    with _on(dev, stream):
        _check(_lib().pf_qk_norm_rope(cfg, pos.data_ptr(), *args, *outs, _raw_stream(dev)), "pf_qk_norm_rope")


def pf_qk_norm_rope_bwd_workspace_bytes(cfg: pf_rope_config) -> int:
    return int(_lib().pf_qk_norm_rope_bwd_workspace_bytes(cfg))


def pf_qk_norm_rope_bwd(dq_out, dk_out, q, k, pos, axes: RopeAxes, dq, dk, gain_q=None, gain_k=None,
                        eps: Optional[float] = None, dgain_q=None, dgain_k=None, workspace=None, stream=None) -> None:
    lead = dq_out if dq_out is not None else dk_out
    cfg = _rope_config(dq_out, dk_out, pos, axes, eps)
    dev = _device(lead, dk_out, q, k, pos, dq, dk, gain_q, gain_k, dgain_q, dgain_k, workspace)
    if (dq_out is None) != (dq is None) or (dk_out is None) != (dk is None):
        raise ValueError("an output for each input")
    if dq_out is None and q is not None or dk_out is None and k is not None:
        raise ValueError("an input without its gradient")
    _no_overlap(dq, "dq")
    _no_overlap(dk, "dk")
    d = (lead.shape[3],)
    args = (_heads_view(dq_out, None, "dq_out") + _heads_view(dk_out, None, "dk_out")
            + _heads_view(q, dq_out, "q") + _heads_view(k, dk_out, "k")
            + (_whole(gain_q, lead.dtype, d, "gain_q"), _whole(gain_k, lead.dtype, d, "gain_k"))
            + _heads_view(dq, dq_out, "dq") + _heads_view(dk, dk_out, "dk")
            + (_whole(dgain_q, lead.dtype, d, "dgain_q"), _whole(dgain_k, lead.dtype, d, "dgain_k")))
    wp = None if workspace is None else _whole(workspace, torch.uint8, workspace.shape, "workspace")
    with _on(dev, stream):
        _check(_lib().pf_qk_norm_rope_bwd(cfg, pos.data_ptr(), *args, wp, 0 if workspace is None else workspace.numel(),
                                          _raw_stream(dev)), "pf_qk_norm_rope_bwd")


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, axes: RopeAxes, *,
                 gain_q: Optional[torch.Tensor] = None, gain_k: Optional[torch.Tensor] = None,
                 eps: Optional[float] = None, stream=None):
    """(q, k) normalised per head (with ``eps``; gains optional) and turned by their tokens' positions.

    q and k are [batch, tokens, heads, head_dim] with contiguous head vectors (views into a packed projection are
    fine); either may be None.  pos is float32 [tokens, axes] or [batch, tokens, axes].  New contiguous tensors are
    returned; ``pf_qk_norm_rope`` works in place."""
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is needed")
    with _on(_device(lead), stream):
        out = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)]
        pf_qk_norm_rope(q, k, pos, axes, out[0], out[1], gain_q, gain_k, eps)
    return out[0], out[1]


def qk_norm_rope_backward(dq_out: Optional[torch.Tensor], dk_out: Optional[torch.Tensor], q: Optional[torch.Tensor],
                          k: Optional[torch.Tensor], pos: torch.Tensor, axes: RopeAxes, *,
                          gain_q: Optional[torch.Tensor] = None, gain_k: Optional[torch.Tensor] = None,
                          eps: Optional[float] = None, stream=None):
    """(dq, dk, dgain_q, dgain_k) from the gradients of ``qk_norm_rope``'s outputs and its inputs; a gain that was
    not given has no gradient (None).  Without a norm q and k are not read and may be None."""
    lead = dq_out if dq_out is not None else dk_out
    if lead is None:
        raise ValueError("dq_out or dk_out is needed")
    with _on(_device(lead), stream):
        new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
        dq, dk, dgq, dgk = new(dq_out), new(dk_out), new(gain_q), new(gain_k)
        ws = None
        if dgq is not None or dgk is not None:
            nbytes = pf_qk_norm_rope_bwd_workspace_bytes(_rope_config(dq_out, dk_out, pos, axes, eps))
            ws = torch.empty(nbytes, dtype=torch.uint8, device=lead.device)
        pf_qk_norm_rope_bwd(dq_out, dk_out, q, k, pos, axes, dq, dk, gain_q, gain_k, eps, dgq, dgk, ws)
    return dq, dk, dgq, dgk


# ------------------------------------------------------------------ masked attention


class ScoreRule:
    """What attention does to its scores before the softmax: ``softmax_scale`` (0: 1/sqrt(head_dim)), a cap
    ``softcap * tanh(s / softcap)`` (0: none), a distance bias ``-slopes[head] * |position - key|``, and which keys a
    query sees: all, or with ``causal`` those up to its position (queries are the last positions) and those before
    ``prefix[batch]``; and, with ``doc_q`` and ``doc_k`` (int32 ids, negative: padding), only keys of its document."""

    def __init__(self, softmax_scale: float = 0.0, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                 causal: bool = False, prefix: Optional[torch.Tensor] = None, doc_q: Optional[torch.Tensor] = None,
                 doc_k: Optional[torch.Tensor] = None):
        if prefix is not None and not causal:
            raise ValueError("a prefix goes with a causal mask")
        if (doc_q is None) != (doc_k is None):
            raise ValueError("doc_q and doc_k come together")
        self.softmax_scale, self.softcap, self.causal = float(softmax_scale), float(softcap), bool(causal)
        self.slopes, self.prefix, self.doc_q, self.doc_k = slopes, prefix, doc_q, doc_k

    def tensors(self):
        return self.slopes, self.prefix, self.doc_q, self.doc_k


def _masked_args(q, k, v, rule: ScoreRule):
    """(configuration, pointers of q, k, v, pointers of the rule's tensors)."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, tokens, heads, head_dim], got {tuple(t.shape)}")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    b, nq, hq, d = q.shape
    nk, hk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (b, nk, hk, d) or v.shape != k.shape:
        raise ValueError(f"q, k, v of shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)} do not go together")
    (qp, qs), (kp, ks), (vp, vs) = _heads_view(q, None, "q"), _heads_view(k, None, "k"), _heads_view(v, None, "v")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _no_overlap(t, name)
    cfg = pf_masked_attn_config(b, hq, hk, d, nq, nk, rule.softmax_scale, rule.softcap, int(rule.causal), qs, ks, vs)
    extra = (_whole(rule.slopes, torch.float32, (hq,), "slopes"), _whole(rule.prefix, torch.int32, (b,), "prefix"),
             _whole(rule.doc_q, torch.int32, (b, nq), "doc_q"), _whole(rule.doc_k, torch.int32, (b, nk), "doc_k"))
    return cfg, (qp, kp, vp), extra


_PLAIN = ScoreRule()


def pf_masked_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                   lse: Optional[torch.Tensor] = None, rule: Optional[ScoreRule] = None, stream=None) -> None:
    rule = rule or _PLAIN
    dev = _device(q, k, v, o, lse, *rule.tensors())
    cfg, ptrs, extra = _masked_args(q, k, v, rule)
    op = _whole(o, torch.bfloat16, q.shape, "o")
    lp = _whole(lse, torch.float32, (q.shape[0], q.shape[2], q.shape[1]), "lse")
    with _on(dev, stream):
        _check(_lib().pf_masked_attn(cfg, *ptrs, *extra, op, lp, _raw_stream(dev)), "pf_masked_attn")


def pf_device_status(stream=None) -> None:
    """Synchronise the stream; raises if a kernel's bounded wait expired on this device."""
    if stream is None:
        stream = torch.cuda.current_stream()
    raw = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    _check(_lib().pf_device_status(raw), "pf_device_status")


def masked_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rule: Optional[ScoreRule] = None, *,
                     want_lse: bool = False, stream=None):
    """Attention of bf16 q [batch, n_q, heads_q, d] over k, v [batch, n_k, heads_kv, d] (views with contiguous head
    vectors are fine; heads_q a multiple of heads_kv; d in 64, 72, 128) with the scores changed and masked by
    ``rule``.  Returns o, or (o, lse) with the fp32 [batch, heads_q, n_q] statistics of the backward pass."""
    with _on(_device(q), stream):
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = None
        if want_lse:
            lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
        pf_masked_attn(q, k, v, o, lse, rule)
    return (o, lse) if want_lse else o


def pf_masked_attn_bwd_workspace_bytes(cfg: pf_masked_attn_config) -> int:
    return int(_lib().pf_masked_attn_bwd_workspace_bytes(cfg))


def pf_masked_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                       workspace: torch.Tensor, rule: Optional[ScoreRule] = None, stream=None) -> None:
    rule = rule or _PLAIN
    dev = _device(q, k, v, dout, o, lse, dq, dk, dv, workspace, *rule.tensors())
    cfg, ptrs, extra = _masked_args(q, k, v, rule)
    bf = torch.bfloat16
    dop, op, dqp = (_whole(t, bf, q.shape, n) for t, n in ((dout, "dout"), (o, "o"), (dq, "dq")))
    dkp, dvp = (_whole(t, bf, k.shape, n) for t, n in ((dk, "dk"), (dv, "dv")))
    lp = _whole(lse, torch.float32, (q.shape[0], q.shape[2], q.shape[1]), "lse")
    wp = _whole(workspace, torch.uint8, workspace.shape, "workspace")
    with _on(dev, stream):
        _check(_lib().pf_masked_attn_bwd(cfg, dop, *ptrs, op, lp, *extra, dqp, dkp, dvp, wp, workspace.numel(),
                                         _raw_stream(dev)), "pf_masked_attn_bwd")


def masked_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                              lse: torch.Tensor, rule: Optional[ScoreRule] = None, *, stream=None):
    """(dq, dk, dv) of ``masked_attention`` from the gradient of its output, its inputs, and the o and lse that it
    returned; contiguous, dk and dv summed over the query heads that share a key head."""
    with _on(_device(q), stream):
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        ws = torch.empty(4 * q.shape[0] * q.shape[1] * q.shape[2], dtype=torch.uint8, device=q.device)
        pf_masked_attn_bwd(dout, q, k, v, o, lse, dq, dk, dv, ws, rule)
    return dq, dk, dv
