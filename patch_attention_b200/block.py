"""Operators of a diffusion transformer's block around the patch attention: layer norm with an
affine or a per-sample modulation, QK norm with a rotary embedding over several position axes,
and attention over capped, biased and masked scores, each with its gradients.

The ``pf_*`` functions carry the C ABI's names (``include/patchattn.h``) and fill tensors that
the caller allocated; the others allocate their outputs with torch.  All tensors of a call are on
one device, which need not be the current one; ``stream`` (a ``torch.cuda.Stream`` of that device or
a raw handle; default: the device's current stream) is where the call is enqueued and where its
outputs and workspace are allocated.  Nothing here is differentiated by autograd: the backward
functions are called by the program.

The argument checks of a layout (shapes, strides, types) are done once and kept, with the C
structures they lead to, so that a call of a layout seen before costs little more than its launch.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional, Sequence, Tuple

import torch

from . import PF_BF16, PF_F16, PF_F32, _check, _lib, pf_masked_attn_config, pf_rope_config, pf_strides

_DTYPES = {torch.bfloat16: PF_BF16, torch.float16: PF_F16, torch.float32: PF_F32}
_BF, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_MOST_LAYOUTS = 4096
_keeping = threading.Lock()


def _index(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """Index of the one CUDA device of a call's tensors (None is skipped)."""
    i = first.get_device()
    if i < 0:
        raise ValueError("expected CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device per call")
    return i


def _elsewhere(i: int, stream) -> bool:
    """Whether device i and `stream` have to be made current for the call."""
    return stream is not None or torch._C._cuda_getDevice() != i


def _on(i: int, stream):
    """Context in which device i is current and `stream` its current stream."""
    if stream is None:
        return torch.cuda.device(i)
    dev = torch.device("cuda", i)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    return torch.cuda.stream(stream)


_raw_stream = torch._C._cuda_getCurrentRawStream


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
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _kept_in_32_bits(x: float, name: str) -> float:
    """x, refused where the C ABI's float would be 0, which stands for a default or for none, and x is not."""
    if x != 0 and ctypes.c_float(x).value == 0:
        raise ValueError(f"{name} of {x} is 0 in 32 bits")
    return x


def _layout(t: Optional[torch.Tensor]):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _kept(plans: dict, key, make):
    """plans[key], made on first use; the oldest layouts go when there are too many.  Threads may ask at once: what is
    there is read without the lock, two that make the same plan keep one of them."""
    plan = plans.get(key)
    if plan is None:
        plan = make()
        with _keeping:
            while len(plans) >= _MOST_LAYOUTS:
                plans.pop(next(iter(plans)), None)
            plans[key] = plan
    return plan


# ------------------------------------------------------------------ layer norm

_ln_plans: dict = {}


def _ln_layout(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor]):
    """(groups, rows per group, channels, weight row stride, bias row stride, x's type, parameter type)."""
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least one channel")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    c = x.shape[-1]
    groups, wdtype, strides = None, x.dtype, [0, 0]
    for at, (t, name) in enumerate(((weight, "weight"), (bias, "bias"))):
        if t is None:
            continue
        if t.dtype != x.dtype and t.dtype != _F32:
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
    return groups, rows // groups, c, strides[0], strides[1], _dtype_of(x, "x"), _DTYPES[wdtype]


def _ln_plan(x, weight, bias):
    return _kept(_ln_plans, (_layout(x), _layout(weight), _layout(bias)), lambda: _ln_layout(x, weight, bias))


def pf_layernorm(x: torch.Tensor, y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, weight_offset: float = 0.0, eps: float = 1e-6,
                 mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None) -> None:
    i = _index(x, y, weight, bias, mean, rstd)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_layernorm(x, y, weight, bias, weight_offset, eps, mean, rstd)
    groups, rpg, c, ws, bs, code, wcode = _ln_plan(x, weight, bias)
    yp = _whole(y, x.dtype, x.shape, "y")
    mp, rp = _whole(mean, _F32, x.shape[:-1], "mean"), _whole(rstd, _F32, x.shape[:-1], "rstd")
    _check(_lib().pf_layernorm(x.data_ptr(), yp, groups, rpg, c, _ptr(weight), ws, _ptr(bias), bs, weight_offset, eps,
                               code, wcode, mp, rp, _raw_stream(i)), "pf_layernorm")


def pf_layernorm_bwd_workspace_bytes(groups: int, rows_per_group: int, channels: int) -> int:
    return int(_lib().pf_layernorm_bwd_workspace_bytes(groups, rows_per_group, channels))


def pf_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], weight_offset: float,
                     mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                     dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dweight and dbias are [C] or [x.shape[0], C] as the forward call's parameters were (weight's own shape
    when there is one) and share their type."""
    i = _index(x, dy, weight, mean, rstd, dx, dweight, dbias, workspace)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_layernorm_bwd(dy, x, weight, weight_offset, mean, rstd, dx, dweight, dbias, workspace)
    lead = weight if weight is not None else dweight if dweight is not None else dbias
    groups, rpg, c, ws, _, code, wcode = _ln_plan(x, lead, None)
    dyp, dxp = _whole(dy, x.dtype, x.shape, "dy"), _whole(dx, x.dtype, x.shape, "dx")
    mp, rp = _whole(mean, _F32, x.shape[:-1], "mean"), _whole(rstd, _F32, x.shape[:-1], "rstd")
    dwp = dbp = None
    if lead is not None:
        dwp, dbp = _whole(dweight, lead.dtype, lead.shape, "dweight"), _whole(dbias, lead.dtype, lead.shape, "dbias")
    wp = None if workspace is None else _whole(workspace, _U8, workspace.shape, "workspace")
    _check(_lib().pf_layernorm_bwd(dyp, x.data_ptr(), groups, rpg, c, _ptr(weight), ws, weight_offset, code, wcode, mp,
                                   rp, dxp, dwp, dbp, wp, 0 if workspace is None else workspace.numel(), _raw_stream(i)),
           "pf_layernorm_bwd")


def layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
              weight_offset: float = 0.0, eps: float = 1e-6, want_stats: bool = False, stream=None):
    """Layer norm over the last dimension of the contiguous x.

    weight and bias are [C], or [x.shape[0], C] (rows may be views into a wider modulation tensor) for one
    modulation per sample, then usually with ``weight_offset=1``.  They have x's type or float32.  Returns y,
    or (y, mean, rstd) with the fp32 statistics that ``layernorm_backward`` takes."""
    i = _index(x, weight, bias)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return layernorm(x, weight, bias, weight_offset=weight_offset, eps=eps, want_stats=want_stats)
    groups, rpg, c, ws, bs, code, wcode = _ln_plan(x, weight, bias)
    y = torch.empty_like(x)
    mp = rp = None
    if want_stats:
        mean, rstd = torch.empty((2,) + x.shape[:-1], dtype=_F32, device=x.device).unbind()
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _check(_lib().pf_layernorm(x.data_ptr(), y.data_ptr(), groups, rpg, c, _ptr(weight), ws, _ptr(bias), bs,
                               weight_offset, eps, code, wcode, mp, rp, _raw_stream(i)), "pf_layernorm")
    return (y, mean, rstd) if want_stats else y


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                       rstd: torch.Tensor, *, weight_offset: float = 0.0, want_dweight: bool = True,
                       want_dbias: bool = True, bias_like: Optional[torch.Tensor] = None, stream=None):
    """(dx, dweight, dbias) of ``layernorm``; a gradient that is not wanted is None.  The sums have the shape and
    type of weight, or of ``bias_like`` (the bias) for a norm without a weight, which then has no dweight."""
    like = weight if weight is not None else bias_like
    i = _index(x, dy, like, mean, rstd)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return layernorm_backward(dy, x, weight, mean, rstd, weight_offset=weight_offset, want_dweight=want_dweight,
                                      want_dbias=want_dbias, bias_like=bias_like)
    groups, rpg, c = _ln_plan(x, like, None)[:3]
    dx = torch.empty_like(x)
    dw = db = ws = None
    if weight is not None and want_dweight:
        dw = torch.empty(like.shape, dtype=like.dtype, device=x.device)
    if like is not None and want_dbias:
        db = torch.empty(like.shape, dtype=like.dtype, device=x.device)
    if dw is not None or db is not None:
        ws = torch.empty(_lib().pf_layernorm_bwd_workspace_bytes(groups, rpg, c), dtype=_U8, device=x.device)
    pf_layernorm_bwd(dy, x, weight, weight_offset, mean, rstd, dx, dw, db, ws)
    return dx, dw, db


# ------------------------------------------------------------------ QK norm + rotary

_rope_plans: dict = {}


class RopeAxes:
    """How a head vector is cut into rotary sections: ``dims[a]`` elements turn with position axis a (even; the
    elements past them do not turn), at frequencies theta^(-2i/dims[a]).  ``interleaved`` pairs elements
    (2i, 2i + 1) of a section, otherwise (i, i + dims[a]/2)."""

    def __init__(self, dims: Sequence[int], theta=10000.0, interleaved: bool = True):
        self._dims: Tuple[int, ...] = tuple(int(d) for d in dims)
        if not 1 <= len(self._dims) <= 4:
            raise ValueError("one to four axes")
        self._theta = (tuple(float(t) for t in theta) if isinstance(theta, (tuple, list))
                       else (float(theta),) * len(self._dims))
        if len(self._theta) != len(self._dims):
            raise ValueError("one theta, or one per axis")
        self._interleaved = bool(interleaved)
        self._key = (self._dims, self._theta, self._interleaved)

    dims = property(lambda self: self._dims)
    theta = property(lambda self: self._theta)
    interleaved = property(lambda self: self._interleaved)


def _heads_view(t: Optional[torch.Tensor], name: str) -> Optional[pf_strides]:
    """Strides of a [batch, tokens, heads, head_dim] tensor with contiguous head vectors."""
    if t is None:
        return None
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, tokens, heads, head_dim], got {tuple(t.shape)}")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}'s head vectors must be contiguous")
    # the stride of a dimension of one element is never used: any multiple of 16 bytes will do
    return pf_strides(*(t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)))


def _like(t: Optional[torch.Tensor], like: Optional[torch.Tensor], name: str) -> None:
    if t is not None and like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {like.dtype} {tuple(like.shape)}")


def _no_overlap(t: Optional[torch.Tensor], name: str) -> None:
    """Refuses an expanded tensor."""
    if t is not None and any(t.stride(i) == 0 and t.shape[i] > 1 for i in range(t.dim())):
        raise ValueError(f"{name} has overlapping elements")


def _rope_config(q, k, pos, axes: RopeAxes, eps) -> pf_rope_config:
    """The configuration of a call on q and k (or their gradients)."""
    lead = q if q is not None else k
    if lead.dim() != 4:
        raise ValueError(f"expected [batch, tokens, heads, head_dim], got {tuple(lead.shape)}")
    b, n, _, d = lead.shape
    if k is not None and (k.dim() != 4 or (k.shape[0], k.shape[1], k.shape[3]) != (b, n, d) or k.dtype != lead.dtype):
        raise ValueError("q and k must agree but for their heads")
    na = len(axes.dims)
    if pos.dtype != _F32 or tuple(pos.shape) not in ((n, na), (b, n, na)):
        raise ValueError(f"pos must be float32 of shape ({n}, {na}) or ({b}, {n}, {na}), got {pos.dtype} {tuple(pos.shape)}")
    if not pos.is_contiguous():
        raise ValueError("pos must be contiguous")
    if eps is not None and not eps > 0:
        raise ValueError("eps must be positive (None: no norm)")
    _kept_in_32_bits(eps or 0.0, "eps")
    pad = (0,) * (4 - na)
    return pf_rope_config(b, n, 0 if q is None else q.shape[2], 0 if k is None else k.shape[2], d, na,
                          (ctypes.c_int * 4)(*(axes.dims + pad)), (ctypes.c_double * 4)(*(axes.theta + pad)),
                          int(axes.interleaved), _dtype_of(lead, "q"), 0.0 if eps is None else eps,
                          n * na if pos.dim() == 3 else 0)


class _RopePlan:
    """Configuration and operand strides of a rotary call, checked; outputs like q and k."""

    def __init__(self, q, k, pos, axes, eps, q_out, k_out, q_in, k_in):
        cfg = _rope_config(q, k, pos, axes, eps)
        for t, like, name in ((q_out, q, "q's output"), (k_out, k, "k's output"), (q_in, q, "q"), (k_in, k, "k")):
            _like(t, like, name)
        _no_overlap(q_out, "q's output")
        _no_overlap(k_out, "k's output")
        ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
        self.cfg = ctypes.byref(cfg)
        self.q, self.k = ref(_heads_view(q, "q")), ref(_heads_view(k, "k"))
        self.q_out, self.k_out = ref(_heads_view(q_out, "q's output")), ref(_heads_view(k_out, "k's output"))
        self.q_in, self.k_in = ref(_heads_view(q_in, "q")), ref(_heads_view(k_in, "k"))
        self.gain_shape = (q if q is not None else k).shape[3:]
        self.bytes = int(_lib().pf_qk_norm_rope_bwd_workspace_bytes(cfg))


def _rope_plan(q, k, pos, axes, eps, q_out, k_out, q_in=None, k_in=None) -> _RopePlan:
    key = (axes._key, eps, _layout(q), _layout(k), _layout(pos), _layout(q_out), _layout(k_out), _layout(q_in), _layout(k_in))
    return _kept(_rope_plans, key, lambda: _RopePlan(q, k, pos, axes, eps, q_out, k_out, q_in, k_in))


def pf_qk_norm_rope(q, k, pos, axes: RopeAxes, q_out, k_out, gain_q=None, gain_k=None, eps: Optional[float] = None,
                    stream=None) -> None:
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is needed")
    i = _index(lead, k, pos, q_out, k_out, gain_q, gain_k)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_qk_norm_rope(q, k, pos, axes, q_out, k_out, gain_q, gain_k, eps)
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("an output for each input")
    p = _rope_plan(q, k, pos, axes, eps, q_out, k_out)
    gq, gk = _whole(gain_q, lead.dtype, p.gain_shape, "gain_q"), _whole(gain_k, lead.dtype, p.gain_shape, "gain_k")
    _check(_lib().pf_qk_norm_rope(p.cfg, pos.data_ptr(), _ptr(q), p.q, _ptr(k), p.k, gq, gk, _ptr(q_out), p.q_out,
                                  _ptr(k_out), p.k_out, _raw_stream(i)), "pf_qk_norm_rope")


def pf_qk_norm_rope_bwd_workspace_bytes(cfg: pf_rope_config) -> int:
    return int(_lib().pf_qk_norm_rope_bwd_workspace_bytes(cfg))


def pf_qk_norm_rope_bwd(dq_out, dk_out, q, k, pos, axes: RopeAxes, dq, dk, gain_q=None, gain_k=None,
                        eps: Optional[float] = None, dgain_q=None, dgain_k=None, workspace=None, stream=None) -> None:
    lead = dq_out if dq_out is not None else dk_out
    if lead is None:
        raise ValueError("dq_out or dk_out is needed")
    i = _index(lead, dk_out, q, k, pos, dq, dk, gain_q, gain_k, dgain_q, dgain_k, workspace)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_qk_norm_rope_bwd(dq_out, dk_out, q, k, pos, axes, dq, dk, gain_q, gain_k, eps, dgain_q, dgain_k,
                                       workspace)
    if (dq_out is None) != (dq is None) or (dk_out is None) != (dk is None):
        raise ValueError("an output for each input")
    if dq_out is None and q is not None or dk_out is None and k is not None:
        raise ValueError("an input without its gradient")
    p = _rope_plan(dq_out, dk_out, pos, axes, eps, dq, dk, q, k)
    g = [_whole(t, lead.dtype, p.gain_shape, n) for t, n in ((gain_q, "gain_q"), (gain_k, "gain_k"),
                                                             (dgain_q, "dgain_q"), (dgain_k, "dgain_k"))]
    wp = None if workspace is None else _whole(workspace, _U8, workspace.shape, "workspace")
    _check(_lib().pf_qk_norm_rope_bwd(p.cfg, pos.data_ptr(), _ptr(dq_out), p.q, _ptr(dk_out), p.k, _ptr(q), p.q_in,
                                      _ptr(k), p.k_in, g[0], g[1], _ptr(dq), p.q_out, _ptr(dk), p.k_out, g[2], g[3], wp,
                                      0 if workspace is None else workspace.numel(), _raw_stream(i)),
           "pf_qk_norm_rope_bwd")


def _new(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """A contiguous tensor like t."""
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


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
    i = _index(lead, k, pos, gain_q, gain_k)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return qk_norm_rope(q, k, pos, axes, gain_q=gain_q, gain_k=gain_k, eps=eps)
    q_out, k_out = _new(q), _new(k)
    # outputs made here need no look at their layout
    key = (axes._key, eps, _layout(q), _layout(k), _layout(pos))
    p = _kept(_rope_plans, key, lambda: _RopePlan(q, k, pos, axes, eps, q_out, k_out, None, None))
    gq, gk = _whole(gain_q, lead.dtype, p.gain_shape, "gain_q"), _whole(gain_k, lead.dtype, p.gain_shape, "gain_k")
    _check(_lib().pf_qk_norm_rope(p.cfg, pos.data_ptr(), _ptr(q), p.q, _ptr(k), p.k, gq, gk, _ptr(q_out), p.q_out,
                                  _ptr(k_out), p.k_out, _raw_stream(i)), "pf_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out: Optional[torch.Tensor], dk_out: Optional[torch.Tensor], q: Optional[torch.Tensor],
                          k: Optional[torch.Tensor], pos: torch.Tensor, axes: RopeAxes, *,
                          gain_q: Optional[torch.Tensor] = None, gain_k: Optional[torch.Tensor] = None,
                          eps: Optional[float] = None, stream=None):
    """(dq, dk, dgain_q, dgain_k) from the gradients of ``qk_norm_rope``'s outputs and its inputs; a gain that was
    not given has no gradient (None).  Without a norm q and k are not read and may be None."""
    lead = dq_out if dq_out is not None else dk_out
    if lead is None:
        raise ValueError("dq_out or dk_out is needed")
    i = _index(lead)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return qk_norm_rope_backward(dq_out, dk_out, q, k, pos, axes, gain_q=gain_q, gain_k=gain_k, eps=eps)
    dq, dk, dgq, dgk = _new(dq_out), _new(dk_out), _new(gain_q), _new(gain_k)
    ws = None
    if dgq is not None or dgk is not None:
        plan = _rope_plan(dq_out, dk_out, pos, axes, eps, dq, dk, q, k)
        ws = torch.empty(plan.bytes, dtype=_U8, device=lead.device)
    pf_qk_norm_rope_bwd(dq_out, dk_out, q, k, pos, axes, dq, dk, gain_q, gain_k, eps, dgq, dgk, ws)
    return dq, dk, dgq, dgk


# ------------------------------------------------------------------ masked attention

_attn_plans: dict = {}


class ScoreRule:
    """What attention does to its scores before the softmax: ``softmax_scale`` (0: 1/sqrt(head_dim)), a cap
    ``softcap * tanh(s / softcap)`` (0: none; at most 1e30 times the scale), a distance bias
    ``-slopes[head] * |position - key|``, and which keys a query sees: all, or with ``causal`` those up to its position
    (queries are the last positions) and those before ``prefix[batch]`` (zero and below: none); and, with ``doc_q`` and
    ``doc_k`` (int32 ids, negative: padding), only keys of its document."""

    def __init__(self, softmax_scale: float = 0.0, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                 causal: bool = False, prefix: Optional[torch.Tensor] = None, doc_q: Optional[torch.Tensor] = None,
                 doc_k: Optional[torch.Tensor] = None):
        if prefix is not None and not causal:
            raise ValueError("a prefix goes with a causal mask")
        if (doc_q is None) != (doc_k is None):
            raise ValueError("doc_q and doc_k come together")
        self.softmax_scale, self.softcap, self.causal = float(softmax_scale), float(softcap), bool(causal)
        self.slopes, self.prefix, self.doc_q, self.doc_k = slopes, prefix, doc_q, doc_k


def _masked_config(q, k, v, scale, cap, causal):
    """(reference to the configuration, shapes of lse, slopes, prefix, doc_q, doc_k)."""
    _kept_in_32_bits(scale, "softmax_scale")
    _kept_in_32_bits(cap, "softcap")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, tokens, heads, head_dim], got {tuple(t.shape)}")
        if t.dtype != _BF:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
        _no_overlap(t, name)
    b, nq, hq, d = q.shape
    nk, hk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (b, nk, hk, d) or v.shape != k.shape:
        raise ValueError(f"q, k, v of shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)} do not go together")
    cfg = pf_masked_attn_config(b, hq, hk, d, nq, nk, scale, cap, int(causal), _heads_view(q, "q"), _heads_view(k, "k"),
                                _heads_view(v, "v"))
    return ctypes.byref(cfg), (b, hq, nq), (hq,), (b,), (b, nq), (b, nk)


def _masked_plan(q, k, v, r: ScoreRule):
    key = (_layout(q), _layout(k), _layout(v), r.softmax_scale, r.softcap, r.causal)
    return _kept(_attn_plans, key, lambda: _masked_config(q, k, v, r.softmax_scale, r.softcap, r.causal))


def _rule_ptrs(r: ScoreRule, plan):
    return (_whole(r.slopes, _F32, plan[2], "slopes"), _whole(r.prefix, _I32, plan[3], "prefix"),
            _whole(r.doc_q, _I32, plan[4], "doc_q"), _whole(r.doc_k, _I32, plan[5], "doc_k"))


_PLAIN = ScoreRule()


def pf_masked_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                   lse: Optional[torch.Tensor] = None, rule: Optional[ScoreRule] = None, stream=None) -> None:
    r = rule or _PLAIN
    i = _index(q, k, v, o, lse, r.slopes, r.prefix, r.doc_q, r.doc_k)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_masked_attn(q, k, v, o, lse, rule)
    plan = _masked_plan(q, k, v, r)
    op, lp = _whole(o, _BF, q.shape, "o"), _whole(lse, _F32, plan[1], "lse")
    _check(_lib().pf_masked_attn(plan[0], q.data_ptr(), k.data_ptr(), v.data_ptr(), *_rule_ptrs(r, plan), op, lp,
                                 _raw_stream(i)), "pf_masked_attn")


def pf_device_status(stream=None, device=None) -> None:
    """Synchronise the stream; raises if a kernel's bounded wait expired on its device, and clears that report.  The
    device is the stream's; ``device`` names it for a raw handle or for the current stream of another device (default:
    the current device)."""
    if isinstance(stream, torch.cuda.Stream):
        if device is not None and device not in (stream.device, stream.device.index, str(stream.device)):
            raise ValueError(f"the stream belongs to {stream.device}, not {device}")
        device, stream = stream.device, stream.cuda_stream
    with torch.cuda.device(device):  # the status word is the current device's
        raw = torch.cuda.current_stream().cuda_stream if stream is None else int(stream)
        _check(_lib().pf_device_status(raw), "pf_device_status")


def masked_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rule: Optional[ScoreRule] = None, *,
                     want_lse: bool = False, stream=None):
    """Attention of bf16 q [batch, n_q, heads_q, d] over k, v [batch, n_k, heads_kv, d] (views with contiguous head
    vectors are fine; heads_q a multiple of heads_kv; d in 64, 72, 128) with the scores changed and masked by
    ``rule``.  Returns o, or (o, lse) with the fp32 [batch, heads_q, n_q] statistics of the backward pass."""
    r = rule or _PLAIN
    i = _index(q, k, v, r.slopes, r.prefix, r.doc_q, r.doc_k)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return masked_attention(q, k, v, rule, want_lse=want_lse)
    plan = _masked_plan(q, k, v, r)
    o = _new(q)
    lse = torch.empty(plan[1], dtype=_F32, device=q.device) if want_lse else None
    _check(_lib().pf_masked_attn(plan[0], q.data_ptr(), k.data_ptr(), v.data_ptr(), *_rule_ptrs(r, plan), o.data_ptr(),
                                 _ptr(lse), _raw_stream(i)), "pf_masked_attn")
    return (o, lse) if want_lse else o


def pf_masked_attn_bwd_workspace_bytes(cfg: pf_masked_attn_config) -> int:
    return int(_lib().pf_masked_attn_bwd_workspace_bytes(cfg))


def pf_masked_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                       workspace: torch.Tensor, rule: Optional[ScoreRule] = None, stream=None) -> None:
    r = rule or _PLAIN
    i = _index(q, k, v, dout, o, lse, dq, dk, dv, workspace, r.slopes, r.prefix, r.doc_q, r.doc_k)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return pf_masked_attn_bwd(dout, q, k, v, o, lse, dq, dk, dv, workspace, rule)
    plan = _masked_plan(q, k, v, r)
    dop, op, dqp = (_whole(t, _BF, q.shape, n) for t, n in ((dout, "dout"), (o, "o"), (dq, "dq")))
    dkp, dvp = (_whole(t, _BF, k.shape, n) for t, n in ((dk, "dk"), (dv, "dv")))
    lp = _whole(lse, _F32, plan[1], "lse")
    wp = _whole(workspace, _U8, workspace.shape, "workspace")
    _check(_lib().pf_masked_attn_bwd(plan[0], dop, q.data_ptr(), k.data_ptr(), v.data_ptr(), op, lp,
                                     *_rule_ptrs(r, plan), dqp, dkp, dvp, wp, workspace.numel(), _raw_stream(i)),
           "pf_masked_attn_bwd")


def masked_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                              lse: torch.Tensor, rule: Optional[ScoreRule] = None, *, stream=None):
    """(dq, dk, dv) of ``masked_attention`` from the gradient of its output (contiguous, as o), its inputs, and the o and
    lse that it returned; contiguous, dk and dv summed over the query heads that share a key head."""
    i = _index(q)
    if _elsewhere(i, stream):
        with _on(i, stream):
            return masked_attention_backward(dout, q, k, v, o, lse, rule)
    dq, dk, dv = _new(q), _new(k), _new(v)
    ws = torch.empty(4 * q.shape[0] * q.shape[1] * q.shape[2], dtype=_U8, device=q.device)
    pf_masked_attn_bwd(dout, q, k, v, o, lse, dq, dk, dv, ws, rule)
    return dq, dk, dv
