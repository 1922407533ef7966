"""The block's operators as they are used together: layer norm with one shift and scale per image, a projection, the
QK norm with rotary positions, attention under a score rule, and the same way back to x and every weight.

The exact chain is torch's own differentiation in fp64.  A second chain goes through the formulas in fp64 and rounds to
bf16 at every place where the kernels round (each stage's output, p and ds inside the attention).

Tolerance.  The kernels' error and the second chain's are two draws of the same roundings (those before the first sum
agree in nearly all elements, so the draws are alike rather than independent); what the kernels add is fp32's, 2^-16 of
a bf16 rounding per operation.  Over a whole tensor (at least 2^9 elements, most 2^15) the norms of two such draws differ by a
few per cent; 1.5 of the second chain's norm is allowed.  One token's row, 64 elements or more, may have 3 times its own
error there plus the tensor's mean row error: a row's norm spreads by 1 / sqrt(2 * 64) = 9%, and rows whose leading
roundings cancel are covered by the mean.
"""
import os
import subprocess
import sys
import threading

import pytest
import torch

import patch_attention_b200 as pa
from tests.test_gpu_masked_attention import slopes

pytestmark = pytest.mark.gpu

BF, F64 = torch.bfloat16, torch.float64
B, N, C, HQ, HK, D, EPS = 2, 200, 256, 4, 2, 64, 1e-6
AXES = pa.RopeAxes((16, 24, 24), theta=10000.0)


def _params(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return {
        "x": r(B, N, C).to(BF), "mod": (0.2 * r(B, 2, C)).to(BF), "w": (r(C, (HQ + 2 * HK) * D) / C ** 0.5).to(BF),
        "gq": (1 + 0.1 * r(D)).to(BF), "gk": (1 + 0.1 * r(D)).to(BF), "do": r(B, N, HQ, D).to(BF),
    }


def _pos():
    i = torch.arange(N, device="cuda", dtype=torch.float32)
    return torch.stack([i // 50, (i // 10) % 5, i % 10], -1).expand(B, N, 3).contiguous()


def _rule(kind):
    if kind == "documents":
        d = torch.zeros(B, N, device="cuda", dtype=torch.int32)
        d[0, 70:] = 1
        d[0, 131:] = 2
        d[1, 5:] = 4
        d[1, 180:] = -1  # padding
        return pa.ScoreRule(doc_q=d, doc_k=d)
    if kind == "prefix":
        p = torch.tensor([0, 64], device="cuda", dtype=torch.int32)
        return pa.ScoreRule(causal=True, prefix=p, softcap=5.0, slopes=slopes(HQ))
    return pa.ScoreRule()


def _split(t):
    return t[:, :, :HQ], t[:, :, HQ:HQ + HK], t[:, :, HQ + HK:]


def _run(p, pos, rule):
    """Both directions through the public calls; the projection and its gradients are torch's."""
    shift, scale = p["mod"][:, 0], p["mod"][:, 1]
    h, mean, rstd = pa.layernorm(p["x"], scale, shift, weight_offset=1.0, eps=EPS, want_stats=True)
    qkv = (h @ p["w"]).view(B, N, HQ + 2 * HK, D)
    q0, k0, v = _split(qkv)
    q, k = pa.qk_norm_rope(q0, k0, pos, AXES, gain_q=p["gq"], gain_k=p["gk"], eps=EPS)
    o, lse = pa.masked_attention(q, k, v, rule, want_lse=True)
    dq, dk, dv = pa.masked_attention_backward(p["do"], q, k, v, o, lse, rule)
    dq0, dk0, dgq, dgk = pa.qk_norm_rope_backward(dq, dk, q0, k0, pos, AXES, gain_q=p["gq"], gain_k=p["gk"], eps=EPS)
    dqkv = torch.cat([dq0, dk0, dv], 2).view(B, N, -1)
    dh = dqkv @ p["w"].t()
    dw = h.view(B * N, C).t() @ dqkv.view(B * N, -1)
    dx, dscale, dshift = pa.layernorm_backward(dh, p["x"], scale, mean, rstd, weight_offset=1.0, bias_like=shift)
    return {"o": o, "dx": dx, "dscale": dscale, "dshift": dshift, "dw": dw, "dgq": dgq, "dgk": dgk}


def _turns(pos):
    out = []
    for a, w in enumerate(AXES.dims):
        f = AXES.theta[a] ** (-2.0 * torch.arange(w // 2, device="cuda", dtype=F64) / w)
        out.append(pos[..., a:a + 1].double() * f)
    return torch.cat(out, -1)[:, :, None]  # [B, N, 1, D / 2]


def _rotate(z, t):
    """Neighbouring elements form the pairs, and the axes follow one another."""
    a, b = z[..., 0::2], z[..., 1::2]
    return torch.stack([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1).flatten(-2)


def _hidden(rule):
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")[None]
    ok = torch.ones(B, N, N, dtype=torch.bool, device="cuda")
    if rule.causal:
        ok &= (j <= i)[None] | (j[None] < rule.prefix[:, None, None])
    if rule.doc_q is not None:
        ok &= (rule.doc_q[:, :, None] == rule.doc_k[:, None]) & (rule.doc_k[:, None] >= 0)
    return ~ok[:, None], -(i - j).abs().double()


def _scores(q, k, rule, away):
    """Capped and biased scores and the cap's derivative; k has as many heads as q."""
    s = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
    t = torch.tanh(s / rule.softcap) if rule.softcap else torch.zeros_like(s)
    s = rule.softcap * t if rule.softcap else s
    if rule.slopes is not None:
        s = s + rule.slopes.double()[None, :, None, None] * away
    return s, 1 - t * t


def _softmax(s, hidden):
    s = s.masked_fill(hidden, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m.isinf(), 0.0, m)).masked_fill(hidden, 0.0)
    n = p.sum(-1, keepdim=True)
    return p / torch.where(n == 0, 1.0, n)


def _forward(p, pos, rule, r):
    shift, scale = p["mod"][:, 0, None], p["mod"][:, 1, None]
    x = p["x"]
    xh = (x - x.mean(-1, keepdim=True)) * (x.var(-1, correction=0, keepdim=True) + EPS).rsqrt()
    h = r(xh * (1 + scale) + shift)
    q0, k0, v = _split(r(h @ p["w"]).view(B, N, HQ + 2 * HK, D))
    norm = lambda z, g: z * (z.square().mean(-1, keepdim=True) + EPS).rsqrt() * g  # noqa: E731
    t = _turns(pos)
    q, k = r(_rotate(norm(q0, p["gq"]), t)), r(_rotate(norm(k0, p["gk"]), t))
    hidden, away = _hidden(rule)
    wide = lambda z: z.repeat_interleave(HQ // HK, 2)  # noqa: E731
    s, damp = _scores(q, wide(k), rule, away)
    P = _softmax(s, hidden)
    o = r(torch.einsum("bhij,bjhd->bihd", r(P), wide(v)))
    return o, (xh, h, q0, k0, v, q, k, t, P, damp)


def _exact(p, pos, rule):
    p = {n: v.double().requires_grad_(n != "do") for n, v in p.items()}
    o, _ = _forward(p, pos, rule, lambda t: t)
    o.backward(p["do"])
    return {"o": o.detach(), "dx": p["x"].grad, "dscale": p["mod"].grad[:, 1], "dshift": p["mod"].grad[:, 0],
            "dw": p["w"].grad, "dgq": p["gq"].grad, "dgk": p["gk"].grad}


def _by_formula(p, pos, rule, r):
    p = {n: v.double() for n, v in p.items()}
    o, (xh, h, q0, k0, v, q, k, t, P, damp) = _forward(p, pos, rule, r)
    do, scale = p["do"], p["mod"][:, 1, None]
    wide = lambda z: z.repeat_interleave(HQ // HK, 2)  # noqa: E731
    heads = lambda z: z.view(B, N, HK, HQ // HK, D).sum(3)  # noqa: E731
    dv = r(heads(torch.einsum("bhij,bihd->bjhd", r(P), do)))
    dp = torch.einsum("bihd,bjhd->bhij", do, wide(v))
    ds = r(P * (dp - (o * do).sum(-1).transpose(1, 2)[..., None]) * damp)
    dq = r(torch.einsum("bhij,bjhd->bihd", ds, wide(k)) * D ** -0.5)
    dk = r(heads(torch.einsum("bhij,bihd->bjhd", ds, q)) * D ** -0.5)

    def norm_back(dy, z, g):
        dz = _rotate(dy, -t)
        rs = (z.square().mean(-1, keepdim=True) + EPS).rsqrt()
        zh, a = z * rs, dz * g
        return r(rs * (a - zh * (a * zh).mean(-1, keepdim=True))), r((dz * zh).sum((0, 1, 2)))

    dq0, dgq = norm_back(dq, q0, p["gq"])
    dk0, dgk = norm_back(dk, k0, p["gk"])
    dqkv = torch.cat([dq0, dk0, dv], 2).view(B, N, -1)
    dh = r(dqkv @ p["w"].t())
    dw = r(h.view(B * N, C).t() @ dqkv.view(B * N, -1))
    a = dh * (1 + scale)
    rs = (p["x"].var(-1, correction=0, keepdim=True) + EPS).rsqrt()
    dx = r(rs * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True)))
    return {"o": o, "dx": dx, "dscale": r((dh * xh).sum(1)), "dshift": r(dh.sum(1)), "dw": dw, "dgq": dgq, "dgk": dgk}


def _round(t):
    return t.to(BF).double()


@pytest.mark.parametrize("kind", ["all", "documents", "prefix"])
def test_both_directions(kind):
    p, pos, rule = _params(1), _pos(), _rule(kind)
    exact = _exact(p, pos, rule)
    again = _by_formula(p, pos, rule, lambda t: t)
    rounded = _by_formula(p, pos, rule, _round)
    got = _run(p, pos, rule)
    torch.cuda.synchronize()
    pa.pf_device_status()
    for name, want in exact.items():
        # the formulas themselves: fp64 sums of at most 2^16 terms
        assert (again[name] - want).norm() <= 1e-10 * want.norm(), name
        err, ref = got[name].double() - want, rounded[name] - want
        assert got[name].shape == want.shape
        assert err.norm() <= 1.5 * ref.norm(), (name, float(err.norm() / ref.norm()))
        if name in ("o", "dx"):
            e, f = err.reshape(B * N, -1).norm(dim=1), ref.reshape(B * N, -1).norm(dim=1)
            assert bool((e <= 3 * (f + f.mean())).all()), (name, float((e / (f + f.mean())).max()))
    if kind == "documents":  # padded tokens: no output, and nothing comes back through their attention
        assert not got["o"][1, 180:].any() and not got["dx"][1, 180:].any()


def test_captured_replayed_and_on_another_stream():
    """One graph of both directions, replayed after its inputs changed and between eager runs, gives the eager bits."""
    pos, rule = _pos(), _rule("documents")
    a, b = _params(2), _params(3)
    eager_a, eager_b = _run(a, pos, rule), _run(b, pos, rule)
    live = {n: t.clone() for n, t in a.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = _run(live, pos, rule)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(live, pos, rule)
    for source, want in ((a, eager_a), (b, eager_b), (a, eager_a)):
        for n, t in source.items():
            live[n].copy_(t)
        graph.replay()
        now = _run(source, pos, rule)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]) and torch.equal(now[n], want[n]), n
    for n, t in eager_a.items():
        assert torch.equal(there[n], t), n


def test_two_graphs_and_two_streams_at_once():
    """Two captured blocks replayed side by side on two streams keep apart."""
    pos, rule = _pos(), _rule("prefix")
    ps = [_params(4), _params(5)]
    want = [_run(p, pos, rule) for p in ps]
    graphs, outs = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_run(p, pos, rule))
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for n in w:
            assert torch.equal(o[n], w[n]), n


def test_gradients_right_before_the_patch_attention():
    """The patch attention reads its inputs as soon as it may start.  A backward call without parameter gradients
    launches no second kernel, and with none to give way to it must hold the patch call back until its end."""
    rows, c = 400_000, 256
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(rows, c, device="cuda", generator=g).to(BF) for _ in range(2))
    mean, rstd = torch.zeros(2, rows, device="cuda").unbind()
    rstd += 1
    dx = torch.empty_like(x)
    pos = torch.arange(rows, device="cuda", dtype=torch.float32)[:, None]
    axes = pa.RopeAxes((64,))
    heads = x.view(1, rows, 4, 64)
    pat = pa.PatchAttention(1, 4, 64, 1024, 4, 0, 1)
    whole = x[:1024].view(1, 1024, 4, 64)
    try:
        for kind in ("norm", "rope"):
            outs = []
            for wait in (True, False, False, False):
                pat.init_layer(0, whole, whole)
                dx.zero_()
                torch.cuda.synchronize()
                if kind == "norm":
                    pa.pf_layernorm_bwd(dy, x, None, 1.0, mean, rstd, dx, None, None, None)
                else:
                    pa.pf_qk_norm_rope_bwd(dy.view(heads.shape), None, heads, None, pos, axes, dx.view(heads.shape), None,
                                           None, None, 1e-6, None, None, None)
                last = dx[-256:].view(1, 256, 4, 64)
                if wait:
                    torch.cuda.synchronize()
                outs.append(pat.step(0, 0, last, last, last).clone())
                torch.cuda.synchronize()
                pat.check()
            assert outs[0].any()
            for o in outs[1:]:
                assert torch.equal(o, outs[0]), kind
    finally:
        pat.close()


FIRST_CALLS = """
import torch
from tests.test_gpu_block import _params, _pos, _rule, _run
p, pos, rule = _params(7), _pos(), _rule("documents")
torch.cuda.synchronize()
torch.randn(8, 8, device="cuda") @ torch.randn(8, 8, device="cuda")  # torch's own library is not what is looked at
p["x"][0] @ p["w"], p["x"][0].t() @ p["x"][0], p["x"] @ p["w"]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = _run(p, pos, rule)
graph.replay()
torch.cuda.synchronize()
want = _run(p, pos, rule)
assert all(torch.equal(out[n], want[n]) for n in want)
print("equal")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


def test_four_host_threads_with_a_stream_each():
    pos, rule = _pos(), _rule("documents")
    ps = [_params(8 + i) for i in range(4)]
    want = [_run(p, pos, rule) for p in ps]
    torch.cuda.synchronize()
    same = {}

    def go(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = _run(ps[i], pos, rule)
            stream.synchronize()
            same[i] = all(torch.equal(got[n], want[i][n]) for n in got)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == {0: True, 1: True, 2: True, 3: True}
