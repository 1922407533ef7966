"""Workloads of the transformer-block operators around the patch attention.

Three operators of a diffusion transformer's block, each for inference and for a training
pass (forward and backward):

  ln    layer normalisation with an affine or a per-sample (scale, shift) modulation,
        y = x^ (weight + offset) + bias, and its gradients dx, dweight, dbias
  rope  per-head RMS normalisation of queries and keys followed by a rotary embedding over
        several position axes (time, height, width), and its gradients dx, dgain
  attn  attention over capped, distance-biased and masked scores (documents of a packed
        sequence, a causal mask with a fully visible prefix), and dq, dk, dv

`run` computes them in plain torch operations, or (`own`) through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the text stream's affine norm: 154 tokens, one of the shortest calls of a block
        dict(name="ln_text", kind="ln", batch=1, rows=154, channels=1536, dtype="bf16", mod=False, train=False),
        # modulated norm of both guidance halves of a 128x128-token image
        dict(name="ln_mod_image", kind="ln", batch=2, rows=16384, channels=1536, dtype="bf16", mod=True, train=False),
        # modulated norm of a fine-tuning batch of 64x64-token images, with its gradients
        dict(name="ln_mod_train", kind="ln", batch=4, rows=4096, channels=1152, dtype="bf16", mod=True, train=True),
        # affine norm in 32 bits with an odd width: no row starts on a 16-byte boundary
        dict(name="ln_odd_train", kind="ln", batch=1, rows=8191, channels=1153, dtype="fp32", mod=False, train=True),
        # one new token per sequence (a class or register token): launch latency
        dict(name="rope_one_token", kind="rope", batch=2, tokens=1, heads_q=24, heads_k=24, head_dim=128,
             axes="16,56,56", interleaved=True, norm=True, dtype="bf16", train=False),
        # one patch of a 256x256-token image
        dict(name="rope_patch", kind="rope", batch=1, tokens=4096, heads_q=24, heads_k=24, head_dim=128,
             axes="16,56,56", interleaved=True, norm=True, dtype="bf16", train=False),
        # a video clip with half-split pairs, with the gradients
        dict(name="rope_video_train", kind="rope", batch=1, tokens=16384, heads_q=24, heads_k=24, head_dim=64,
             axes="16,24,24", interleaved=False, norm=True, dtype="bf16", train=True),
        # a causal prompt encoder over one short prompt
        dict(name="attn_prompt", kind="attn", batch=1, n_q=154, n_k=154, heads_q=24, heads_kv=24, head_dim=64,
             softcap=0.0, bias=False, causal=True, prefix=False, docs=0, train=False),
        # one query token per sequence against a long cache with shared key heads
        dict(name="attn_one_token", kind="attn", batch=8, n_q=1, n_k=16538, heads_q=24, heads_kv=8, head_dim=128,
             softcap=0.0, bias=False, causal=True, prefix=False, docs=0, train=False),
        # several images of different sizes packed into one sequence, padded at its end
        dict(name="attn_packed", kind="attn", batch=1, n_q=16538, n_k=16538, heads_q=24, heads_kv=24, head_dim=64,
             softcap=0.0, bias=False, causal=False, prefix=False, docs=3, train=False),
        # capped scores with a distance bias and a visible prefix
        dict(name="attn_prefix_cap_bias", kind="attn", batch=2, n_q=4216, n_k=4216, heads_q=16, heads_kv=16,
             head_dim=72, softcap=30.0, bias=True, causal=True, prefix=True, docs=0, train=False),
        # fine-tuning on packed sequences with shared key heads
        dict(name="attn_packed_train", kind="attn", batch=1, n_q=4216, n_k=4216, heads_q=24, heads_kv=8,
             head_dim=128, softcap=0.0, bias=False, causal=False, prefix=False, docs=2, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ln", "rope", "attn"])
    train = rng.random() < 0.5
    if kind == "ln":
        c = _log_int(rng, 16, 4096)
        if rng.random() < 0.6:
            c = max(8, c // 8 * 8)
        case = dict(kind="ln", batch=rng.randint(1, 4), rows=_log_int(rng, 1, 16384), channels=c,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), mod=rng.random() < 0.5, train=train)
        while case["batch"] * case["rows"] * case["channels"] > 2 * 16384 * 1536 // 2:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    if kind == "rope":
        axes, d = rng.choice([("16,56,56", 128), ("16,24,24", 64), ("36,36", 72), ("64,64", 128), ("24,20,20", 64),
                              ("64", 72), ("8,28,28", 64), ("44,42,42", 128)])
        h = rng.randint(1, 24)
        case = dict(kind="rope", batch=rng.randint(1, 4), tokens=_log_int(rng, 1, 16384), heads_q=h,
                    heads_k=rng.choice([h, max(1, h // 3), 1]), head_dim=d, axes=axes,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), train=train)
        while case["batch"] * case["tokens"] * h * d > 16384 * 24 * 64:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    hkv = rng.choice([1, 2, 4, 8, 12])
    n_k = _log_int(rng, 1, 16538)
    causal = rng.random() < 0.5
    form = rng.choice(["one", "few", "square", "square"])
    n_q = {"one": 1, "few": min(n_k, rng.randint(2, 200)), "square": n_k}[form]
    docs = rng.choice([0, 0, 2, 5]) if n_k >= 16 and form == "square" else 0
    case = dict(kind="attn", batch=rng.randint(1, 4), n_q=n_q, n_k=n_k, heads_q=hkv * rng.choice([1, 1, 2, 3]),
                heads_kv=hkv, head_dim=rng.choice([64, 72, 128]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                bias=rng.random() < 0.3, causal=causal, prefix=causal and rng.random() < 0.5, docs=docs, train=train)
    limit = 24 * 4216 * 4216 if train else 12 * 16538 * 16538
    while case["batch"] * case["heads_q"] * case["n_q"] * case["n_k"] > limit:
        case["n_k"] = max(16, case["n_k"] * 3 // 4)
        case["n_q"] = min(case["n_q"], case["n_k"]) if form != "square" else case["n_k"]
    return case


# ------------------------------------------------------------------ inputs


def _axes(case):
    return tuple(int(a) for a in case["axes"].split(","))


def _doc_lengths(case):
    """Tokens of each document, then of the padding at the end (not attended, attends nothing)."""
    n, d = case["n_k"], case["docs"]
    pad = n // 50 + 1
    weights = [1.0 + 0.61803 * ((3 * i) % 5) for i in range(d)]
    lens = [max(1, int((n - pad) * w / sum(weights))) for w in weights]
    return lens, n - sum(lens)


def _prefix(case):
    return [min(case["n_k"], case["n_k"] // 3 + 7 * b) for b in range(case["batch"])]


def _positions(case, dev):
    """Token positions on each axis: a (time, height, width) grid walked in row-major order, from a token
    inside it on; a single axis counts tokens."""
    t = torch.arange(case["tokens"], device=dev) + 4096
    side = 64
    grid = [t // (side * side), t // side % side, t % side]
    n = len(_axes(case))
    return torch.stack(grid[3 - n:] if n > 1 else [t], dim=-1).to(torch.float32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, device=dev, generator=g).to(dtype)

    s = dict(case=case)
    if case["kind"] == "ln":
        dt, b, r, c = DTYPES[case["dtype"]], case["batch"], case["rows"], case["channels"]
        # a residual stream: channels with offsets and scales of their own
        s["x"] = (rand(b, r, c) * (0.5 + rand(c).abs()) + rand(c)).to(dt)
        if case["mod"]:
            mod = (0.3 * rand(b, 3, c)).to(dt)  # shift, scale, gate from one projection
            s["bias"], s["weight"], s["offset"] = mod[:, 0], mod[:, 1], 1.0
        else:
            s["weight"], s["bias"], s["offset"] = (1 + 0.2 * rand(c)).to(dt), (0.2 * rand(c)).to(dt), 0.0
        if case["train"]:
            s["dy"] = rand(b, r, c, dtype=dt)
        return s
    if case["kind"] == "rope":
        dt, b, n, d = DTYPES[case["dtype"]], case["batch"], case["tokens"], case["head_dim"]
        s["q"], s["k"] = rand(b, n, case["heads_q"], d, dtype=dt), rand(b, n, case["heads_k"], d, dtype=dt)
        s["pos"] = _positions(case, dev)
        s["gain_q"] = (1 + 0.2 * rand(d)).to(dt) if case["norm"] else None
        s["gain_k"] = (1 + 0.2 * rand(d)).to(dt) if case["norm"] else None
        if case["train"]:
            s["dq"], s["dk"] = rand(b, n, case["heads_q"], d, dtype=dt), rand(b, n, case["heads_k"], d, dtype=dt)
        return s
    bf, b, d = torch.bfloat16, case["batch"], case["head_dim"]
    s["q"] = rand(b, case["n_q"], case["heads_q"], d, dtype=bf)
    s["k"], s["v"] = rand(b, case["n_k"], case["heads_kv"], d, dtype=bf), rand(b, case["n_k"], case["heads_kv"], d, dtype=bf)
    h = case["heads_q"]
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=dev) if case["bias"] else None
    s["prefix"] = torch.tensor(_prefix(case), device=dev, dtype=torch.int32) if case["prefix"] else None
    s["doc"] = None
    if case["docs"]:
        lens, pad = _doc_lengths(case)
        ids = torch.repeat_interleave(torch.tensor(list(range(len(lens))) + [-1]), torch.tensor(lens + [pad]))
        s["doc"] = ids.to(torch.int32).to(dev).expand(b, -1).contiguous()
    if case["train"]:
        s["do"] = rand(b, case["n_q"], h, d, dtype=bf)
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    if own:
        return _run_own(state)
    return {"ln": _plain_ln, "rope": _plain_rope, "attn": _plain_attn}[state["case"]["kind"]](state)


def _run_own(s):
    import patch_attention_b200 as pa

    case = s["case"]
    if case["kind"] == "ln":
        if not case["train"]:
            return pa.layernorm(s["x"], s["weight"], s["bias"], weight_offset=s["offset"], eps=EPS)
        y, mean, rstd = pa.layernorm(s["x"], s["weight"], s["bias"], weight_offset=s["offset"], eps=EPS,
                                     want_stats=True)
        dx, dw, db = pa.layernorm_backward(s["dy"], s["x"], s["weight"], mean, rstd, weight_offset=s["offset"])
        return dict(y=y, dx=dx, dw=dw, db=db)
    if case["kind"] == "rope":
        axes = pa.RopeAxes(_axes(case), theta=THETA, interleaved=case["interleaved"])
        eps = EPS if case["norm"] else None
        q, k = pa.qk_norm_rope(s["q"], s["k"], s["pos"], axes, gain_q=s["gain_q"], gain_k=s["gain_k"], eps=eps)
        if not case["train"]:
            return dict(q=q, k=k)
        dq, dk, dgq, dgk = pa.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], axes,
                                                    gain_q=s["gain_q"], gain_k=s["gain_k"], eps=eps)
        out = dict(q=q, k=k, dq=dq, dk=dk)
        if case["norm"]:
            out.update(dgq=dgq, dgk=dgk)
        return out
    rule = pa.ScoreRule(softcap=case["softcap"], slopes=s["slopes"], causal=case["causal"], prefix=s["prefix"],
                        doc_q=s["doc"], doc_k=s["doc"])
    if not case["train"]:
        return pa.masked_attention(s["q"], s["k"], s["v"], rule)
    o, lse = pa.masked_attention(s["q"], s["k"], s["v"], rule, want_lse=True)
    dq, dk, dv = pa.masked_attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse, rule)
    return dict(o=o, dq=dq, dk=dk, dv=dv)


def _plain_ln(s):
    case, x = s["case"], s["x"]
    w, b = s["weight"].float(), s["bias"].float()
    if case["mod"]:
        w, b = w[:, None], b[:, None]
    w = w + s["offset"]
    xf = x.float()
    xc = xf - xf.mean(-1, keepdim=True)
    rstd = torch.rsqrt(xc.square().mean(-1, keepdim=True) + EPS)
    xh = xc * rstd
    y = (xh * w + b).to(x.dtype)
    if not case["train"]:
        return y
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    dims = 1 if case["mod"] else (0, 1)
    # sums over thousands of rows, held in 64 bits
    dw, db = (dy * xh).sum(dims, dtype=torch.float64), dy.sum(dims, dtype=torch.float64)
    return dict(y=y, dx=dx.to(x.dtype), dw=dw.to(s["weight"].dtype), db=db.to(s["weight"].dtype))


def _angles(case, pos):
    """cos and sin of every pair's angle, [tokens, 1, pairs], from 64-bit angles; pairs past the axes turn by 0."""
    parts = [pos[:, a:a + 1].double() * THETA ** (-torch.arange(0, w, 2, device=pos.device, dtype=torch.float64) / w)
             for a, w in enumerate(_axes(case))]
    ang = torch.cat(parts, -1)
    return ang.cos().float()[:, None], ang.sin().float()[:, None]


def _pair_index(case, dev):
    """First and second element of every rotated pair."""
    first, second, base = [], [], 0
    for w in _axes(case):
        i = torch.arange(w // 2, device=dev)
        first.append(base + (2 * i if case["interleaved"] else i))
        second.append(base + (2 * i + 1 if case["interleaved"] else i + w // 2))
        base += w
    return torch.cat(first), torch.cat(second)


def _turn(x, cos, sin, i0, i1):
    y = x.clone()
    y[..., i0] = x[..., i0] * cos - x[..., i1] * sin
    y[..., i1] = x[..., i0] * sin + x[..., i1] * cos
    return y


def _plain_rope(s):
    case = s["case"]
    cos, sin = _angles(case, s["pos"])
    i0, i1 = _pair_index(case, s["pos"].device)
    out = {}
    for name in ("q", "k"):
        x, gain = s[name].float(), s["gain_" + name]
        xh, z = x, x
        if case["norm"]:
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            xh = x * r
            z = xh * gain.float()
        out[name] = _turn(z, cos, sin, i0, i1).to(s[name].dtype)
        if case["train"]:
            dz = _turn(s["d" + name].float(), cos, -sin, i0, i1)
            if case["norm"]:
                out["dg" + name] = (dz * xh).sum((0, 1, 2), dtype=torch.float64).to(gain.dtype)
                g = dz * gain.float()
                dz = r * (g - xh * (g * xh).mean(-1, keepdim=True))
            out["d" + name] = dz.to(s[name].dtype)
    return out


def _plain_attn(s):
    case = s["case"]
    b, n_q, n_k, h, hk, d = (case[k] for k in ("batch", "n_q", "n_k", "heads_q", "heads_kv", "head_dim"))
    scale = d ** -0.5
    q = s["q"].float().transpose(1, 2)
    k = s["k"].float().transpose(1, 2).repeat_interleave(h // hk, 1)
    v = s["v"].float().transpose(1, 2).repeat_interleave(h // hk, 1)
    x = (q * scale) @ k.transpose(-1, -2)
    t = None
    if case["softcap"]:
        x.div_(case["softcap"]).tanh_()
        t = x.clone() if case["train"] else None
        x.mul_(case["softcap"])
    i = torch.arange(n_q, device=x.device)[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device=x.device)[None]
    if case["bias"]:
        x.sub_(s["slopes"][:, None, None] * (i - j).abs())
    hidden = torch.zeros(1, 1, n_q, n_k, dtype=torch.bool, device=x.device)
    if case["causal"]:
        seen = (j <= i)[None, None]
        if s["prefix"] is not None:
            seen = seen | (j < s["prefix"][:, None, None])[:, None]
        hidden = hidden | ~seen
    if s["doc"] is not None:
        doc = s["doc"]
        hidden = hidden | ((doc[:, :, None] != doc[:, None]) | (doc < 0)[:, :, None])[:, None]
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = x.sum(-1, keepdim=True)
    p = x.div_(torch.where(z == 0, 1.0, z))
    o = p @ v
    out = o.transpose(1, 2).to(torch.bfloat16).contiguous()
    if not case["train"]:
        return out
    do = s["do"].float().transpose(1, 2)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if t is not None:
        ds.mul_(1 - t.square())
    dq, dk = (ds @ k) * scale, (ds.transpose(-1, -2) @ q) * scale

    def shared(a):  # the query heads of a key head add up
        return a.view(b, hk, h // hk, n_k, d).sum(2).transpose(1, 2).to(torch.bfloat16).contiguous()

    return dict(o=out, dq=dq.transpose(1, 2).to(torch.bfloat16).contiguous(), dk=shared(dk), dv=shared(dv))


# ------------------------------------------------------------------ what a pass cannot do without


def _visible_pairs(case):
    """(query, key) pairs of one head that the masks leave, over the batch."""
    n_q, n_k = case["n_q"], case["n_k"]
    if case["docs"]:
        lens, _ = _doc_lengths(case)
        per = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return per * case["batch"]  # a prefix only adds pairs inside one document: not counted
    if not case["causal"]:
        return n_q * n_k * case["batch"]
    total = 0
    for p in (_prefix(case) if case["prefix"] else [0] * case["batch"]):
        first = n_k - n_q + 1  # keys that query 0 sees; one more for each further query
        if p <= first:
            total += n_q * (first + n_k) // 2
        else:
            total += p * (p - first) + (p + n_k) * (n_k - p + 1) // 2
    return total


def work(case):
    if case["kind"] == "ln":
        e = SIZES[case["dtype"]]
        n = case["batch"] * case["rows"] * case["channels"]
        p = case["channels"] * (case["batch"] if case["mod"] else 1)
        if not case["train"]:
            return {"bytes": 2 * n * e + 2 * p * e, "flops": 8 * n}
        return {"bytes": 4 * n * e + 4 * p * e, "flops": 22 * n}
    if case["kind"] == "rope":
        e = SIZES[case["dtype"]]
        n = case["batch"] * case["tokens"] * (case["heads_q"] + case["heads_k"]) * case["head_dim"]
        pos = case["tokens"] * len(_axes(case)) * 4
        return {"bytes": (4 if case["train"] else 2) * n * e + pos, "flops": (20 if case["train"] else 8) * n}
    d, b = case["head_dim"], case["batch"]
    q, kv = b * case["n_q"] * case["heads_q"] * d * 2, b * case["n_k"] * case["heads_kv"] * d * 2
    pairs = _visible_pairs(case) * case["heads_q"]
    if not case["train"]:
        return {"bytes": 2 * q + 2 * kv, "flops": 4 * d * pairs}
    return {"bytes": 4 * q + 4 * kv, "flops": 14 * d * pairs}


# ------------------------------------------------------------------ 64-bit definitions


def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "rope": _exact_rope, "attn": _exact_attn}[case["kind"]](case, s)


def _exact_ln(case, s):
    x = s["x"].double()
    n = x.shape[-1]
    w, b = s["weight"].double() + s["offset"], s["bias"].double()
    shape = (x.shape[0], 1, n) if case["mod"] else (1, 1, n)
    w, b = w.reshape(shape), b.reshape(shape)
    mean = x.sum(-1, keepdim=True) / n
    var = (x - mean).pow(2).sum(-1, keepdim=True) / n
    sigma = (var + EPS).sqrt()
    y = (x - mean) / sigma * w + b
    if not case["train"]:
        return y
    dy = s["dy"].double()
    # through the mean and the deviation: dL/dsigma, then dL/dvar, dL/dmean
    gx = dy * w
    dsigma = -(gx * (x - mean)).sum(-1, keepdim=True) / sigma.pow(2)
    dvar = dsigma / (2 * sigma)
    dmean = -gx.sum(-1, keepdim=True) / sigma
    dx = gx / sigma + 2 * dvar * (x - mean) / n + dmean / n
    over = [1] if case["mod"] else [0, 1]
    return dict(y=y, dx=dx, dw=(dy * (x - mean) / sigma).sum(over), db=dy.sum(over))


def _exact_rope(case, s):
    pos = s["pos"].double()
    d = case["head_dim"]
    # one orthogonal matrix per token: y = R z, dz = R^T dy, in slices of tokens
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        gain = s["gain_" + name].double() if case["norm"] else torch.ones(d, dtype=torch.float64, device=x.device)
        norm = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() if case["norm"] else torch.ones_like(x[..., :1])
        z = x / norm * gain
        ys, gs = [], []
        for t in range(0, case["tokens"], 1024):
            rot = torch.eye(d, dtype=torch.float64, device=x.device).repeat(min(1024, case["tokens"] - t), 1, 1)
            base = 0
            for a, w in enumerate(_axes(case)):
                for i in range(w // 2):
                    e, f = (base + 2 * i, base + 2 * i + 1) if case["interleaved"] else (base + i, base + i + w // 2)
                    phi = pos[t:t + 1024, a] / THETA ** (2 * i / w)
                    rot[:, e, e], rot[:, f, f] = phi.cos(), phi.cos()
                    rot[:, e, f], rot[:, f, e] = -phi.sin(), phi.sin()
                base += w
            ys.append(torch.einsum("nij,bnhj->bnhi", rot, z[:, t:t + 1024]))
            if case["train"]:
                gs.append(torch.einsum("nji,bnhj->bnhi", rot, s["d" + name][:, t:t + 1024].double()))
        out[name] = torch.cat(ys, 1)
        if case["train"]:
            dz = torch.cat(gs, 1)
            dx = dz
            if case["norm"]:
                out["dg" + name] = (dz * x / norm).flatten(0, 2).sum(0)
                dn = -(dz * gain * x).sum(-1, keepdim=True) / norm.pow(2)
                dx = dz * gain / norm + dn * x / (norm * d)
            out["d" + name] = dx
    return out


def _exact_attn(case, s):
    b, n_q, n_k, h, hk, d = (case[k] for k in ("batch", "n_q", "n_k", "heads_q", "heads_kv", "head_dim"))
    o = torch.zeros(b, n_q, h, d, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk = torch.zeros(b, n_k, hk, d, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    at = torch.arange(n_k - n_q, n_k, device="cuda").unsqueeze(1)
    key = torch.arange(n_k, device="cuda").unsqueeze(0)
    for bi in range(b):
        ok = torch.ones(n_q, n_k, dtype=torch.bool, device="cuda")
        if case["causal"]:
            ok &= key <= at
            if s["prefix"] is not None:
                ok |= key < s["prefix"][bi]
        if s["doc"] is not None:
            ok &= (s["doc"][bi].unsqueeze(1) == s["doc"][bi].unsqueeze(0)) & (s["doc"][bi] >= 0).unsqueeze(1)
        some = ok.any(1)
        for hi in range(h):
            q, k, v = s["q"][bi, :, hi].double(), s["k"][bi, :, hi * hk // h].double(), s["v"][bi, :, hi * hk // h].double()
            raw = q.mm(k.t()) / math.sqrt(d)
            score = case["softcap"] * torch.tanh(raw / case["softcap"]) if case["softcap"] else raw
            slope = 1.0
            if case["softcap"] and case["train"]:
                slope = 1 - (score / case["softcap"]).pow(2)
            if case["bias"]:
                score = score - s["slopes"][hi].double() * (key - at).abs()
            score = score.masked_fill(~ok, -math.inf)
            score[~some] = 0.0
            p = torch.softmax(score, -1) * some.unsqueeze(1)
            o[bi, :, hi] = p.mm(v)
            if case["train"]:
                do = s["do"][bi, :, hi].double()
                dp = do.mm(v.t())
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * slope / math.sqrt(d)
                dq[bi, :, hi] = ds.mm(k)
                dk[bi, :, hi * hk // h] += ds.t().mm(q)
                dv[bi, :, hi * hk // h] += p.t().mm(do)
    return dict(o=o, dq=dq, dk=dk, dv=dv) if case["train"] else o
