"""Cases of the training-side operators of the packed block, in plain torch and as library calls.

Four groups of operators, each one pass through which a training or serving program calls:

* attention under a mask that gives each query row one interval of keys (documents packed
  into one sequence, prefix masks), grouped heads, forward and forward + backward;
* layer norm with weight and bias, forward and forward + backward;
* the backward pass of the per-row AdaLN modulation, with its table's gradient;
* the three-axis rotation of Q and K with grouped heads, forward and backward.

``listed()`` names the fixed cases, ``draw()`` gives more of the same ranges, ``prepare()``
makes the inputs on the GPU, ``run()`` is one pass (plain torch in fp32, or with ``own`` the
library's calls), ``exact()`` the same values in 64 bits.
"""
import math

import torch

own = False

HEAD_DIM = 128
MODES = ("document", "prefix_causal", "prefix_block")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SECTIONS = (32, 48, 48)
THETA = 10000.0


def _h3():
    import packed_mm_rope_b200
    return packed_mm_rope_b200


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # three tiny requests share the 82-row sequence of the smallest workload: launch latency
        {"name": "attend 82 rows", "op": "attention", "train": False, "mode": "document", "docs": "30,1,51",
         "prefix": "0,0,0", "pad": 0, "heads": 1, "kv_heads": 1},
        # serving: requests of uneven length in one packed sequence (a 4,584-row clip among them)
        {"name": "attend documents", "op": "attention", "train": False, "mode": "document",
         "docs": "4584,82,2292,0,701", "prefix": "0,0,0,0,0", "pad": 1, "heads": 8, "kv_heads": 8},
        # reference rows as a prefix that the rest attends to and that does not look back at it
        {"name": "attend block prefix grouped", "op": "attention", "train": False, "mode": "prefix_block",
         "docs": "4096,3564", "prefix": "1201,880", "pad": 0, "heads": 8, "kv_heads": 2},
        # training on short samples, causal behind each prefix, a padded tail and an empty document
        {"name": "train causal prefix small", "op": "attention", "train": True, "mode": "prefix_causal",
         "docs": "513,0,129,458", "prefix": "16,0,0,7", "pad": 27, "heads": 8, "kv_heads": 8},
        # training on two long samples, one third of the 42 heads (one rank's share), grouped 7 to 1
        {"name": "train documents large", "op": "attention", "train": True, "mode": "document",
         "docs": "9001,5097", "prefix": "0,0", "pad": 0, "heads": 14, "kv_heads": 2},
        # the worked example's rows through a norm with weight and bias
        {"name": "layer norm forward", "op": "layer_norm", "train": False, "rows": 28196, "hidden": 5376,
         "dtype": "bf16", "params": "fp32"},
        # a small odd head of a model, in 32 bits
        {"name": "layer norm train odd", "op": "layer_norm", "train": True, "rows": 82, "hidden": 129,
         "dtype": "fp32", "params": "fp32"},
        # one training step's norm at the worked example
        {"name": "layer norm train", "op": "layer_norm", "train": True, "rows": 28196, "hidden": 5376,
         "dtype": "bf16", "params": "fp32"},
        # the small workload, its rows shuffled over two noise levels and three modalities
        {"name": "adaln backward shuffled", "op": "adaln", "rows": 4584, "hidden": 5376, "levels": 2,
         "shuffled": True},
        # the worked example: rows in runs of one modality, one noise level per latent frame
        {"name": "adaln backward frames", "op": "adaln", "rows": 28196, "hidden": 5376, "levels": 31,
         "shuffled": False},
        # serving: a small clip with grouped heads
        {"name": "rotate grouped", "op": "rotate", "rows": 4584, "heads": 8, "kv_heads": 2, "inverse": False,
         "pair_layout": 0},
        # gradients of Q and K at the worked example
        {"name": "rotate back", "op": "rotate", "rows": 28196, "heads": 42, "kv_heads": 42, "inverse": True,
         "pair_layout": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "layer_norm", "layer_norm", "adaln", "rotate"])
    if op == "attention":
        train = rng.random() < 0.5
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 3, 4])
        most = int(math.sqrt(14098.0 ** 2 * 14 / heads))
        # a gradient needs a document of some length: over one key the softmax has none
        rows = _log_int(rng, 80 if train else 1, min(most, 14098))
        docs, left = [], rows
        if train or rng.random() < 0.7:
            docs.append(max(1, int(rows * rng.uniform(0.5, 0.95))))
            left -= docs[0]
        while left > 0 and len(docs) < 40:
            n = min(left, rng.choice([0, 1, 2, rng.randint(1, max(1, left)), rng.randint(1, max(1, left))]))
            docs.append(n)
            left -= n
        if left:
            docs.append(left)
        rng.shuffle(docs)
        mode = rng.choice(MODES)
        prefix = [0 if mode == "document" else rng.choice([0, 1, rng.randint(0, max(0, n)), n]) for n in docs]
        return {"op": "attention", "train": train, "mode": mode, "docs": ",".join(map(str, docs)),
                "prefix": ",".join(map(str, prefix)), "pad": rng.choice([0, 0, 1, rng.randint(1, 200)]),
                "heads": heads, "kv_heads": kv}
    if op == "layer_norm":
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 8 * 8)
        rows = _log_int(rng, 1, max(1, min(100000, 28196 * 5376 // hidden)))
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if dtype == "fp32":
            rows = max(1, rows // 2)
        return {"op": "layer_norm", "train": rng.random() < 0.6, "rows": rows, "hidden": hidden, "dtype": dtype,
                "params": rng.choice(["fp32", dtype])}
    if op == "adaln":
        hidden = max(64, _log_int(rng, 64, 8192) // 8 * 8)
        rows = _log_int(rng, 1, max(1, min(81792, 28196 * 5376 // hidden)))
        return {"op": "adaln", "rows": rows, "hidden": hidden, "levels": _log_int(rng, 1, 200),
                "shuffled": rng.random() < 0.5}
    kv = rng.choice([1, 2, 5, 8, 14])
    heads = kv * rng.choice([1, 2, 3])
    rows = _log_int(rng, 1, max(1, min(81792, 28196 * 84 // (heads + kv))))
    return {"op": "rotate", "rows": rows, "heads": heads, "kv_heads": kv, "inverse": rng.random() < 0.5,
            "pair_layout": rng.choice([0, 1])}


# ----------------------------------------------------------------- inputs --

def _ints(text):
    return [int(x) for x in text.split(",")]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "attention":
        docs = _ints(case["docs"])
        n = sum(docs) + case["pad"]
        starts = [0]
        for d in docs:
            starts.append(starts[-1] + d)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["prefix"] = torch.tensor(_ints(case["prefix"]), dtype=torch.int32, device="cuda")
        for name, h in (("q", case["heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
            st[name] = _randn(g, n, h, HEAD_DIM)
        if case["train"]:
            st["do"] = _randn(g, n, case["heads"], HEAD_DIM)
        return st
    if case["op"] == "layer_norm":
        n, c, dt, pt = case["rows"], case["hidden"], DTYPES[case["dtype"]], DTYPES[case["params"]]
        st["x"] = _randn(g, n, c, dtype=dt, scale=1.5, shift=0.25)
        st["weight"] = _randn(g, c, dtype=pt, scale=0.2, shift=1.0)
        st["bias"] = _randn(g, c, dtype=pt, scale=0.2)
        if case["train"]:
            st["dy"] = _randn(g, n, c, dtype=dt)
        return st
    if case["op"] == "adaln":
        n, c, levels = case["rows"], case["hidden"], case["levels"]
        st["x"] = _randn(g, n, c, scale=1.5, shift=0.25)
        st["dy"] = _randn(g, n, c)
        st["table"] = torch.randn(3 * levels, 2, c, generator=g, device="cuda") * 0.3
        # runs: one text stretch, then `levels` latent frames, then audio; shuffled: any order
        r = torch.arange(n, device="cuda")
        text, audio = n // 50, n - n // 40
        tags = torch.where(r < text, 0, torch.where(r < audio, 1, 2))
        level = ((r - text).clamp(min=0) * levels // max(1, audio - text)).clamp(max=levels - 1)
        if case["shuffled"]:
            perm = torch.randperm(n, generator=g, device="cuda")
            tags, level = tags[perm], level[perm]
        st["level"], st["tags"] = level.to(torch.int32).contiguous(), tags.to(torch.int32).contiguous()
        return st
    n = case["rows"]
    st["q"] = _randn(g, n, case["heads"], HEAD_DIM)
    st["k"] = _randn(g, n, case["kv_heads"], HEAD_DIM)
    # text at (i, i, i), then latent frames of 44 x 80 patches cut to 22 x 40, 20/3 units apart
    r = torch.arange(n, device="cuda")
    text = min(n, 200)
    cell = (r - text).clamp(min=0)
    frame, y, x = cell // 880, cell % 880 // 40, cell % 40
    first = torch.randint(-6000, 1, (1,), generator=g, device="cuda")
    t = torch.where(r < text, r.double(), (first + 20 * frame).double() / 3.0)
    hh = torch.where(r < text, r, y)
    ww = torch.where(r < text, r, x)
    st["coords"] = torch.stack([t, hh.double(), ww.double()], 1).float().contiguous()
    return st


# -------------------------------------------------------------- attention --

def _ranges(st, n):
    """Per row the interval [lo, hi) of keys that its mask leaves."""
    starts, prefix = st["starts"].long(), st["prefix"].long()
    r = torch.arange(n, device=starts.device)
    doc = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    inside = (doc < prefix.numel()) & (r >= starts[0])
    doc = doc.clamp(max=prefix.numel() - 1)
    lo, end = starts[doc], starts[doc + 1]
    p = torch.minimum(lo + prefix[doc], end)
    if st["mode"] == "document":
        hi = end
    elif st["mode"] == "prefix_causal":
        hi = torch.maximum(p, r + 1)
    else:
        hi = torch.where(r < p, p, end)
    zero = torch.zeros_like(lo)
    return torch.where(inside, lo, zero), torch.where(inside, hi, zero)


def _plain_attention(st):
    q, k, v = (st[x].float().transpose(0, 1) for x in ("q", "k", "v"))
    group = q.shape[0] // k.shape[0]
    n = q.shape[1]
    lo, hi = _ranges(st, n)
    key = torch.arange(n, device=q.device)
    hidden = (key[None, :] < lo[:, None]) | (key[None, :] >= hi[:, None])
    scale = HEAD_DIM ** -0.5
    kx, vx = k.repeat_interleave(group, 0), v.repeat_interleave(group, 0)
    p = torch.matmul(q, kx.transpose(1, 2)).mul_(scale).masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p, vx)
    out = {"o": o.transpose(0, 1).to(torch.bfloat16).contiguous(), "lse": lse}
    if st["train"]:
        do = st["do"].float().transpose(0, 1)
        delta = (do * o).sum(-1, keepdim=True)
        dv = torch.matmul(p.transpose(1, 2), do)
        ds = torch.matmul(do, vx.transpose(1, 2)).sub_(delta).mul_(p).mul_(scale)
        dq = torch.matmul(ds, kx)
        dk = torch.matmul(ds.transpose(1, 2), q)
        dk = dk.view(-1, group, n, HEAD_DIM).sum(1)
        dv = dv.view(-1, group, n, HEAD_DIM).sum(1)
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            out[name] = t.transpose(0, 1).to(torch.bfloat16).contiguous()
    return out


def _own_attention(st):
    h3 = _h3()
    n, h = st["q"].shape[0], st["heads"]
    ranges = h3.build_key_ranges(st["starts"], n, mode=st["mode"], prefix=st["prefix"])
    lse = torch.empty(h, n, dtype=torch.float32, device="cuda")
    o = h3.masked_attention(st["q"], st["k"], st["v"], ranges, lse=lse)
    out = {"o": o, "lse": lse}
    if st["train"]:
        out["dq"], out["dk"], out["dv"] = h3.masked_attention_backward(st["do"], st["q"], st["k"], st["v"], o, lse,
                                                                       ranges)
    return out


# ------------------------------------------------------------- layer norm --

LN_EPS = 1e-5


def _plain_layer_norm(st):
    x, w, b = st["x"].float(), st["weight"].float(), st["bias"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + LN_EPS)
    xhat = xc * rstd
    out = {"y": (xhat * w + b).to(st["x"].dtype)}
    if not st["train"]:
        return {**out, "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    dy = st["dy"].float()
    g = dy * w
    c1 = g.mean(-1, keepdim=True)
    c2 = (g * xhat).mean(-1, keepdim=True)
    out["dx"] = ((g - c1 - xhat * c2) * rstd).to(st["x"].dtype)
    out["dweight"] = (dy * xhat).sum(0).to(st["weight"].dtype)
    out["dbias"] = dy.sum(0).to(st["bias"].dtype)
    return out


def _own_layer_norm(st):
    h3 = _h3()
    y, mean, rstd = h3.layer_norm(st["x"], st["weight"], st["bias"], eps=LN_EPS)
    if not st["train"]:
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = h3.layer_norm_backward(st["dy"], st["x"], mean, rstd, st["weight"])
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


# ------------------------------------------------------------------ AdaLN --

ADALN_EPS = 1e-6


def _plain_adaln(st):
    x, dy = st["x"].float(), st["dy"].float()
    e = st["level"].long() * 3 + st["tags"].long()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + ADALN_EPS)
    xhat = xc * rstd
    g = dy * (1.0 + st["table"][:, 1][e])
    dx = (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd
    rows_of = (e[None, :] == torch.arange(st["table"].shape[0], device=e.device)[:, None]).float()
    dtable = torch.stack([rows_of @ dy, rows_of @ (dy * xhat)], 1)
    return {"dx": dx.to(st["x"].dtype), "dtable": dtable}


def _own_adaln(st):
    dx, dtable = _h3().adaln_modulate_backward(st["dy"], st["x"], st["level"], st["tags"], st["table"],
                                               eps=ADALN_EPS)
    return {"dx": dx, "dtable": dtable}


# --------------------------------------------------------------- rotation --

def _inv_freq(device):
    f = [torch.pow(torch.tensor(THETA, dtype=torch.float64, device=device),
                   -2.0 * torch.arange(d // 2, dtype=torch.float64, device=device) / d) for d in SECTIONS]
    axis = torch.repeat_interleave(torch.arange(3, device=device),
                                   torch.tensor([d // 2 for d in SECTIONS], device=device))
    return torch.cat(f), axis


def _plain_rotate(st):
    inv, axis = _inv_freq(st["q"].device)
    angle = st["coords"].double()[:, axis] * inv
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if st["inverse"]:
        sin = -sin

    def turn(x):
        f = x.float()
        if st["pair_layout"] == 0:
            a, b = f[..., 0::2], f[..., 1::2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = f[..., :64], f[..., 64:]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return y.to(torch.bfloat16)

    return {"q": turn(st["q"]), "k": turn(st["k"])}


def _own_rotate(st):
    q, k = _h3().mmrope_rotate(st["q"], st["k"], st["coords"], inverse=st["inverse"],
                               pair_layout=st["pair_layout"])
    return {"q": q, "k": k}


# -------------------------------------------------------------- one pass --

def run(state):
    op = state["op"]
    if own:
        return {"attention": _own_attention, "layer_norm": _own_layer_norm, "adaln": _own_adaln,
                "rotate": _own_rotate}[op](state)
    return {"attention": _plain_attention, "layer_norm": _plain_layer_norm, "adaln": _plain_adaln,
            "rotate": _plain_rotate}[op](state)


def work(case):
    if case["op"] == "attention":
        docs, prefix = _ints(case["docs"]), _ints(case["prefix"])
        n, h, kv = sum(docs) + case["pad"], case["heads"], case["kv_heads"]
        pairs = 0
        for d, p in zip(docs, prefix):
            p = min(p, d)
            if case["mode"] == "document":
                pairs += d * d
            elif case["mode"] == "prefix_causal":
                pairs += p * p + (d * (d + 1) - p * (p + 1)) // 2
            else:
                pairs += p * p + (d - p) * d
        row = 2 * HEAD_DIM
        size = n * row * (2 * h + 2 * kv) + 4 * n * h       # q, k, v in, o and the log-sum-exp out
        if case["train"]:
            size += n * row * (2 * h + 2 * kv)              # do in, dq, dk, dv out
        return {"bytes": size, "flops": (14 if case["train"] else 4) * HEAD_DIM * h * pairs}
    if case["op"] == "layer_norm":
        n, c = case["rows"], case["hidden"]
        b = 4 if case["dtype"] == "fp32" else 2
        if case["train"]:
            return {"bytes": 4 * n * c * b, "flops": 20 * n * c}
        return {"bytes": 2 * n * c * b + 8 * n, "flops": 8 * n * c}
    if case["op"] == "adaln":
        n, c = case["rows"], case["hidden"]
        return {"bytes": 6 * n * c + 8 * n + 36 * case["levels"] * c, "flops": 20 * n * c}
    n = case["rows"]
    return {"bytes": n * (case["heads"] + case["kv_heads"]) * 512 + 12 * n,
            "flops": 3 * n * (case["heads"] + case["kv_heads"]) * HEAD_DIM}


# ---------------------------------------------------------------- 64 bits --

def _exact_attention(case, st):
    """Document by document and head by head: rows of different documents never meet."""
    docs, prefix = _ints(case["docs"]), _ints(case["prefix"])
    n, heads, group = sum(docs) + case["pad"], case["heads"], case["heads"] // case["kv_heads"]
    if n * n * heads > 14098 ** 2 * 14:
        return None
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    o = torch.zeros_like(q)
    lse = torch.full((heads, n), -math.inf, dtype=torch.float64, device=q.device)
    if case["train"]:
        do = st["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    first = 0
    for length, pre in zip(docs, prefix):
        rows = slice(first, first + length)
        first += length
        if length == 0:
            continue
        i = torch.arange(length, device=q.device)
        sees = torch.ones(length, length, dtype=torch.bool, device=q.device)
        if case["mode"] == "prefix_causal":
            sees = (i[None, :] <= i[:, None]) | (i[None, :] < pre)
        elif case["mode"] == "prefix_block":
            sees = (i[None, :] < pre) | (i[:, None] >= pre)
        for h in range(heads):
            g = h // group
            logits = (q[rows, h] @ k[rows, g].T) / math.sqrt(HEAD_DIM)
            logits[~sees] = -math.inf
            lse[h, rows] = torch.logsumexp(logits, -1)
            p = torch.exp(logits - lse[h, rows][:, None])
            o[rows, h] = p @ v[rows, g]
            if case["train"]:
                dv[rows, g] += p.T @ do[rows, h]
                dp = do[rows, h] @ v[rows, g].T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(HEAD_DIM)
                dq[rows, h] = ds @ k[rows, g]
                dk[rows, g] += ds.T @ q[rows, h]
    out = {"o": o, "lse": lse}
    if case["train"]:
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _exact_norm(x, eps):
    x = x.double()
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    return (x - mean) * rstd, mean, rstd


def _exact_norm_dx(g, xhat, rstd):
    c = xhat.shape[-1]
    return (c * g - g.sum(-1, keepdim=True) - xhat * (g * xhat).sum(-1, keepdim=True)) * rstd / c


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, st)
    if case["op"] == "layer_norm":
        xhat, mean, rstd = _exact_norm(st["x"], LN_EPS)
        w, b = st["weight"].double(), st["bias"].double()
        out = {"y": torch.addcmul(b, xhat, w)}
        if not case["train"]:
            return {**out, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        dy = st["dy"].double()
        out["dx"] = _exact_norm_dx(dy * w, xhat, rstd)
        out["dweight"], out["dbias"] = torch.einsum("nc,nc->c", dy, xhat), dy.sum(0)
        return out
    if case["op"] == "adaln":
        xhat, _, rstd = _exact_norm(st["x"], ADALN_EPS)
        dy, table = st["dy"].double(), st["table"].double()
        e = (st["level"] * 3 + st["tags"]).long()
        dx = _exact_norm_dx(dy * (1.0 + table[e, 1]), xhat, rstd)
        dtable = torch.zeros_like(table)
        for i in torch.unique(e).tolist():
            rows = e == i
            dtable[i, 0] = dy[rows].sum(0)
            dtable[i, 1] = (dy[rows] * xhat[rows]).sum(0)
        return {"dx": dx, "dtable": dtable}
    parts, c = [], st["coords"].double()
    for a, d in enumerate(SECTIONS):
        j = torch.arange(0, d, 2, dtype=torch.float64, device=c.device)
        parts.append(c[:, a:a + 1] / THETA ** (j / d))
    turn = torch.cat(parts, 1) * (-1.0 if case["inverse"] else 1.0)
    phase = torch.polar(torch.ones_like(turn), turn)[:, None]

    def rotated(x):
        x = x.double()
        if case["pair_layout"] == 0:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (64, 2)).contiguous()) * phase).flatten(-2)
        y = torch.complex(x[..., :64], x[..., 64:]) * phase
        return torch.cat([y.real, y.imag], -1)

    return {"q": rotated(st["q"]), "k": rotated(st["k"])}
