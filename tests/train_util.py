"""64-bit references and error bounds for the training-direction and masked-attention tests.

U is the unit roundoff of fp32; half(t) that of an output type: a value rounded
to t is off by at most half(t) relative to itself.
"""
import torch

U = 2.0 ** -24


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def randn(seed, *shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype).cuda()


def within(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error "
                           f"{err[bad].max().item():.3e} against {bound[bad].min().item():.3e}")


# ------------------------------------------------------------- layer norm --

def norm_terms(x, eps):
    """xhat, mean, rstd of x [N, C] in 64 bits, and a bound on the kernel's error of xhat.

    The mean is a sum of C values: each thread adds at most 32 pairs in a row, then 1 + 5 + 3 additions
    join a row's threads and one division ends it, so it is off by at most 48 U mean|x|.  The squared
    deviations are summed alike: the variance is off by at most 52 U relative (the mean's own error enters
    squared), rstd by half of that and three roundings.  x - mean and the product round once each.
    """
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    xhat = (x - mean) * rstd
    emean = 48 * U * x.abs().mean(-1, keepdim=True)
    ex = rstd * emean + xhat.abs() * 32 * U + (rstd * emean) ** 2 * xhat.abs()
    return xhat, mean, rstd, ex


def norm_y_bound(xhat, ex, w, b, dtype):
    y = xhat * w + b
    return y, half(dtype) * y.abs() + w.abs() * ex + 2 * U * ((xhat * w).abs() + y.abs()) + 1e-300


def norm_backward(dy, x, w, eps, dtype, n_chain):
    """(dx, its bound, dw, its bound, db, its bound) per row weight w [N, C] or [C]; n_chain: additions
    in the longest chain of a column sum."""
    xhat, _, rstd, ex = norm_terms(x, eps)
    dy = dy.double()
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xhat).mean(-1, keepdim=True)
    dx = (g - c1 - xhat * c2) * rstd
    e1 = 50 * U * g.abs().mean(-1, keepdim=True)
    e2 = 52 * U * (g * xhat).abs().mean(-1, keepdim=True) + (g.abs() * ex).mean(-1, keepdim=True)
    inner = 4 * U * (g.abs() + c1.abs() + (xhat * c2).abs()) + e1 + xhat.abs() * e2 + ex * c2.abs() + ex * e2
    bound = half(dtype) * dx.abs() + rstd * inner + 40 * U * dx.abs()
    dw, db = dy * xhat, dy
    chain = (n_chain + 60) * U
    return (dx, bound, dw, dw.abs() * chain + dy.abs() * ex, db, db.abs() * chain)


# -------------------------------------------------------------- attention --

def attend(q, k, v, ranges, scale=None, do=None, chunk_heads=8):
    """64-bit attention of one batch entry: q [Nq, H, D], k, v [Nk, Hkv, D], ranges [Nq, 2].

    Only the keys inside a row's interval enter, whatever the others hold.  Returns a dict with o, lse and
    their bounds, and with do also dq, dk, dv and theirs.

    Bounds.  A logit is a sum of 128 products accumulated in fp32 and scaled: off by at most
    es = 300 U scale sum|q k| + 4 U |logit|, which moves P by es relative (2 es covers the normaliser).  P is
    rounded to bf16 as an MMA operand (half(bf16) relative), the product is accumulated in fp32
    (128 U and less per tile, below 2^-14 over any length tested) and O is rounded once more.
    """
    h16, acc = half(torch.bfloat16), 2.0 ** -14
    nq, heads, d = q.shape
    nk, kv = k.shape[0], k.shape[1]
    group = heads // kv
    scale = d ** -0.5 if scale is None else scale
    key = torch.arange(nk, device=q.device)
    lo, hi = ranges[:, :1].clamp(min=0), ranges[:, 1:].clamp(max=nk)
    sees = (key[None] >= lo) & (key[None] < hi)
    out = {n: torch.zeros(nq, heads, d, dtype=torch.float64, device=q.device) for n in ("o", "eo", "dq", "edq")}
    out.update({n: torch.zeros(nk, kv, d, dtype=torch.float64, device=q.device) for n in ("dk", "edk", "dv", "edv")})
    out["lse"] = torch.full((heads, nq), -float("inf"), dtype=torch.float64, device=q.device)
    out["else"] = torch.zeros(heads, nq, dtype=torch.float64, device=q.device)
    used = sees.any(0)[:, None]
    for h in range(heads):
        qq = q[:, h].double()
        kk = torch.where(used, k[:, h // group].double(), 0.0)
        vv = torch.where(used, v[:, h // group].double(), 0.0)
        live = sees.any(1)
        qq = torch.where(live[:, None], qq, 0.0)
        s = torch.where(sees, qq @ kk.T * scale, -float("inf"))
        es = torch.where(sees, 300 * U * scale * (qq.abs() @ kk.abs().T) + 4 * U * (qq @ kk.T * scale).abs(), 0.0)
        es = es.amax(1, keepdim=True) if nk else torch.zeros(nq, 1, dtype=torch.float64, device=q.device)
        m = s.amax(1, keepdim=True) if nk else torch.full((nq, 1), -float("inf"), dtype=torch.float64, device=q.device)
        m = torch.where(live[:, None], m, 0.0)
        p = torch.exp(s - m)
        total = p.sum(1, keepdim=True)
        p = torch.where(live[:, None], p / torch.where(total == 0, 1.0, total), 0.0)
        out["lse"][h] = torch.where(live, (m + torch.log(total))[:, 0], -float("inf"))
        out["else"][h] = 2 * es[:, 0] + 2.0 ** -20 * (1 + torch.where(live, out["lse"][h].abs(), 0.0))
        o = p @ vv
        rel = h16 + acc + 2 * es
        eo = rel * (p @ vv.abs())
        out["o"][:, h], out["eo"][:, h] = o, eo + h16 * o.abs()
        if do is None:
            continue
        dd = torch.where(live[:, None], do[:, h].double(), 0.0)
        dp = dd @ vv.T
        edp = 300 * U * (dd.abs() @ vv.abs().T)
        delta = (dd * o).sum(1, keepdim=True)
        # delta comes from the rounded O, whose error enters every dS of the row; for rows of at most 32 keys
        # from P and dP in fp32 (an approximate exp2, sums of 32 terms)
        edelta = (dd.abs() * (eo + h16 * o.abs())).sum(1, keepdim=True) + 40 * U * (dd * o).abs().sum(1, keepdim=True)
        few = (p * (edp + (2 * es + 2.0 ** -20) * dp.abs())).sum(1, keepdim=True)
        edelta = torch.where(sees.sum(1, keepdim=True) <= 32, few, edelta)
        ds = p * (dp - delta)
        eds = p * (edp + edelta + (2 * es + 4 * U) * (dp - delta).abs()) + (h16 + acc) * ds.abs()
        dq, edq = ds @ kk * scale, eds @ kk.abs() * scale
        out["dq"][:, h], out["edq"][:, h] = dq, edq + h16 * dq.abs()
        out["dk"][:, h // group] += ds.T @ qq * scale
        out["edk"][:, h // group] += eds.T @ qq.abs() * scale
        out["dv"][:, h // group] += p.T @ dd
        out["edv"][:, h // group] += (rel * p).T @ dd.abs()
    out["edk"] += h16 * out["dk"].abs()
    out["edv"] += h16 * out["dv"].abs()
    return out


def check_attention(got, want, names):
    for n in names:
        g, w, e = got[n], want[n], want["e" + n]
        if n == "lse":
            empty = torch.isinf(w)
            assert torch.equal(torch.isinf(g), empty) and bool((g[empty] < 0).all()), "rows without keys: lse"
            g, w, e = g[~empty], w[~empty], e[~empty]
        within(g, w, e + 1e-30, n)
