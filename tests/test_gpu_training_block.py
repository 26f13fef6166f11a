"""The training-direction calls together, as a block uses them: modulate, project, rotate, attend, normalise, and back."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_masked_attention import starts_of
from tests.train_util import randn

pytestmark = pytest.mark.gpu

N, C, H, KV = 330, 256, 4, 2
DOCS, PREFIX = [150, 0, 120, 31], [20, 0, 7, 31]


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


def _inputs():
    width = (H + 2 * KV) * 128
    t = {"x": randn(1, N, C), "wqkv": randn(2, width, C, scale=C ** -0.5), "wo": randn(3, C, H * 128, scale=0.05),
         "table": randn(4, 6, 2, C, dtype=torch.float32, scale=0.2), "gain": randn(5, C, dtype=torch.float32, shift=1.0, scale=0.1),
         "bias": randn(6, C, dtype=torch.float32, scale=0.1)}
    r = torch.arange(N, device="cuda")
    t["coords"] = torch.stack([r * (20 / 3), r % 7, r % 11], 1).float().contiguous()
    t["level"], t["tags"] = (r % 2).int(), (r % 3).int()
    t["dy"] = randn(7, N, C)
    t["starts"], t["prefix"] = starts_of(DOCS), torch.tensor(PREFIX, dtype=torch.int32, device="cuda")
    return t


def _ranges(h3, t):
    return h3.build_key_ranges(t["starts"], N, "prefix_causal", prefix=t["prefix"])


def _step(h3, t):
    """Forward and backward by the library's calls (the projections by torch in bf16)."""
    h = h3.adaln_modulate(t["x"], t["level"], t["tags"], t["table"])
    qkv = (h @ t["wqkv"].T).view(N, H + 2 * KV, 128)
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    qr, kr = h3.mmrope_rotate(q, k, t["coords"])
    ranges = _ranges(h3, t)
    lse = torch.empty(H, N, device="cuda")
    o = h3.masked_attention(qr, kr, v, ranges, lse=lse)
    z = o.view(N, H * 128) @ t["wo"].T
    y, mean, rstd = h3.layer_norm(z, t["gain"], t["bias"])

    dz, dgain, dbias = h3.layer_norm_backward(t["dy"], z, mean, rstd, t["gain"])
    dwo = dz.T @ o.view(N, H * 128)
    do = (dz @ t["wo"]).view(N, H, 128)
    dqkv = torch.empty_like(qkv)
    dq, dk, _ = h3.masked_attention_backward(do, qr, kr, v, o, lse, ranges, dv=dqkv[:, H + KV:])
    h3.mmrope_rotate(dq, dk, t["coords"], q_out=dqkv[:, :H], k_out=dqkv[:, H:H + KV], inverse=True)
    dwqkv = dqkv.view(N, -1).T @ h
    dh = dqkv.view(N, -1) @ t["wqkv"]
    dx, dtable = h3.adaln_modulate_backward(dh, t["x"], t["level"], t["tags"], t["table"])
    return {"y": y, "dx": dx, "dwqkv": dwqkv, "dwo": dwo, "dgain": dgain, "dbias": dbias, "dtable": dtable}


def _reference(t, ranges):
    """The same block in 64 bits, gradients by automatic differentiation."""
    f = {k: (v.double().requires_grad_() if k in ("x", "wqkv", "wo", "table", "gain", "bias") else v)
         for k, v in t.items()}

    def norm(x, eps):
        m = x.mean(-1, keepdim=True)
        return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)

    e = t["level"].long() * 3 + t["tags"].long()
    h = norm(f["x"], 1e-6) * (1 + f["table"][e, 1]) + f["table"][e, 0]
    qkv = (h @ f["wqkv"].T).view(N, H + 2 * KV, 128)
    parts = [t["coords"].double()[:, a:a + 1] * 10000.0 ** (-torch.arange(0, d, 2, device="cuda").double() / d)
             for a, d in enumerate((32, 48, 48))]
    turn = torch.polar(torch.ones(N, 64, dtype=torch.float64, device="cuda"), torch.cat(parts, 1))[:, None]

    def rotate(x):
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (64, 2)).contiguous()) * turn).flatten(-2)

    q, k = rotate(qkv[:, :H]), rotate(qkv[:, H:H + KV]).repeat_interleave(H // KV, 1)
    v = qkv[:, H + KV:].repeat_interleave(H // KV, 1)
    key = torch.arange(N, device="cuda")
    sees = (key[None] >= ranges[:, :1]) & (key[None] < ranges[:, 1:])
    s = torch.einsum("qhd,khd->hqk", q, k) * 128 ** -0.5
    p = torch.softmax(s.masked_fill(~sees, -1e300), -1) * sees
    o = torch.einsum("hqk,khd->qhd", p, v).reshape(N, H * 128)
    y = norm(o @ f["wo"].T, 1e-5) * f["gain"] + f["bias"]
    y.backward(t["dy"].double())
    return {"y": y.detach(), "dx": f["x"].grad, "dwqkv": f["wqkv"].grad, "dwo": f["wo"].grad, "dgain": f["gain"].grad,
            "dbias": f["bias"].grad, "dtable": f["table"].grad}


def test_block_against_64_bits(h3):
    """Every tensor passed on is rounded to bf16 (2^-8 relative at most, in the 2-norm about 2^-9.8): forward six
    of them in a row (h, qkv, rotation, P with O, z, y), backward seven more (dz, do, dS with dq, rotation, dh,
    dx, and the rounded operands of the forward pass again).  In the 2-norm independent roundings add up like
    sqrt(13) 2^-9.8 = 0.4 %; rows of y with no key (the padding and z = 0) have the norm of a zero row amplified by
    1 / sqrt(eps) = 316 at most, and it is exactly 0 here.  The layer norm divides by the deviation of z, whose
    relative error it keeps.  2 % leaves a factor five for correlated roundings."""
    t = _inputs()
    got = _step(h3, t)
    assert h3.h3_check_device_error() == h3.H3_OK
    want = _reference(t, _ranges(h3, t))
    for name, w in want.items():
        rel = float((got[name].double() - w).norm() / w.norm())
        assert rel <= 0.02, (name, rel)


def test_block_repeats_and_replays(h3):
    """The same bits on every run, and from a captured graph whose inputs have changed."""
    t = _inputs()
    first = _step(h3, t)
    again = _step(h3, t)
    assert all(torch.equal(first[k], again[k]) for k in first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(h3, t)                                  # library handles of torch's products
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):                                # two graphs with workspaces of their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(h3, t))
        graphs.append(g)
    t["x"].copy_(randn(21, N, C))
    for g in graphs:
        g.replay()
    want = _step(h3, t)
    for out in outs:
        assert all(torch.equal(want[k], out[k]) for k in want)


def test_prefix_rows_can_be_reused(h3):
    """Under the block-prefix mask the prefix rows' outputs do not depend on the rest, and fresh query rows against
    all keys give the rows of the whole call: K and V of a prefix are computed once."""
    n, p = 500, 180
    q, k, v = randn(1, n, H, 128), randn(2, n, KV, 128), randn(3, n, KV, 128)
    s, pre = starts_of([n]), torch.tensor([p], dtype=torch.int32, device="cuda")
    ranges = h3.build_key_ranges(s, n, "prefix_block", prefix=pre)
    whole = h3.masked_attention(q, k, v, ranges)
    fresh = h3.masked_attention(q[p:], k, v, ranges[p:].contiguous())
    alone = h3.masked_attention(q[:p], k[:p], v[:p], ranges[:p].contiguous())
    bound = 2 * 2.0 ** -8 * v.double().abs().amax()   # two roundings of the same value each
    assert float((whole[p:].double() - fresh.double()).abs().max()) <= bound
    assert float((whole[:p].double() - alone.double()).abs().max()) <= bound
    k2, v2 = k.clone(), v.clone()
    k2[p:], v2[p:] = randn(8, n - p, KV, 128), randn(9, n - p, KV, 128)
    assert torch.equal(h3.masked_attention(q, k2, v2, ranges)[:p], whole[:p])


def test_offsets_past_32_bits(h3):
    """Rows 2^30 elements apart: the last of three lies past element 2^31.  Each call gives what it gives packed."""
    apart, rows = 1 << 30, 3
    buf = torch.empty((rows - 1) * apart + 4096, dtype=torch.bfloat16, device="cuda")
    used = [0]

    def far(t):
        t = t.view(rows, -1)
        at = used[0]
        used[0] += (t.shape[1] + 7) // 8 * 8
        view = buf.as_strided((rows, t.shape[1]), (apart, 1), at)
        view.copy_(t)
        return view

    def heads(t):
        f = far(t)
        return f.as_strided((rows, f.shape[1] // 128, 128), (apart, 128, 1), f.storage_offset())

    q, do = randn(1, rows, 4, 128), randn(4, rows, 4, 128)
    k, v = randn(2, rows, 2, 128), randn(3, rows, 2, 128)
    ranges = torch.tensor([[0, 1], [0, 2], [1, 3]], dtype=torch.int32, device="cuda")
    fq, fk, fv, fdo = (heads(t) for t in (q, k, v, do))
    lse, flse = torch.empty(4, rows, device="cuda"), torch.empty(4, rows, device="cuda")
    o = h3.masked_attention(q, k, v, ranges, lse=lse)
    fo = h3.masked_attention(fq, fk, fv, ranges, out=heads(torch.zeros_like(q)), lse=flse)
    assert torch.equal(o, fo) and torch.equal(lse, flse)
    want = h3.masked_attention_backward(do, q, k, v, o, lse, ranges)
    got = h3.masked_attention_backward(fdo, fq, fk, fv, fo, flse, ranges, *(heads(torch.zeros_like(t)) for t in want))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    used[0] = 0
    fq, fk = heads(q), heads(k)
    coords = randn(5, rows, 3, dtype=torch.float32, scale=30.0)
    want = h3.mmrope_rotate(q, k, coords)
    got = h3.mmrope_rotate(fq, fk, coords, q_out=fq, k_out=fk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for c in (256, 1280):                              # a warp per row, a ring of rows
        used[0] = 0
        x, dy = randn(6, rows, c), randn(7, rows, c)
        fx, fdy = far(x), far(dy)
        y, mean, rstd = h3.layer_norm(x)
        fy, _, _ = h3.layer_norm(fx, out=far(torch.zeros_like(x)))
        assert torch.equal(y, fy)
        table = randn(8, 2, 2, c, dtype=torch.float32)
        level, tag = torch.tensor([0, 0, 0], device="cuda").int(), torch.tensor([1, 0, 1], device="cuda").int()
        want = h3.adaln_modulate_backward(dy, x, level, tag, table)
        got = h3.adaln_modulate_backward(fdy, fx, level, tag, table, dx=fy)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        want = h3.layer_norm_backward(dy, x, mean, rstd)
        got = h3.layer_norm_backward(fdy, fx, mean, rstd, dx=fdy)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert h3.h3_check_device_error() == h3.H3_OK


def test_calls_at_once_on_two_streams(h3):
    """Two blocks whose calls interleave on two streams give what they give alone."""
    t, u = _inputs(), _inputs()
    u["x"], u["dy"] = randn(31, N, C), randn(32, N, C)
    want = _step(h3, t), _step(h3, u)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    here = torch.cuda.current_stream()
    for _ in range(5):
        got = []
        for s, inputs in zip(streams, (t, u)):
            s.wait_stream(here)
            with torch.cuda.stream(s):
                got.append(_step(h3, inputs))
        for s in streams:
            here.wait_stream(s)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[k], w[k]) for k in w)
    for s in streams:
        assert h3.h3_check_device_error(s.cuda_stream) == h3.H3_OK


def test_calls_behind_other_work(h3):
    """Inputs written just before by fills, copies, torch kernels, another stream or another call, eagerly and in a
    captured graph with branches: each call waits for what precedes it."""
    n, c = 1200, 1280
    src = [randn(40 + i, n, c) for i in range(2)]
    x, dy = torch.empty_like(src[0]), torch.empty_like(src[0])
    level, tag = (torch.arange(n, device="cuda") % 7).int(), (torch.arange(n, device="cuda") % 3).int()
    table, zero = torch.empty(21, 2, c, device="cuda"), torch.zeros(21, 2, c, device="cuda")
    side = torch.cuda.Stream()

    def run():
        x.zero_()
        table.copy_(zero)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            dy.zero_()
            dy.add_(src[1])
            b = h3.layer_norm(dy)[0]
        x.copy_(src[0])
        table.add_(0.25)
        here.wait_stream(side)
        dx, dt = h3.adaln_modulate_backward(dy, x, level, tag, table)
        y, mean, rstd = h3.layer_norm(dx, out=dx)      # in place behind the call that wrote it
        g = h3.layer_norm_backward(b, y, mean, rstd, dx=b)
        q = y.view(n, 10, 128)
        qr, _ = h3.mmrope_rotate(q, None, coords, q_out=q)
        r = h3.build_key_ranges(starts, n, "prefix_causal")
        lse = torch.empty(10, n, device="cuda")
        o = h3.masked_attention(qr, qr, qr, r, lse=lse)
        return (dt, *g, o, *h3.masked_attention_backward(o, qr, qr, qr, o, lse, r))

    coords, starts = randn(44, n, 3, dtype=torch.float32), starts_of([700, 3, 497])
    torch.cuda.synchronize()
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(20):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert h3.h3_check_device_error() == h3.H3_OK


def test_single_rows_and_heads_of_larger_tensors(h3):
    """Sizes of one: their strides say nothing."""
    q, k, v = randn(1, 3, 5, 4, 128), randn(2, 3, 5, 2, 128), randn(3, 3, 5, 2, 128)
    one = torch.tensor([[0, 5]] * 3, dtype=torch.int32, device="cuda").view(3, 1, 2)
    row = h3.masked_attention(q[:, 2:3], k, v, one)    # one row of each batch entry
    for b in range(3):
        assert torch.equal(row[b], h3.masked_attention(q[b, 2:3].contiguous(), k[b], v[b], one[b]))
    x = randn(4, 7, 128).t().contiguous().t()          # [7, 128] with columns apart: refused as it is
    with pytest.raises(ValueError):
        h3.masked_attention(x[:, None], x[:, None], x[:, None], one.view(3, 2))
    y = randn(5, 7, 128)
    r = torch.tensor([[0, 7]] * 7, dtype=torch.int32, device="cuda")
    head = y.as_strided((7, 1, 128), (128, 999, 1))
    assert torch.equal(h3.masked_attention(head, head, head, r), h3.masked_attention(*[y[:, None]] * 3, r))
    empty = h3.masked_attention(q[:, :0], k, v, one[:, :0])
    assert empty.shape == (3, 0, 4, 128)


def test_views_of_one_buffer(h3):
    """Columns of one buffer as inputs and outputs of one call."""
    n = 200
    buf = torch.zeros(n, 3 * H, 128, dtype=torch.bfloat16, device="cuda")
    buf[:, :2 * H] = randn(1, n, 2 * H, 128)
    q, k, out = buf.split(H, 1)
    r = _full(n)
    want = h3.masked_attention(q.contiguous(), k.contiguous(), k.contiguous(), r)
    assert torch.equal(h3.masked_attention(q, k, k, r, out=out), want)
    with pytest.raises(h3.H3Error):
        h3.masked_attention(q, k, k, r, out=q)


def _full(n):
    return torch.tensor([[0, n]] * n, dtype=torch.int32, device="cuda")
