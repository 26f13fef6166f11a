"""Attention under one key interval per row (documents, prefixes), grouped heads, against 64-bit references."""
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import attend, check_attention, randn

pytestmark = pytest.mark.gpu

MODES = ("document", "prefix_causal", "prefix_block")


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


def starts_of(docs, first=0):
    s = [first]
    for d in docs:
        s.append(s[-1] + d)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def python_ranges(docs, prefix, n, mode, first=0):
    out = torch.zeros(n, 2, dtype=torch.int32)
    at = first
    for d, p in zip(docs, prefix):
        p = min(p, d)
        for i in range(at, at + d):
            hi = at + d
            if mode == "prefix_causal":
                hi = max(at + p, i + 1)
            elif mode == "prefix_block" and i < at + p:
                hi = at + p
            out[i, 0], out[i, 1] = at, hi
        at += d
    return out.cuda()


# (documents, prefixes, padding rows before, behind)
TABLES = [([1], [0], 0, 0), ([2, 0, 5, 1], [1, 0, 9, 1], 0, 3), ([127, 1, 128, 129], [5, 0, 128, 64], 0, 0),
          ([300, 0, 0, 213], [64, 0, 0, 213], 7, 130), ([0], [0], 0, 40), ([640], [1], 0, 0)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("docs,prefix,before,behind", TABLES)
def test_key_ranges(h3, docs, prefix, before, behind, mode):
    n = before + sum(docs) + behind
    p = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    got = h3.build_key_ranges(starts_of(docs, before), n, mode, prefix=p)
    assert torch.equal(got, python_ranges(docs, prefix, n, mode, before))
    if mode == "prefix_causal":
        none = h3.build_key_ranges(starts_of(docs, before), n, mode)
        assert torch.equal(none, python_ranges(docs, [0] * len(docs), n, mode, before))
    assert h3.h3_check_device_error() == h3.H3_OK


def test_key_ranges_bad_tables(h3):
    for bad, prefix in (([0, 5, 3, 9], [0, 0, 0]), ([-2, 4], [0]), ([0, 99], [0]), ([0, 9], [-1])):
        s = torch.tensor(bad, dtype=torch.int32, device="cuda")
        r = h3.build_key_ranges(s, 9, "prefix_causal", prefix=torch.tensor(prefix, dtype=torch.int32, device="cuda"))
        assert h3.h3_check_device_error() == h3.H3_ERR_DEVICE_INPUT
        assert int(r.min()) >= 0 and int(r.max()) <= 9
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert not h3.build_key_ranges(s, 4).any()                              # no documents at all
    assert h3.build_key_ranges(s, 0).shape == (0, 2)
    with pytest.raises(ValueError):
        h3.build_key_ranges(s, 4, "causal")
    with pytest.raises(ValueError):
        h3.build_key_ranges(s.long(), 4)
    with pytest.raises(ValueError):
        h3.build_key_ranges(s, 4, prefix=s)


def _run(h3, q, k, v, ranges, **kw):
    lse = torch.full((q.shape[-2], q.shape[0]), 3.0, device="cuda")
    o = h3.masked_attention(q, k, v, ranges, lse=lse, **kw)
    assert h3.h3_check_device_error() == h3.H3_OK
    return {"o": o, "lse": lse}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("docs,prefix,before,behind", TABLES)
@pytest.mark.parametrize("h,kv", [(2, 2), (4, 1)])
def test_forward_documents(h3, docs, prefix, before, behind, mode, h, kv):
    n = before + sum(docs) + behind
    q, k, v = randn(1, n, h, 128), randn(2, n, kv, 128), randn(3, n, kv, 128)
    ranges = python_ranges(docs, prefix, n, mode, before)
    check_attention(_run(h3, q, k, v, ranges), attend(q, k, v, ranges), ("o", "lse"))


def _intervals(nq, nk, seed):
    """Arbitrary intervals: short, long, empty, reversed, outside the keys."""
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-20, nk + 20, (nq, 2), generator=g)
    short = torch.rand(nq, generator=g) < 0.4
    a[short, 1] = a[short, 0] + torch.randint(0, 9, (int(short.sum()),), generator=g)
    return a.int().cuda().contiguous()


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 700), (3, 129), (130, 64), (256, 256), (257, 1000), (640, 1)])
def test_forward_any_intervals(h3, nq, nk):
    q, k, v = randn(1, nq, 3, 128), randn(2, nk, 3, 128), randn(3, nk, 3, 128)
    ranges = _intervals(nq, nk, nq + nk)
    check_attention(_run(h3, q, k, v, ranges), attend(q, k, v, ranges), ("o", "lse"))


def test_forward_without_keys_or_queries(h3):
    q, none = randn(1, 5, 2, 128), torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    got = _run(h3, q, none, none, torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
    assert not got["o"].any() and bool((got["lse"] == -float("inf")).all())
    k = randn(2, 9, 1, 128)
    assert h3.masked_attention(q[:0], k, k, torch.zeros(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 2, 128)


def test_forward_equals_the_unmasked_call(h3):
    """Where every row sees every key the arithmetic is that of packed_attention, bit for bit, unless several CTAs
    share a row's keys (few rows and heads, many keys: the sums are joined in another order)."""
    for n, h, shared in ((1, 3, False), (82, 3, False), (384, 3, False), (1000, 3, True), (1000, 80, False)):
        q, k, v = (randn(s, n, h, 128) for s in (1, 2, 3))
        ranges = torch.tensor([0, n], dtype=torch.int32, device="cuda").repeat(n, 1)
        lse = torch.empty(h, n, device="cuda")
        want = h3.packed_attention(q, k, v, lse=lse)
        got = _run(h3, q, k, v, ranges)
        if shared:
            check_attention(got, attend(q, k, v, ranges), ("o", "lse"))
        else:
            assert torch.equal(want, got["o"]) and torch.equal(lse, got["lse"])


@pytest.mark.parametrize("scale", [0.02, 0.5, 3.0])
def test_forward_scales(h3, scale):
    """Peaked and flat rows; with the large scale the running reference has to be raised in mid-row."""
    n = 700
    q, k, v = randn(1, n, 2, 128), randn(2, n, 2, 128), randn(3, n, 2, 128)
    ranges = python_ranges([400, 300], [100, 7], n, "prefix_causal")
    check_attention(_run(h3, q, k, v, ranges, softmax_scale=scale), attend(q, k, v, ranges, scale=scale), ("o", "lse"))


def test_forward_growing_logits(h3):
    """Keys whose logits grow along the sequence by far more than the headroom of the numerators."""
    n = 600
    q, v = randn(1, n, 1, 128), randn(3, n, 1, 128)
    k = (q[:1].double() * torch.linspace(-40, 40, n, device="cuda", dtype=torch.float64)[:, None, None]).bfloat16()
    q = q[:1].expand(n, 1, 128).contiguous()
    ranges = python_ranges([n], [0], n, "prefix_causal")
    check_attention(_run(h3, q, k, v, ranges), attend(q, k, v, ranges), ("o", "lse"))


def test_forward_strides_and_batch(h3):
    b, n, h, kv = 2, 300, 4, 2
    fused = randn(1, b, n, h + 2 * kv, 128)
    q, k, v = fused[:, :, :h], fused[:, :, h:h + kv], fused[:, :, h + kv:]
    tables = [python_ranges([n - 31], [9], n, "prefix_causal"), python_ranges([100, n - 100], [0, 0], n, "document")]
    ranges = torch.stack(tables).contiguous()
    out = torch.full((b, n, h + 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(b, h, n, device="cuda")
    h3.masked_attention(q, k, v, ranges, out=out[:, :, :h], lse=lse)
    assert bool((out[:, :, h:] == 9).all())
    for i in range(b):
        want = attend(q[i], k[i], v[i], tables[i])
        check_attention({"o": out[i, :, :h], "lse": lse[i]}, want, ("o", "lse"))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_forward_masked_places_do_not_matter(h3, what):
    """Rows of another document, padding rows and masked-out keys may hold anything, in Q, K and V."""
    docs, n = [150, 200], 400
    q, k, v = randn(1, n, 2, 128), randn(2, n, 2, 128), randn(3, n, 2, 128)
    ranges = python_ranges(docs, [0, 30], n, "prefix_causal")
    clean = _run(h3, q, k, v, ranges)
    for t in (q, k, v):
        t[360:] = what                     # padding
        t[10, 1, 5] = what                 # inside the first document, seen by its rows from 10 on
    got = _run(h3, q, k, v, ranges)
    for name, dim in (("o", 0), ("lse", 1)):
        a, c = got[name], clean[name]
        if dim == 1:
            a, c = a.T, c.T
        assert torch.equal(a[:10], c[:10]) and torch.equal(a[150:], c[150:])
        assert torch.equal(a[10:150, 0], c[10:150, 0])
    # what a row attends to is never hidden: the rows that see the key are not finite
    assert not bool(torch.isfinite(got["o"][10:150, 1]).all(-1).any())
    full = torch.tensor([0, 128], dtype=torch.int32, device="cuda").repeat(128, 1)
    o = h3.masked_attention(randn(1, 128, 2, 128), randn(2, 128, 2, 128), v[:128], full)
    assert not bool(torch.isfinite(o[:, 1]).all(-1).any()) and bool(torch.isfinite(o[:, 0]).all())


def test_forward_on_a_side_stream_and_captured(h3):
    n = 500
    q, k, v = randn(1, n, 4, 128), randn(2, n, 2, 128), randn(3, n, 2, 128)
    s = starts_of([200, 290])
    p = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    want = h3.masked_attention(q, k, v, h3.build_key_ranges(s, n, "prefix_block", prefix=p))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = h3.masked_attention(q, k, v, h3.build_key_ranges(s, n, "prefix_block", prefix=p, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = h3.masked_attention(q, k, v, h3.build_key_ranges(s, n, "prefix_block", prefix=p))
    s.copy_(starts_of([100, 400]))
    q.copy_(randn(9, n, 4, 128))
    graph.replay()
    want = h3.masked_attention(q, k, v, h3.build_key_ranges(s, n, "prefix_block", prefix=p))
    assert torch.equal(want, got)


def test_masked_binding_refuses(h3):
    q, k = randn(1, 8, 4, 128), randn(2, 9, 2, 128)
    r = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    A = h3.masked_attention
    for f in (lambda: A(q, k, k[:8], r), lambda: A(q, k[:, :1].expand(9, 3, 128).contiguous(), k, r),
              lambda: A(q, torch.cat([k, k[:, :1]], 1), torch.cat([k, k[:, :1]], 1), r),
              lambda: A(q, k, k, r[:7]), lambda: A(q, k, k, r.long()), lambda: A(q, k, k, r.cpu()),
              lambda: A(q, k, k, r, out=k), lambda: A(q, k, k, r, lse=torch.empty(8, device="cuda")),
              lambda: A(q[..., :64], k, k, r), lambda: A(q.float(), k, k, r), lambda: A(q.cpu(), k, k, r)):
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(h3.H3Error):
        A(q, k, k, r, softmax_scale=float("nan"))


@pytest.mark.parametrize("nq,nk,h,kv", [(1, 20000, 1, 1), (5, 4099, 6, 2), (300, 5000, 2, 2), (700, 1500, 4, 1),
                                        (1100, 1100, 16, 16), (2000, 2000, 20, 5)])
def test_forward_shared_walks(h3, nq, nk, h, kv):
    """Few query rows against many keys: several CTAs share a walk; parts without a visible key for a row too."""
    q, k, v = randn(1, nq, h, 128), randn(2, nk, kv, 128), randn(3, nk, kv, 128)
    full = torch.tensor([0, nk], dtype=torch.int32, device="cuda").repeat(nq, 1)
    narrow = _intervals(nq, nk, 7)
    narrow[: nq // 2, 1] = narrow[: nq // 2, 0].clamp(min=0) + 3           # three keys somewhere
    for ranges in (full, _intervals(nq, nk, nq + nk), narrow):
        got = _run(h3, q, k, v, ranges)
        check_attention(got, attend(q, k, v, ranges), ("o", "lse"))
        again = _run(h3, q, k, v, ranges)
        assert torch.equal(got["o"], again["o"]) and torch.equal(got["lse"], again["lse"])


def test_forward_shared_walks_with_bad_keys(h3):
    """As above with inf and NaN in masked places of K and V: the rows that do not see them keep their bits."""
    nq, nk = 200, 6000
    q, k, v = randn(1, nq, 2, 128), randn(2, nk, 1, 128), randn(3, nk, 1, 128)
    ranges = torch.tensor([100, 5000], dtype=torch.int32, device="cuda").repeat(nq, 1)
    ranges[77] = torch.tensor([0, 6000])
    clean = _run(h3, q, k, v, ranges)
    for t in (k, v):
        t[5100:5300] = float("nan")
        t[3, 0, 9] = float("inf")
    got = _run(h3, q, k, v, ranges)
    keep = torch.arange(nq, device="cuda") != 77
    assert torch.equal(got["o"][keep], clean["o"][keep]) and torch.equal(got["lse"][:, keep], clean["lse"][:, keep])
    assert not bool(torch.isfinite(got["o"][77]).any())
