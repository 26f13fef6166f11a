"""Gradients of the masked attention against 64-bit references (formula and differences)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_masked_attention import MODES, TABLES, _intervals, python_ranges
from tests.train_util import attend, check_attention, randn

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv")


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


def _grads(h3, do, q, k, v, ranges, **kw):
    lse = torch.empty(q.shape[-2], q.shape[0], device="cuda")
    o = h3.masked_attention(q, k, v, ranges, lse=lse, **kw)
    got = dict(zip(NAMES, h3.masked_attention_backward(do, q, k, v, o, lse, ranges, **kw)))
    assert h3.h3_check_device_error() == h3.H3_OK
    return got


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("docs,prefix,before,behind", TABLES)
@pytest.mark.parametrize("h,kv", [(2, 2), (4, 1)])
def test_documents(h3, docs, prefix, before, behind, mode, h, kv):
    n = before + sum(docs) + behind
    q, k, v, do = randn(1, n, h, 128), randn(2, n, kv, 128), randn(3, n, kv, 128), randn(4, n, h, 128)
    ranges = python_ranges(docs, prefix, n, mode, before)
    check_attention(_grads(h3, do, q, k, v, ranges), attend(q, k, v, ranges, do=do), NAMES)


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 700), (3, 129), (130, 64), (256, 256), (257, 1000), (640, 1)])
def test_any_intervals(h3, nq, nk):
    q, do = randn(1, nq, 6, 128), randn(4, nq, 6, 128)
    k, v = randn(2, nk, 3, 128), randn(3, nk, 3, 128)
    ranges = _intervals(nq, nk, nq + nk)
    check_attention(_grads(h3, do, q, k, v, ranges), attend(q, k, v, ranges, do=do), NAMES)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("h,kv,heads_like", [(2, 2, False), (6, 2, True)])
def test_rows_of_few_keys(h3, mode, h, kv, heads_like):
    """Documents around 32 rows, where O's rounding does not enter the gradients; values with a common part
    (a mean of 3), which makes dO.O large beside dP - D."""
    docs = [1, 20, 32, 33, 2, 31, 64, 7, 16, 100, 3]
    n = sum(docs) + 5
    q, k, v, do = randn(1, n, h, 128), randn(2, n, kv, 128), randn(3, n, kv, 128), randn(4, n, h, 128)
    v, do = (v.float() + 3).to(v.dtype), (do.float() + 3).to(do.dtype)
    if heads_like:                                     # views of one buffer, rows further apart
        q, k, v = torch.cat([q, k, v], 1).split([h, kv, kv], 1)
    ranges = python_ranges(docs, [min(5, d) for d in docs], n, mode, 2)
    check_attention(_grads(h3, do, q, k, v, ranges), attend(q, k, v, ranges, do=do), NAMES)


@pytest.mark.parametrize("scale", [0.02, 0.5])
def test_scales(h3, scale):
    n = 700
    q, k, v, do = (randn(s, n, 2, 128) for s in (1, 2, 3, 4))
    ranges = python_ranges([400, 300], [100, 7], n, "prefix_causal")
    check_attention(_grads(h3, do, q, k, v, ranges, softmax_scale=scale),
                    attend(q, k, v, ranges, scale=scale, do=do), NAMES)


def test_gradients_match_differences(h3):
    """sum(dO * O) changes along a direction as the gradients say: differences of the 64-bit forward form."""
    n, h, kv = 200, 4, 2
    q, k, v, do = randn(1, n, h, 128), randn(2, n, kv, 128), randn(3, n, kv, 128), randn(4, n, h, 128)
    ranges = python_ranges([120, 60], [11, 60], n, "prefix_causal")
    got = _grads(h3, do, q, k, v, ranges)
    bounds = attend(q, k, v, ranges, do=do)

    def loss(q_, k_, v_):
        return (do.double() * attend(q_, k_, v_, ranges)["o"]).sum()

    args = [q.double(), k.double(), v.double()]
    step = 1e-4
    for i, name in enumerate(NAMES):
        d = randn(20 + i, *args[i].shape, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        diff = (loss(*up) - loss(*down)) / (2 * step)
        # the elements' own bounds, and step^2 / 6 times third derivatives (below 1e3 here: |d| ~ 10 per row)
        slack = (bounds["e" + name] * d.abs()).sum() + 1e-4
        assert abs(diff - (got[name].double() * d).sum()) <= slack


def test_without_keys_or_queries(h3):
    q, k = randn(1, 5, 2, 128), randn(2, 9, 1, 128)
    none_k, none_q = k[:0], q[:0]
    r = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    lse = torch.full((2, 5), -float("inf"), device="cuda")
    dq, dk, dv = h3.masked_attention_backward(q, q, none_k, none_k, q, lse, r)
    assert not dq.any() and dk.shape == (0, 1, 128)
    dq, dk, dv = h3.masked_attention_backward(none_q, none_q, k, k, none_q, lse[:, :0].contiguous(), r[:0])
    assert not dk.any() and not dv.any() and dq.shape == (0, 2, 128)
    dq, dk, dv = h3.masked_attention_backward(q, q, k, k, q, lse, r)          # rows that see nothing
    assert not dq.any() and not dk.any() and not dv.any()


def test_strides_batch_and_untouched_columns(h3):
    b, n, h, kv = 2, 300, 4, 2
    fused = randn(1, b, n, h + 2 * kv, 128)
    q, k, v = fused[:, :, :h], fused[:, :, h:h + kv], fused[:, :, h + kv:]
    do = randn(2, b, n, h + 1, 128)[:, :, :h]
    tables = [python_ranges([n - 31], [9], n, "prefix_causal"), python_ranges([100, n - 100], [0, 0], n, "document")]
    ranges = torch.stack(tables).contiguous()
    lse = torch.empty(b, h, n, device="cuda")
    out = torch.empty(b, n, h + 2, 128, dtype=torch.bfloat16, device="cuda")[:, :, :h]
    h3.masked_attention(q, k, v, ranges, out=out, lse=lse)
    grad = torch.full((b, n, h + 2 * kv + 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    h3.masked_attention_backward(do, q, k, v, out, lse, ranges, dq=grad[:, :, :h], dk=grad[:, :, h:h + kv],
                                 dv=grad[:, :, h + kv:h + 2 * kv])
    assert bool((grad[:, :, -1] == 9).all())
    for i in range(b):
        got = {"dq": grad[i, :, :h], "dk": grad[i, :, h:h + kv], "dv": grad[i, :, h + kv:h + 2 * kv]}
        check_attention(got, attend(q[i], k[i], v[i], tables[i], do=do[i]), NAMES)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_masked_places_do_not_matter(h3, what):
    """Padding rows and another document's rows may hold anything, in Q, K, V and dO; attended ones are not hidden."""
    docs, n = [150, 200], 400
    q, k, v, do = (randn(s, n, 2, 128) for s in (1, 2, 3, 4))
    ranges = python_ranges(docs, [0, 30], n, "prefix_causal")
    clean = _grads(h3, do, q, k, v, ranges)
    for t in (q, k, v, do):
        t[360:] = what
    got = _grads(h3, do, q, k, v, ranges)
    for name in NAMES:
        assert torch.equal(got[name], clean[name]), name
    # a bad row of dO in head 1 of the first document: the second one and head 0 stay as they were
    do[40, 1, 7] = what
    got = _grads(h3, do, q, k, v, ranges)
    for name in NAMES:
        assert torch.equal(got[name][150:], clean[name][150:]) and torch.equal(got[name][:, 0], clean[name][:, 0])
    assert not bool(torch.isfinite(got["dv"][:41, 1]).all(-1).any())          # keys that row 40 sees
    assert torch.equal(got["dv"][41:150, 1], clean["dv"][41:150, 1])
    assert not bool(torch.isfinite(got["dq"][40, 1]).any())
    assert torch.equal(got["dq"][:40, 1], clean["dq"][:40, 1])
    # a bad key of head 0, seen by rows 60 and up of the first document
    do[40, 1, 7] = 1.0
    k[60, 0, 3] = what
    got = _grads(h3, do, q, k, v, ranges)
    assert not bool(torch.isfinite(got["dq"][60:150, 0]).all(-1).any())
    for lo, hi in ((0, 60), (150, 360)):
        assert torch.equal(got["dq"][lo:hi, 0], clean["dq"][lo:hi, 0])


def test_repeats_bit_for_bit_with_a_dirty_workspace(h3):
    n, h, kv = 900, 4, 2
    q, k, v, do = randn(1, n, h, 128), randn(2, n, kv, 128), randn(3, n, kv, 128), randn(4, n, h, 128)
    ranges = python_ranges([500, 380], [20, 0], n, "prefix_block")
    lse = torch.empty(h, n, device="cuda")
    o = h3.masked_attention(q, k, v, ranges, lse=lse)
    shape = h3.h3_attn_shape(n, n, 1, h, kv, 128, 0.0)
    work = torch.full((h3.h3_masked_attention_backward_workspace_bytes(shape),), 255, dtype=torch.uint8, device="cuda")
    first = h3.masked_attention_backward(do, q, k, v, o, lse, ranges)
    for _ in range(3):
        again = h3.masked_attention_backward(do, q, k, v, o, lse, ranges, workspace=work)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_on_a_side_stream_and_captured(h3):
    n = 500
    q, k, v, do = randn(1, n, 4, 128), randn(2, n, 2, 128), randn(3, n, 2, 128), randn(4, n, 4, 128)
    ranges = python_ranges([200, 290], [10, 20], n, "prefix_causal")
    lse = torch.empty(4, n, device="cuda")
    o = h3.masked_attention(q, k, v, ranges, lse=lse)
    want = h3.masked_attention_backward(do, q, k, v, o, lse, ranges)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = h3.masked_attention_backward(do, q, k, v, o, lse, ranges, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = h3.masked_attention_backward(do, q, k, v, o, lse, ranges)
    do.copy_(randn(9, n, 4, 128))
    graph.replay()
    want = h3.masked_attention_backward(do, q, k, v, o, lse, ranges)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refuses(h3):
    q, k = randn(1, 8, 4, 128), randn(2, 9, 2, 128)
    r = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    lse = torch.zeros(4, 8, device="cuda")
    B = h3.masked_attention_backward
    for f in (lambda: B(q[:7], q, k, k, q, lse, r), lambda: B(q, q, k, k, q[:7], lse, r),
              lambda: B(q, q, k, k, q, lse[:, :7], r), lambda: B(q, q, k, k, q, lse.double(), r),
              lambda: B(q, q, k, k, q, lse, r[:7]), lambda: B(q, q, k, k, q, lse, r, dq=k),
              lambda: B(q, q, k, k, q, lse, r, dk=q), lambda: B(q, q, k, k, q, lse, r, dv=k[:8]),
              lambda: B(q[:, :1].expand(8, 4, 128), q, k, k, q, lse, r),
              lambda: B(q, q, k, k, q, lse, r, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f()
