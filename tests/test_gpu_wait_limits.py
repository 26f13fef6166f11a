"""Waits that run out inside the masked attention, its gradients and the ring kernels of the norms.

With a limit of 1 ns a wait gives up unless what it waits for is there already.  Each kernel then stops what it
started (copies, products, tensor memory, the cluster's barriers) and returns; the host reads H3_ERR_TIMEOUT, and the
next call gives the same bits as before.  The last product of a walk over keys and the rows of a norm are never
there at first sight.
"""
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


def _expires_and_recovers(h3, call):
    want = [t.clone() for t in call()]
    assert h3.h3_check_device_error() == h3.H3_OK
    for _ in range(3):
        try:
            h3.h3_set_wait_limit_ns(1)
            call()
            assert h3.h3_check_device_error() == h3.H3_ERR_TIMEOUT
        finally:
            h3.h3_set_wait_limit_ns(0)
        assert h3.h3_check_device_error() == h3.H3_OK          # reported once
        assert all(torch.equal(a, b) for a, b in zip(want, call()))
        assert h3.h3_check_device_error() == h3.H3_OK


# (rows, heads, K/V heads, documents, mode): one CTA per block of rows, and clusters of two to eight that share its
# keys; a causal mask, short documents beside long ones, rows in no document, an uneven last tile
ATTENTION = [(1500, 40, 8, [0, 700, 1500], "prefix_causal"), (9472, 4, 4, [0, 9472], "document"),
             (2304, 8, 8, [0, 1000, 2304], "document"), (2304, 1, 1, [0, 2304], "document"),
             (4099, 2, 1, [0, 30, 4000], "prefix_causal"), (4096, 1, 1, [0, 4096], "document"),
             (82, 1, 1, [0, 30, 31, 82], "document")]


@pytest.mark.parametrize("nonfinite", [False, True])
@pytest.mark.parametrize("n,heads,kv,docs,mode", ATTENTION)
def test_masked_attention_and_gradients(h3, n, heads, kv, docs, mode, nonfinite):
    q, k, v, do = (randn(i, n, h, 128) for i, h in enumerate((heads, kv, kv, heads)))
    ranges = h3.build_key_ranges(torch.tensor(docs, dtype=torch.int32, device="cuda"), n, mode)
    if nonfinite:                       # in places that no row of the first half sees: second runs
        ranges[: n // 2] = torch.minimum(ranges[: n // 2], torch.tensor(n // 2 - 5, device="cuda", dtype=torch.int32))
        ranges[n // 2:, 0].clamp_(min=n // 2)
        ranges[n // 2:, 1].clamp_(min=n // 2)
        v[n // 2 - 3], k[n // 2 - 2] = float("inf"), float("nan")
        ranges[n - 1] = 0
        q[n - 1], do[n - 1] = float("nan"), float("inf")
    lse = torch.empty(1, heads, n, device="cuda")

    def forward():
        o = h3.masked_attention(q, k, v, ranges, lse=lse)
        return o, lse

    o = h3.masked_attention(q, k, v, ranges, lse=lse).clone()
    kept = lse.clone()
    if nonfinite:
        assert bool(torch.isfinite(o).all())
    _expires_and_recovers(h3, forward)
    _expires_and_recovers(h3, lambda: h3.masked_attention_backward(do, q, k, v, o, kept, ranges))


# (rows, elements): every ring shape, one, two and four rows a step
NORM = [(4000, 1032), (700, 2056), (4000, 5376), (2403, 6152), (2500, 8192), (1300, 11520)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,c", NORM)
def test_layer_norm_and_gradients(h3, n, c, dtype):
    x, dy, w = randn(1, n, c, dtype=dtype), randn(2, n, c, dtype=dtype), randn(3, c, dtype=torch.float32)
    _, mean, rstd = h3.layer_norm(x, w)
    _expires_and_recovers(h3, lambda: h3.layer_norm(x, w))
    _expires_and_recovers(h3, lambda: h3.layer_norm_backward(dy, x, mean, rstd, w))


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("n,c", [(4000, 1032), (3000, 2056), (4584, 5376), (2500, 8192)])
def test_adaln_gradients(h3, n, c, shuffled):
    x, dy = randn(1, n, c), randn(2, n, c)
    rows = torch.arange(n, device="cuda")
    level = (rows % 5 if shuffled else rows * 5 // n).int()
    tag = (rows // 7 % 3 if shuffled else rows * 3 // n).int()
    table = randn(4, 15, 2, c, dtype=torch.float32)
    _expires_and_recovers(h3, lambda: h3.adaln_modulate_backward(dy, x, level, tag, table))
