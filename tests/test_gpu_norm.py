"""Layer norm, its gradients and the AdaLN gradients on the GPU against 64-bit references."""
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import half, norm_backward, norm_terms, norm_y_bound, randn, within

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


SIZES = [(1, 1), (3, 2), (5, 7), (82, 129), (33, 256), (7, 257), (9, 1024), (5, 1032), (4, 4096), (6, 4104),
         (3, 5376), (2, 8192), (2, 8200), (3, 11520), (2, 11528), (3, 16384), (3, 16377), (2500, 64), (700, 5376),
         (1301, 1800), (2403, 2056), (1, 6152), (601, 7680)]
TYPES = [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
         (torch.float16, torch.float16), (torch.float32, torch.float32)]


def _chain(n, c):
    """Additions in a row of one column sum: a group's rows, then the partial rows."""
    return n // 296 + 1 + 2368 // 8


@pytest.mark.parametrize("types", TYPES, ids=lambda t: f"{t[0]}-{t[1]}".replace("torch.", ""))
@pytest.mark.parametrize("n,c", SIZES)
def test_layer_norm_and_gradients(h3, n, c, types):
    dt, pt = types
    x = randn(1, n, c, dtype=dt, scale=1.5, shift=0.75)
    w, b = randn(2, c, dtype=pt, scale=0.3, shift=1.0), randn(3, c, dtype=pt)
    dy = randn(4, n, c, dtype=dt)
    y, mean, rstd = h3.layer_norm(x, w, b, eps=EPS)
    xhat, m64, r64, ex = norm_terms(x, EPS)
    want, bound = norm_y_bound(xhat, ex, w.double(), b.double(), dt)
    within(y, want, bound, "y")
    within(mean, m64[:, 0], 50 * 2.0 ** -24 * x.double().abs().mean(1) + 1e-300, "mean")
    within(rstd, r64[:, 0], 64 * 2.0 ** -24 * r64[:, 0], "rstd")
    dx, dw, db = h3.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.dtype == dt and dw.dtype == pt and db.dtype == pt
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, w.double(), EPS, dt, _chain(n, c))
    within(dx, rdx, bdx + 1e-300, "dx")
    within(dw, rdw.sum(0), bdw.sum(0) + half(pt) * rdw.sum(0).abs() + 1e-300, "dweight")
    within(db, rdb.sum(0), bdb.sum(0) + half(pt) * rdb.sum(0).abs() + 1e-300, "dbias")


def test_layer_norm_without_parameters_and_without_their_gradients(h3):
    x, dy = randn(1, 37, 520), randn(2, 37, 520)
    y, mean, rstd = h3.layer_norm(x, eps=EPS)
    xhat, _, _, ex = norm_terms(x, EPS)
    one, zero = torch.ones((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64, device="cuda")
    want, bound = norm_y_bound(xhat, ex, one, zero, x.dtype)
    within(y, want, bound, "y")
    dx, dw, db = h3.layer_norm_backward(dy, x, mean, rstd)
    dx2, none_w, none_b = h3.layer_norm_backward(dy, x, mean, rstd, param_grads=False)
    assert none_w is None and none_b is None and torch.equal(dx, dx2) and dw.dtype == torch.float32
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, one, EPS, x.dtype, _chain(37, 520))
    within(dx, rdx, bdx, "dx")
    within(dw, rdw.sum(0), bdw.sum(0), "dweight")
    within(db, rdb.sum(0), bdb.sum(0), "dbias")


def test_layer_norm_no_rows(h3):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = h3.layer_norm(x, w, w)
    assert y.shape == (0, 64)
    dx, dw, db = h3.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("c", [129, 512, 5376])
def test_layer_norm_strides_offsets_and_in_place(h3, c):
    """Rows inside a wider buffer, at an odd offset too: in bounds, the rest untouched, in place alike.

    Rows that are not 16-byte aligned may be summed in another order than aligned ones, so results are held to
    the bounds of the formula, not to another call's bits.
    """
    n = 21
    for off in (0, 1, 8):
        for dt in (torch.bfloat16, torch.float32):
            wide = randn(5, n, c + 24, dtype=dt)
            keep = wide.clone()
            x = wide[:, off:off + c]
            w = randn(6, c, dtype=torch.float32)
            dy = randn(7, n, c, dtype=dt)
            out = torch.full_like(wide, 7.0)
            y, mean, rstd = h3.layer_norm(x, w, eps=EPS, out=out[:, off:off + c])
            xhat, _, _, ex = norm_terms(x, EPS)
            want, bound = norm_y_bound(xhat, ex, w.double(), torch.zeros_like(w).double(), dt)
            within(y, want, bound, "y")
            y = y.clone()
            assert torch.equal(wide, keep)
            assert bool((out[:, :off] == 7).all()) and bool((out[:, off + c:] == 7).all())
            g = h3.layer_norm_backward(dy, x, mean, rstd, w, dx=out[:, off:off + c])
            rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, w.double(), EPS, dt, _chain(n, c))
            within(g[0], rdx, bdx, "dx")
            within(g[1], rdw.sum(0), bdw.sum(0) + half(torch.float32) * rdw.sum(0).abs(), "dweight")
            within(g[2], rdb.sum(0), bdb.sum(0) + half(torch.float32) * rdb.sum(0).abs(), "dbias")
            dx = g[0].clone()
            assert bool((out[:, :off] == 7).all()) and bool((out[:, off + c:] == 7).all())
            # in place: the same bits
            h3.layer_norm(x, w, eps=EPS, out=x)
            assert torch.equal(x, y) and torch.equal(wide[:, :off], keep[:, :off])
            wide_dy = keep.clone()
            wide_dy[:, off:off + c] = dy
            view = wide_dy[:, off:off + c]
            first = h3.layer_norm_backward(view, keep[:, off:off + c], mean, rstd, w)[0]
            assert torch.equal(h3.layer_norm_backward(view, keep[:, off:off + c], mean, rstd, w, dx=view)[0], first)
            within(view, dx.double(), 2 * bdx, "dx in place")


def test_layer_norm_large_mean_and_infinite_rows(h3):
    """A mean a thousand deviations away costs no digits beyond the bound; a row with inf or NaN spoils itself only."""
    x = randn(1, 40, 1000, dtype=torch.float32, scale=1.0, shift=1000.0)
    y, mean, rstd = h3.layer_norm(x, eps=EPS)
    xhat, _, _, ex = norm_terms(x, EPS)
    within(y, xhat, half(torch.float32) * xhat.abs() + ex, "y")
    x = randn(1, 9, 520)
    clean = h3.layer_norm(x)[0]
    x[4, 3] = float("inf")
    x[6, 519] = float("nan")
    y = h3.layer_norm(x)[0]
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[6]).all()) and bool(torch.isnan(y[4, 3]))


def test_layer_norm_repeats_bit_for_bit(h3):
    x, dy = randn(1, 3000, 1288), randn(2, 3000, 1288)
    w = randn(3, 1288, dtype=torch.float32)
    _, mean, rstd = h3.layer_norm(x, w)
    first = h3.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(3):
        for a, b in zip(first, h3.layer_norm_backward(dy, x, mean, rstd, w)):
            assert torch.equal(a, b)


def test_layer_norm_gradients_match_differences(h3):
    """sum(dy * y) changes along a direction as the gradients say (64-bit forward form, fp32 gradients)."""
    n, c = 6, 37
    x, dy = randn(1, n, c, dtype=torch.float32), randn(2, n, c, dtype=torch.float32)
    w, b = randn(3, c, dtype=torch.float32), randn(4, c, dtype=torch.float32)
    _, mean, rstd = h3.layer_norm(x, w, b, eps=EPS)
    dx, dw, db = h3.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x_, w_, b_):
        xhat, _, _, _ = norm_terms(x_, EPS)
        return (dy.double() * (xhat * w_ + b_)).sum()

    step = 1e-5
    for i, (g, t) in enumerate(((dx, x), (dw, w), (db, b))):
        d = randn(9 + i, *t.shape, dtype=torch.float64)
        args = [x.double(), w.double(), b.double()]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        diff = (loss(*up) - loss(*down)) / (2 * step)
        # central differences are off by step^2 (third derivatives of order 1, n c terms), the gradient by fp32 sums
        assert abs(diff - (g.double() * d).sum()) <= 1e-4 * (g.double() * d).abs().sum()


# ------------------------------------------------------------------ AdaLN --

def _rows(n, levels, shuffled, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = torch.arange(n)
    ts, tags = (r * levels // max(1, n)).int(), (r * 5 // max(1, n) % 3).int()
    if shuffled:
        perm = torch.randperm(n, generator=g)
        ts, tags = ts[perm], tags[perm]
    return ts.cuda().contiguous(), tags.cuda().contiguous()


@pytest.mark.parametrize("n,c,levels,shuffled", [(1, 64, 1, False), (82, 128, 2, True), (33, 8, 3, False),
                                                 (2049, 256, 40, True), (700, 1032, 7, True), (4584, 5376, 2, True),
                                                 (1500, 5376, 31, False), (300, 8192, 100, True), (5000, 64, 2730, True),
                                                 (2000, 8192, 5, True), (9000, 1288, 3, True), (3000, 4096, 900, True)])
def test_adaln_backward(h3, n, c, levels, shuffled):
    x, dy = randn(1, n, c, scale=1.5, shift=0.5), randn(2, n, c)
    ts, tags = _rows(n, levels, shuffled)
    e = 3 * levels
    table = randn(3, e, 2, c, dtype=torch.float32, scale=0.3)
    dx, dt = h3.adaln_modulate_backward(dy, x, ts, tags, table, eps=1e-6)
    assert h3.h3_check_device_error() == h3.H3_OK
    idx = ts.long() * 3 + tags.long()
    w = 1.0 + table[:, 1].double()[idx]
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, w, 1e-6, torch.bfloat16, n // 296 + 400)
    # the weight 1 + scale is rounded once more
    within(dx, rdx, bdx + 2.0 ** -23 * norm_terms(x, 1e-6)[2] * ((dy.double() * w).abs() + 1), "dx")
    for half_, v, bound in ((1, rdw, bdw), (0, rdb, bdb)):
        want = torch.zeros(e, c, dtype=torch.float64, device="cuda").index_add_(0, idx, v)
        tol = torch.zeros(e, c, dtype=torch.float64, device="cuda").index_add_(0, idx, bound)
        within(dt[:, half_], want, tol, "table")


def test_adaln_backward_is_the_gradient_of_the_forward_call(h3):
    """With scale 0 it is layer norm's, and the rows of one entry add up to layer norm's parameter gradients."""
    n, c = 500, 520
    x, dy = randn(1, n, c), randn(2, n, c)
    ts, tags = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 2, c, device="cuda")
    dx, dt = h3.adaln_modulate_backward(dy, x, ts, tags, table, eps=EPS)
    _, mean, rstd = h3.layer_norm(x, eps=EPS)
    gx, gw, gb = h3.layer_norm_backward(dy, x, mean, rstd)
    assert not dt[0].any() and not dt[2].any()
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, torch.ones((), dtype=torch.float64, device="cuda"), EPS,
                                               x.dtype, 400)
    within(dx, gx.double(), 2 * bdx, "dx")
    within(dt[1, 1], gw.double(), 2 * bdw.sum(0), "scale")
    within(dt[1, 0], gb.double(), 2 * bdb.sum(0), "shift")


def test_adaln_backward_bad_index_in_place_and_strides(h3):
    n, c = 300, 256
    wide = randn(1, n, c + 64)
    x, dy = wide[:, :c], randn(2, n, c)
    ts, tags = _rows(n, 4, True)
    table = randn(3, 12, 2, c, dtype=torch.float32)
    dx0, dt0 = h3.adaln_modulate_backward(dy, x.contiguous(), ts, tags, table)
    dy2 = dy.clone()
    dx1, dt1 = h3.adaln_modulate_backward(dy2, x, ts, tags, table, dx=dy2)
    assert dx1 is dy2 and torch.equal(dx0, dx1) and torch.equal(dt0, dt1)
    ts2 = ts.clone()
    ts2[17], ts2[200] = 9, -1                    # no such entries
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[17] = good[200] = False
    dx2, dt2 = h3.adaln_modulate_backward(dy, x, ts2, tags, table)
    assert h3.h3_check_device_error() == h3.H3_ERR_DEVICE_INPUT
    assert torch.equal(dx2[good], dx0[good]) and bool(torch.isnan(dx2[~good]).all())
    dx3, dt3 = h3.adaln_modulate_backward(dy[good], x[good], ts[good].contiguous(), tags[good].contiguous(), table)
    within(dt2, dt3.double(), 1e-4 + 1e-4 * dt3.double().abs(), "table without the bad rows")
    zero = h3.adaln_modulate_backward(dy[:0], x[:0], ts[:0], tags[:0], table)[1]
    assert not zero.any()


def test_norm_calls_on_a_side_stream_and_captured(h3):
    x, dy = randn(1, 600, 1032), randn(2, 600, 1032)
    w = randn(3, 1032, dtype=torch.float32)
    ts, tags = _rows(600, 4, True)
    table = randn(4, 12, 2, 1032, dtype=torch.float32)

    def all_of(stream=None):
        y, mean, rstd = h3.layer_norm(x, w, stream=stream)
        return (y, *h3.layer_norm_backward(dy, x, mean, rstd, w, stream=stream),
                *h3.adaln_modulate_backward(dy, x, ts, tags, table, stream=stream))

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    x2 = randn(11, 600, 1032)
    x.copy_(x2)
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(all_of(), got))


def test_norm_binding_refuses(h3):
    x = randn(1, 8, 64)
    w = torch.ones(64, device="cuda")
    y, mean, rstd = h3.layer_norm(x, w)
    bad = [lambda: h3.layer_norm(x.double()), lambda: h3.layer_norm(x[0]), lambda: h3.layer_norm(x.t()),
           lambda: h3.layer_norm(x, w[:32]), lambda: h3.layer_norm(x, w.cpu()),
           lambda: h3.layer_norm(x, w, w.bfloat16()), lambda: h3.layer_norm(x, out=x.float()),
           lambda: h3.layer_norm(x, mean=mean[:4]), lambda: h3.layer_norm_backward(x[:4], x, mean, rstd, w),
           lambda: h3.layer_norm_backward(x, x, mean[:4], rstd, w),
           lambda: h3.layer_norm_backward(x, x, mean, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    ts = torch.zeros(8, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 2, 64, device="cuda")
    A = h3.adaln_modulate_backward
    bad += [lambda: A(x, x, ts[:4], ts, table), lambda: A(x, x, ts, ts.long(), table), lambda: A(x, x, ts, ts, table[:, :1]),
            lambda: A(x, x, ts, ts, table.double()), lambda: A(x.float(), x, ts, ts, table),
            lambda: A(x[:, :60], x[:, :60], ts, ts, torch.zeros(3, 2, 60, device="cuda")),
            lambda: A(x, x, ts, ts, table, dtable=torch.zeros(2, 2, 64, device="cuda"))]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(h3.H3Error):
        h3.layer_norm(x.float(), w.bfloat16())          # parameters neither of x's type nor fp32
    with pytest.raises(h3.H3Error):
        h3.layer_norm(torch.zeros(2, 16385, device="cuda"))


def test_norm_waits_are_bounded(h3):
    """With a wait limit of 1 ns a call either ends with its results or reports the expiry; the next ones are right.

    (A wait looks several times before it looks at the clock, so rows that come quickly are not missed.)
    """
    x, dy = randn(1, 400, 2056), randn(2, 400, 2056)
    w = randn(3, 2056, dtype=torch.float32)
    ts, tags = _rows(400, 4, True)
    table = randn(4, 12, 2, 2056, dtype=torch.float32)
    _, mean, rstd = h3.layer_norm(x, w)
    calls = (lambda: h3.layer_norm(x, w), lambda: h3.layer_norm_backward(dy, x, mean, rstd, w),
             lambda: h3.adaln_modulate_backward(dy, x, ts, tags, table))
    for call in calls:
        want = call()
        assert h3.h3_check_device_error() == h3.H3_OK
        h3.h3_set_wait_limit_ns(1)
        try:
            got = call()
            status = h3.h3_check_device_error()
        finally:
            h3.h3_set_wait_limit_ns(0)
        assert status in (h3.H3_OK, h3.H3_ERR_TIMEOUT)
        if status == h3.H3_OK:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert h3.h3_check_device_error() == h3.H3_OK
        assert all(torch.equal(a, b) for a, b in zip(want, call()))
