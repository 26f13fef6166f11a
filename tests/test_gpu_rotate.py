"""h3_mmrope_rotate (grouped heads, both directions) against the fp64 oracle and the equal-heads call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import workload as W
from oracle import rope as orope
from tests.gpu_util import bf16_bits_to_f64, check_rope, from_dev_bf16
from tests.train_util import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


def _coords(n, seed=0):
    rng = np.random.default_rng(seed)
    c = np.stack([rng.uniform(-6000, 6000, n), rng.integers(0, 44, n), rng.integers(0, 80, n)], 1)
    return c.astype(np.float32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout,rule", [(0, 0), (1, 1)])
@pytest.mark.parametrize("n,h,kv", [(1, 1, 1), (5, 3, 1), (82, 8, 2), (301, 42, 14), (1200, 40, 5), (7, 64, 64)])
def test_rotate_matches_oracle(h3, n, h, kv, layout, rule, inverse):
    c = _coords(n, n)
    q, k = randn(1, n, h, 128), randn(2, n, kv, 128)
    qo, ko = h3.mmrope_rotate(q, k, torch.from_numpy(c).cuda(), inverse=inverse, pair_layout=layout, freq_rule=rule)
    ang = orope.angles(c, 10000.0, freq_rule=rule) * (-1.0 if inverse else 1.0)
    for x, y in ((q, qo), (k, ko)):
        x64 = bf16_bits_to_f64(from_dev_bf16(x))
        frac, _ = check_rope(from_dev_bf16(y), orope.rotate(x64, ang, layout), x64, layout)
        assert frac > 0.99


def test_rotate_equals_the_equal_heads_call(h3):
    wl = W.workload(0)
    coords = h3.build_coords(wl.segments, wl.n_rows)
    q, k = randn(1, wl.n_rows, 8, 128), randn(2, wl.n_rows, 8, 128)
    for layout in (0, 1):
        a = h3.mmrope_qk(q, k, coords, pair_layout=layout)
        b = h3.mmrope_rotate(q, k, coords, pair_layout=layout)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # without either tensor, and k alone with fewer heads
        assert torch.equal(h3.mmrope_rotate(q, None, coords, pair_layout=layout)[0], a[0])
        assert torch.equal(h3.mmrope_rotate(None, k[:, :3], coords, pair_layout=layout)[1], a[1][:, :3])


def test_rotate_is_orthogonal(h3):
    """<g, R x> = <R^T g, x> up to the two bf16 roundings: the rotation back is the gradient."""
    n = 200
    c = torch.from_numpy(_coords(n)).cuda()
    x, g = randn(1, n, 5, 128), randn(2, n, 5, 128)
    y = h3.mmrope_rotate(x, None, c)[0]
    gx = h3.mmrope_rotate(g, None, c, inverse=True)[0]
    a, b = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
    slack = 2.0 ** -8 * ((g.double() * y.double()).abs().sum() + (gx.double() * x.double()).abs().sum())
    assert abs(a - b) <= slack


def test_rotate_strides_in_place_batches_and_untouched_rows(h3):
    n, h, kv = 33, 6, 2
    c = torch.from_numpy(_coords(2 * n)).cuda()
    fused = randn(3, 2, n, h + 2 * kv, 128)
    keep = fused.clone()
    q, k = fused[:, :, :h], fused[:, :, h:h + kv]
    want = h3.mmrope_rotate(q.contiguous(), k.contiguous(), c)
    got = h3.mmrope_rotate(q, k, c)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(fused, keep)
    h3.mmrope_rotate(q, k, c, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(fused[:, :, h + kv:], keep[:, :, h + kv:])
    out = torch.full((2, n, h + 3, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    h3.mmrope_rotate(keep[:, :, :h], None, c, q_out=out[:, :, :h])
    assert torch.equal(out[:, :, :h], want[0]) and bool((out[:, :, h:] == 5).all())


def test_rotate_refuses(h3):
    q, k = randn(1, 4, 2, 128), randn(2, 4, 1, 128)
    c = torch.zeros(4, 3, device="cuda")
    R = h3.mmrope_rotate
    for f in (lambda: R(None, None, c), lambda: R(q, k[:3], c), lambda: R(q, k, c[:3]), lambda: R(q, k, c.double()),
              lambda: R(q, k, c, q_out=k), lambda: R(None, k, c, q_out=q), lambda: R(q.float(), k, c),
              lambda: R(q, k, c.cpu())):
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(h3.H3Error):
        R(q, k, c, sections=(32, 48, 46))
    empty = R(q[:0], k[:0], c[:0])
    assert empty[0].shape == (0, 2, 128) and empty[1].shape == (0, 1, 128)
