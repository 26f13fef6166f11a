"""Layer norm, its gradients and AdaLN's on rows whose mean is many deviations away from zero.

The mean is rounded to fp32, so xhat is off by some 2^-24 |mean| / deviation, whatever form the kernels give it; the
sums add the roundings of their chains.  The bounds are those of the other tests (``norm_terms``): 48 U mean|x| for
the mean, the variance from squared deviations.
"""
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


# short and long rows, in 16-byte pieces (rings of rows from 1,025 to 11,520 elements) and not
@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1000.0), (torch.float32, -30000.0), (torch.float16, 300.0),
                                         (torch.bfloat16, -64.0)])
@pytest.mark.parametrize("n,c", [(40, 1000), (700, 1032), (41, 2057), (1300, 5376), (37, 5377), (50, 8192), (9, 16384)])
def test_layer_norm_and_gradients(h3, n, c, dtype, shift):
    x = randn(1, n, c, dtype=dtype, shift=shift)
    w, b = randn(2, c, dtype=torch.float32, scale=0.3, shift=1.0), randn(3, c, dtype=torch.float32)
    if dtype == torch.float32:
        dy = randn(4, n, c, dtype=dtype)
    else:
        dy = randn(4, n, c, dtype=dtype, shift=3.0)
    y, mean, rstd = h3.layer_norm(x, w, b, eps=EPS)
    xhat, m64, r64, ex = norm_terms(x, EPS)
    want, bound = norm_y_bound(xhat, ex, w.double(), b.double(), dtype)
    within(y, want, bound, "y")
    within(mean, m64[:, 0], 50 * 2.0 ** -24 * x.double().abs().mean(1), "mean")
    # the mean's error enters the variance squared
    emean = 48 * 2.0 ** -24 * x.double().abs().mean(1)
    within(rstd, r64[:, 0], (64 * 2.0 ** -24 + (emean * r64[:, 0]) ** 2) * r64[:, 0], "rstd")
    dx, dw, db = h3.layer_norm_backward(dy, x, mean, rstd, w)
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, w.double(), EPS, dtype, n // 296 + 1 + 2368 // 8)
    within(dx, rdx, bdx, "dx")
    within(dw, rdw.sum(0), bdw.sum(0) + half(torch.float32) * rdw.sum(0).abs(), "dweight")
    within(db, rdb.sum(0), bdb.sum(0) + half(torch.float32) * rdb.sum(0).abs(), "dbias")


@pytest.mark.parametrize("n,c", [(300, 520), (500, 1032), (1300, 5376), (400, 8192)])
def test_adaln_gradients(h3, n, c):
    x, dy = randn(1, n, c, shift=64.0), randn(2, n, c, shift=1.0)
    rows = torch.arange(n, device="cuda")
    level, tag = (rows % 4).int(), (rows // 5 % 3).int()
    table = randn(3, 12, 2, c, dtype=torch.float32, scale=0.3)
    dx, dt = h3.adaln_modulate_backward(dy, x, level, tag, table, eps=1e-6)
    e = (level * 3 + tag).long()
    w = 1.0 + table[:, 1].double()[e]
    rdx, bdx, rdw, bdw, rdb, bdb = norm_backward(dy, x, w, 1e-6, torch.bfloat16, n // 148 + 400)
    within(dx, rdx, bdx + 2.0 ** -23 * norm_terms(x, 1e-6)[2] * ((dy.double() * w).abs() + 1), "dx")
    for half_, v, bound in ((1, rdw, bdw), (0, rdb, bdb)):
        want = torch.zeros(12, c, dtype=torch.float64, device="cuda").index_add_(0, e, v)
        tol = torch.zeros(12, c, dtype=torch.float64, device="cuda").index_add_(0, e, bound)
        within(dt[:, half_], want, tol, "table")
