"""The row statistics of the AdaLN gradients where the order of the additions shows."""
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import norm_backward, norm_terms, randn, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [2048, 5376, 8192])
def test_small_elements_behind_large_ones(c):
    """Rows whose first 32 chunks of 8 begin with two elements of +-4,128, the others just below half an ulp of that.

    A chain of additions that begins with a large element loses every small one after it, so the row's mean is off
    by as many of them as the chain is long: the bound of ``norm_terms`` allows a chain of 32.  Each row has a table
    entry of its own, so the scale's gradient is dy * xhat without any further sum, in fp32.
    """
    import packed_mm_rope_b200 as h3
    n, big, small = 40, 4128.0, 2.0 ** -12 * (1 - 2.0 ** -8)
    chunk = torch.arange(c // 8)
    x = torch.full((n, c // 8, 8), small, dtype=torch.float64)
    first = chunk < 32
    sign = torch.where(chunk % 32 < 16, 1.0, -1.0).double()
    x[:, first, 0] = x[:, first, 1] = big * sign[first]
    x = x.reshape(n, c)
    assert torch.equal(x.bfloat16().double(), x)
    x = x.bfloat16().cuda()
    dy, eps = randn(1, n, c), 1e-6
    level = torch.arange(n, dtype=torch.int32, device="cuda")
    tag = torch.zeros_like(level)
    table = randn(2, 3 * n, 2, c, dtype=torch.float32, scale=0.3)
    dx, dtable = h3.adaln_modulate_backward(dy, x, level, tag, table, eps=eps)
    w = 1.0 + table[::3, 1].double()
    rdx, bdx, rdw, bdw, rdb, _ = norm_backward(dy, x, w, eps, torch.bfloat16, 0)
    within(dx, rdx, bdx + 2.0 ** -23 * norm_terms(x, eps)[2] * ((dy.double() * w).abs() + 1), "dx")
    within(dtable[::3, 1], rdw, bdw, "scale")
    assert torch.equal(dtable[::3, 0].double(), rdb)
    assert not dtable[1::3].any() and not dtable[2::3].any()
