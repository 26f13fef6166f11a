"""Host-side refusals of the masked-attention and training-direction calls: nothing is launched, no GPU needed."""
import ctypes

import pytest

import packed_mm_rope_b200 as h3
from packed_mm_rope_b200 import _lib

P = 0x10000
INV, UNS = h3.H3_ERR_INVALID_ARG, h3.H3_ERR_UNSUPPORTED


def _err(fn, *a, **kw):
    with pytest.raises(h3.H3Error) as e:
        fn(*a, **kw)
    return e.value.status


def test_attn_shape_layout():
    assert ctypes.sizeof(h3.h3_attn_shape) == 40


def test_rotate():
    R, cfg = h3.h3_mmrope_rotate, h3.rope_cfg()
    ok = (P, P, P, P, P, 4, 2, 1, 256, 128, 256, 128, cfg)
    R(0, 0, 0, 0, 0, 0, 2, 1, 256, 128, 256, 128, cfg)                     # no rows: no-op

    def but(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return a

    for a in (but(_5=-1), but(_6=-1), but(_6=0, _7=0), but(_0=0), but(_2=0), but(_1=0), but(_3=0), but(_4=0),
              but(_8=248), but(_9=120), but(_10=248), but(_11=0), but(_12=h3.rope_cfg(theta=1.0))):
        assert _err(R, *a) == INV
    assert _err(R, *ok, 2) == INV
    for a in (but(_0=P + 8), but(_3=P + 2), but(_8=260), but(_11=132),
              but(_12=h3.rope_cfg(head_dim=256, sections=(64, 96, 96)))):
        assert _err(R, *a) == UNS


def test_key_ranges():
    B = h3.h3_build_key_ranges
    assert _err(B, P, 0, -1, 4, 0, P) == INV
    assert _err(B, P, 0, 1, -1, 0, P) == INV
    assert _err(B, P, 0, 1, 1 << 31, 0, P) == INV
    assert _err(B, P, 0, 1, 4, 3, P) == INV
    assert _err(B, 0, 0, 1, 4, 0, P) == INV
    assert _err(B, P, 0, 1, 4, 0, 0) == INV
    assert _err(B, P, 0, 1, 4, 0, P + 4) == UNS


def _shape(**kw):
    d = dict(n_q=4, n_k=4, batch=1, n_heads=4, n_kv_heads=2, head_dim=128, softmax_scale=0.0)
    d.update(kw)
    return h3.h3_attn_shape(**d)


def test_masked_attention():
    A = h3.h3_masked_attention
    strides = (512, 256, 256, 512)
    A(0, 0, 0, 0, 0, 0, _shape(n_q=0), *strides)                            # no rows: no-op
    for kw in (dict(batch=0), dict(batch=65536), dict(n_heads=0), dict(n_kv_heads=0), dict(n_heads=5), dict(n_q=-1),
               dict(n_k=-1), dict(n_q=1 << 31), dict(n_k=1 << 31), dict(softmax_scale=float("inf"))):
        assert _err(A, P, P, P, P, 0, P, _shape(**kw), *strides) == INV, kw
    assert _err(A, P, P, P, P, 0, P, _shape(head_dim=64), *strides) == UNS
    for i in range(4):
        s = list(strides)
        s[i] -= 8
        assert _err(A, P, P, P, P, 0, P, _shape(), *s) == INV
        s[i] += 12
        assert _err(A, P, P, P, P, 0, P, _shape(), *s) == UNS
        ptrs = [P, P, P, P]
        ptrs[i] = 0
        assert _err(A, *ptrs, 0, P, _shape(), *strides) == INV
        ptrs[i] = P + 8
        assert _err(A, *ptrs, 0, P, _shape(), *strides) == UNS
    assert _err(A, P, P, P, P, 0, 0, _shape(), *strides) == INV
    assert _err(A, P, P, P, P, 0, P + 4, _shape(), *strides) == UNS


def test_layernorm():
    L, B, W = h3.h3_layernorm, h3.h3_layernorm_backward, h3.h3_layernorm_backward_workspace_bytes
    L(0, 0, 0, 0, 0, 0, 0, 64, 64, 64)                                       # no rows: no-op
    assert _err(L, P, P, 0, 0, 0, 0, -1, 64, 64, 64) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 0, 64, 64) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 63, 64) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 64, 63) == INV
    assert _err(L, P, 0, 0, 0, 0, 0, 4, 64, 64, 64) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 64, 64, 3) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 64, 64, 0, 2, -1.0) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 64, 64, 0, 2, float("nan")) == INV
    assert _err(L, P, P, 0, 0, 0, 0, 4, 64, 64, 64, 0, 1) == UNS            # fp16 parameters of bf16 rows
    assert _err(L, P, P, 0, 0, 0, 0, 4, 16385, 16385, 16385) == UNS
    assert W(-1, 64) == 0 and W(4, 0) == 0 and W(4, 16385) == 0
    assert W(0, 64) >= 256 and W(28196, 5376) >= 2 * 5376 * 4 and W(10 ** 9, 5376) == W(10 ** 6, 5376)
    ok = [P, P, P, P, 0, P, P, P, P, 4, 64, 64, 64, 64]
    for i in (0, 1, 2, 3, 5, 8):
        a = list(ok)
        a[i] = 0
        assert _err(B, *a) == INV
    assert _err(B, *(ok[:8] + [P + 128] + ok[9:])) == INV                    # workspace not 256-byte aligned
    for i in (11, 12, 13):
        a = list(ok)
        a[i] = 63
        assert _err(B, *a) == INV
    assert _err(B, *ok, 0, 1) == UNS


def test_adaln_backward():
    B, W = h3.h3_adaln_modulate_backward, h3.h3_adaln_backward_workspace_bytes
    assert W(4, 60, 3) == 0 and W(4, 8200, 3) == 0 and W(4, 64, 0) == 0 and W(4, 64, 8193) == 0 and W(-1, 64, 3) == 0
    assert W(1 << 31, 64, 3) == 0 and W(0, 64, 3) > 0
    ok = [P, P, P, P, P, P, P, P, 3, 4, 64, 64, 64, 64]
    for i in range(8):
        a = list(ok)
        a[i] = 0
        assert _err(B, *a) == INV
    for i, v, want in ((8, 0, INV), (8, 8193, UNS), (9, -1, INV), (9, 1 << 31, INV), (10, 60, UNS), (10, 4, INV),
                       (10, 8200, UNS), (11, 56, INV), (12, 56, INV), (13, 56, INV), (11, 68, UNS), (12, 68, UNS),
                       (13, 68, UNS), (0, P + 8, UNS), (1, P + 8, UNS), (4, P + 8, UNS), (5, P + 8, UNS),
                       (7, P + 128, INV)):
        a = list(ok)
        a[i] = v
        assert _err(B, *a) == want, (i, v)
    assert _err(B, *ok, -1.0) == INV


def test_masked_attention_backward():
    B, W = h3.h3_masked_attention_backward, h3.h3_masked_attention_backward_workspace_bytes
    names = ("q", "k", "v", "o", "dout", "dq", "dk", "dv")
    ok = dict(q=512, k=256, v=256, o=512, dout=512, dq=512, dk=256, dv=256)
    S = h3.h3_attn_strides
    ptrs = [P] * 11
    assert W(_shape(n_heads=5)) == 0 and W(_shape(head_dim=64)) == 0 and W(_shape(batch=0)) == 0
    assert W(_shape()) >= 128 * 4 * 8 + 128 * 8 + 16
    B(*([0] * 10), P, _shape(n_q=0, n_k=0), S(**ok))                          # nothing to do
    for i in range(11):
        p = list(ptrs)
        p[i] = 0
        assert _err(B, *p, _shape(), S(**ok)) == INV, i
    for i in (0, 1, 2, 3, 4, 7, 8, 9):
        p = list(ptrs)
        p[i] = P + 8
        assert _err(B, *p, _shape(), S(**ok)) == UNS, i
    p = list(ptrs)
    p[10] = P + 128
    assert _err(B, *p, _shape(), S(**ok)) == INV                              # workspace not 256-byte aligned
    p = list(ptrs)
    p[6] = P + 4
    assert _err(B, *p, _shape(), S(**ok)) == UNS
    for n in names:
        assert _err(B, *ptrs, _shape(), S(**{**ok, n: ok[n] - 8})) == INV, n
        assert _err(B, *ptrs, _shape(), S(**{**ok, n: ok[n] + 4})) == UNS, n
    for kw in (dict(batch=0), dict(n_heads=5), dict(n_q=1 << 31), dict(n_k=-1), dict(softmax_scale=float("nan"))):
        assert _err(B, *ptrs, _shape(**kw), S(**ok)) == INV, kw
    assert _err(B, *ptrs, _shape(head_dim=64), S(**ok)) == UNS


def _apart(n, step=1 << 20):
    """n distinct 256-byte aligned addresses, far from one another."""
    return [0x1000000 + i * step for i in range(n)]


def test_outputs_apart_from_inputs():
    """An output may not share memory with an input, except exactly in place where the call allows it."""
    # masked attention: out inside q, k or v
    q, k, v, o, r = _apart(5)
    strides = (512, 256, 256, 512)
    for bad in (q, k, v, q + 1024 * 3, k - 1024, v + 512 * 3):
        assert _err(h3.h3_masked_attention, q, k, v, bad, 0, r, _shape(), *strides) == INV, hex(bad)
    # an input's columns with another row stride
    assert _err(h3.h3_masked_attention, q, k, v, q + 1024, 0, r, _shape(), 1024, 256, 256, 512) == INV

    p = _apart(11)                                     # dout q k v o lse ranges dq dk dv work
    S = h3.h3_attn_strides(q=512, k=256, v=256, o=512, dout=512, dq=512, dk=256, dv=256)
    for i in (7, 8, 9):
        for j in (0, 1, 2, 3, 4, 7, 8, 9):
            if i == j:
                continue
            a = list(p)
            a[i] = a[j]
            assert _err(h3.h3_masked_attention_backward, *a, _shape(), S) == INV, (i, j)

    # rotation: across tensors, or shifted in its own
    q, k, qo, ko, c = _apart(5)
    tail = (c, 4, 2, 1, 256, 128, 256, 128, h3.rope_cfg())
    for a in ((q, k, k, ko), (q, k, qo, q), (q, k, qo, qo), (q, k, q + 512, ko), (q, k, qo, k - 256)):
        assert _err(h3.h3_mmrope_rotate, *a, *tail) == INV
    assert _err(h3.h3_mmrope_rotate, q, k, q, ko, c, 4, 2, 1, 256, 128, 512, 128, h3.rope_cfg()) == INV

    x, y, m, rs, w = _apart(5)
    assert _err(h3.h3_layernorm, x, x + 128, 0, 0, m, rs, 4, 64, 64, 64) == INV
    assert _err(h3.h3_layernorm, x, x, 0, 0, m, rs, 4, 64, 64, 128) == INV
    dy, dx = y, x + (1 << 24)
    for bad, sy, sx, sd in ((x + 128, 64, 64, 64), (dy - 128, 64, 64, 64), (x, 64, 64, 72), (dy, 72, 64, 64)):
        assert _err(h3.h3_layernorm_backward, dy, x, m, rs, 0, bad, 0, 0, 0, 4, 64, sy, sx, sd) == INV
    t, tag, tab, dtab = _apart(9)[5:]
    for bad in (x + 128, dy - 128):
        assert _err(h3.h3_adaln_modulate_backward, dy, x, t, tag, tab, bad, dtab, w, 3, 4, 64, 64, 64, 64) == INV


def test_binding_is_built():
    """The compiled binding imports without a GPU and offers the calls of the package."""
    mod = h3._binding()
    for name in ("rotate", "key_ranges", "attention", "attention_backward", "layer_norm", "layer_norm_backward",
                 "adaln_backward"):
        assert callable(getattr(mod, name))
