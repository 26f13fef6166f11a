"""Launches that the CUDA runtime refuses: the call reports H3_ERR_CUDA and leaves no error behind for the next one.

The refusal is made on the host: a stream whose capture has been invalidated (by a synchronisation, which capture
forbids) takes no launch, and nothing reaches the GPU.
"""
import contextlib
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.train_util import randn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RELAXED = 2


@pytest.fixture(scope="module")
def h3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import packed_mm_rope_b200 as lib
    return lib


@contextlib.contextmanager
def refusing_stream():
    """A stream with an invalidated capture."""
    rt = ctypes.CDLL("libcudart.so.12")
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamSynchronize.argtypes = [ctypes.c_void_p]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(stream.cuda_stream, RELAXED) == 0
    assert rt.cudaStreamSynchronize(stream.cuda_stream) != 0
    rt.cudaGetLastError()                            # torch's runtime; the library has its own
    graph = ctypes.c_void_p()
    try:
        yield stream
    finally:
        rt.cudaStreamEndCapture(stream.cuda_stream, ctypes.byref(graph))
        rt.cudaGetLastError()
    assert not graph.value


def _calls(h3, n=300, c=2056):
    """Every call that launches by itself, with all that it writes given."""
    q, k, v, do = (randn(i, n, h, 128) for i, h in enumerate((4, 2, 2, 4)))
    starts = torch.tensor([0, 100, n], dtype=torch.int32, device="cuda")
    ranges, lse = torch.empty(n, 2, dtype=torch.int32, device="cuda"), torch.empty(1, 4, n, device="cuda")
    h3.build_key_ranges(starts, n, out=ranges)
    o, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    h3.masked_attention(q, k, v, ranges, out=o, lse=lse)
    shape = h3.h3_attn_shape(n, n, 1, 4, 2, 128, 0.0)
    work = torch.empty(h3.h3_masked_attention_backward_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    no_rows = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    x, dy, w = randn(5, n, c), randn(6, n, c), randn(7, c, dtype=torch.float32)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    h3.layer_norm(x, w, w, out=y, mean=mean, rstd=rstd)
    table, dtable = randn(8, 6, 2, c, dtype=torch.float32), torch.empty(6, 2, c, device="cuda")
    index = torch.zeros(n, dtype=torch.int32, device="cuda")
    awork = torch.empty(h3.h3_adaln_backward_workspace_bytes(n, c, 6), dtype=torch.uint8, device="cuda")
    coords = randn(9, n, 3, dtype=torch.float32)
    B = h3.masked_attention_backward
    return {
        "ranges": lambda s: h3.build_key_ranges(starts, n, out=ranges, stream=s),
        "attention": lambda s: h3.masked_attention(q, k, v, ranges, out=o, lse=lse, stream=s),
        "attention backward": lambda s: B(do, q, k, v, o, lse, ranges, dq, dk, dv, workspace=work, stream=s),
        "backward without queries": lambda s: B(none, none, k, v, none, lse[..., :0].contiguous(), no_rows, none, dk, dv,
                                                workspace=work, stream=s),
        "rotate": lambda s: h3.mmrope_rotate(q, k, coords, q_out=dq, k_out=dk, stream=s),
        "layer norm": lambda s: h3.layer_norm(x, w, w, out=y, mean=mean, rstd=rstd, stream=s),
        "layer norm backward": lambda s: h3.layer_norm_backward(dy, x, mean, rstd, w, dx=dx, param_grads=False, stream=s),
        "adaln backward": lambda s: h3.adaln_modulate_backward(dy, x, index, index, table, dx=dx, dtable=dtable,
                                                               workspace=awork, stream=s),
        "adaln backward without rows": lambda s: h3.adaln_modulate_backward(dy[:0], x[:0], index[:0], index[:0], table,
                                                                            dx=dx[:0], dtable=dtable, workspace=awork,
                                                                            stream=s),
    }


@pytest.mark.parametrize("name", ["ranges", "attention", "attention backward", "backward without queries", "rotate",
                                  "layer norm", "layer norm backward", "adaln backward", "adaln backward without rows"])
def test_a_refused_launch_leaves_no_error_for_the_next_call(h3, name):
    q, k, v = (randn(20 + i, 70, 2, 128) for i in range(3))
    call = _calls(h3)[name]
    want = h3.packed_attention(q, k, v)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    with refusing_stream() as stream:
        with pytest.raises(h3.H3Error) as e:
            call(stream)
        assert e.value.status == h3.H3_ERR_CUDA
        h3.packed_attention(q, k, v, out=out)        # reports the thread's last error, if there is one
    assert h3.h3_check_device_error() == h3.H3_OK
    assert torch.equal(out, want)


FIRST_USE = r"""
import sys
sys.path.insert(0, ".")
import torch
import packed_mm_rope_b200 as h3
from tests.test_gpu_launch_errors import randn

n, c = 200, 2056
q, k, v, do = (randn(i, n, h, 128) for i, h in enumerate((4, 2, 2, 4)))
starts = torch.tensor([0, 120, n], dtype=torch.int32, device="cuda")
x, dy, w = randn(5, n, c), randn(6, n, c), randn(7, c, dtype=torch.float32)
table, index = randn(8, 6, 2, c, dtype=torch.float32), torch.zeros(n, dtype=torch.int32, device="cuda")
coords = randn(9, n, 3, dtype=torch.float32)
lse = torch.empty(1, 4, n, device="cuda")

def step():
    qr, kr = h3.mmrope_rotate(q, k, coords)
    r = h3.build_key_ranges(starts, n)
    o = h3.masked_attention(qr, kr, v, r, lse=lse)
    g = h3.masked_attention_backward(do, qr, kr, v, o, lse, r)
    y, mean, rstd = h3.layer_norm(x, w, w)
    return (o, *g, y, *h3.layer_norm_backward(dy, x, mean, rstd, w), *h3.adaln_modulate_backward(dy, x, index, index, table))

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert h3.h3_check_device_error() == h3.H3_OK
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_first_use_of_every_call_inside_a_capture(h3):
    """The library's first calls in a process, all of them inside a capture, as h3_init's text allows."""
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
