"""Host-side checks of the row operators: sizes, refusals of the C ABI before
anything is enqueued, and refusals of the binding.  No kernel runs here."""
import ctypes

import pytest
import torch

import lsd_radix_sort_amd as lrs


def _gpu_present():
    try:
        return torch.cuda.is_available()
    except Exception:
        return False


# fake device addresses, passed only where validation must reject the call
A = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(10)]
BIG = 1 << 40
no_gpu = pytest.mark.skipif(_gpu_present(), reason="fake-pointer validation runs only without a GPU")


def test_topk_workspace_sizes():
    size = lrs.load_library().segmented_row_topk_workspace_size
    assert size(1, 131072, 64, 1, None) >= 8 * 64 * 2
    assert size(256, 131072, 64, 1, None) == 0       # enough rows: one workgroup each
    assert size(4, 1000, 10, 0, None) == 0           # too short to share
    assert size(0, 131072, 64, 1, None) == 0 and size(1, 131072, 0, 1, None) == 0
    assert size(1, 131072, 1025, 1, None) == 0       # k beyond the limit
    assert size(1, 131072, 64, 3, None) == 0         # no such type
    assert size(1, 131072, 64, 1, ctypes.byref(lrs._Options(7, 0, 0, 0, None))) == 0


@no_gpu
def test_topk_refusals():
    f = lrs.load_library().segmented_row_topk
    x, v, i, ws = A[:4]

    def st(x=x, stride=5000, v=v, i=i, rows=4, n=5000, k=10, dtype=0, ws=ws, nb=BIG, opts=None):
        return f(x, stride, v, i, rows, n, k, dtype, 1, ws, nb, None, opts)
    assert st(dtype=3) == 7 and st(dtype=-1) == 7
    assert st(rows=-1) == 4 and st(n=-1) == 4 and st(k=-1) == 4 and st(stride=-1) == 4
    assert st(k=5001) == 4 and st(k=1025) == 4 and st(n=1 << 30) == 4
    assert st(rows=1 << 30, n=2048) == 4 and st(rows=1 << 39, n=1, k=1, stride=1 << 20) == 4
    assert st(x=None) == 1 and st(v=None) == 1 and st(i=None) == 1
    assert st(rows=1, n=100_000, ws=None) == 1 and st(rows=1, n=100_000, nb=8) == 6
    assert st(x=ctypes.c_void_p(0x10000001)) == 9 and st(x=ctypes.c_void_p(0x10000002), dtype=2) == 9
    assert st(i=ctypes.c_void_p(0x30000004)) == 9
    assert st(rows=1, n=100_000, ws=ctypes.c_void_p(0x40000010)) == 9
    assert st(v=x) == 5 and st(i=x) == 5 and st(v=i) == 5
    assert st(v=ctypes.c_void_p(0x10000000 + 2 * (3 * 5000 + 4990))) == 5
    assert st(rows=1, n=100_000, ws=x) == 5
    assert st(opts=ctypes.byref(lrs._Options(7, 0, 0, 0, None))) == 10
    assert st(rows=0, x=None, v=None, i=None) == 0 and st(k=0, x=None, v=None, i=None) == 0


def test_binding_refusals():
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.segmented_row_topk(torch.zeros(2, 4), 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.segmented_row_topk([[1.0]], 1)
