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
    assert size(1, 262144, 64, 1, None) >= 8 * 64 * 2
    assert size(256, 131072, 64, 1, None) == 0       # one workgroup holds a row
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
    assert st(rows=1, n=200_000, ws=None) == 1 and st(rows=1, n=200_000, nb=8) == 6
    assert st(x=ctypes.c_void_p(0x10000001)) == 9 and st(x=ctypes.c_void_p(0x10000002), dtype=2) == 9
    assert st(i=ctypes.c_void_p(0x30000004)) == 9
    assert st(rows=1, n=200_000, ws=ctypes.c_void_p(0x40000010)) == 9
    assert st(v=x) == 5 and st(i=x) == 5 and st(v=i) == 5
    assert st(v=ctypes.c_void_p(0x10000000 + 2 * (3 * 5000 + 4990))) == 5
    assert st(rows=1, n=200_000, ws=x) == 5
    assert st(opts=ctypes.byref(lrs._Options(7, 0, 0, 0, None))) == 10
    assert st(rows=0, x=None, v=None, i=None) == 0 and st(k=0, x=None, v=None, i=None) == 0


def test_binding_refusals():
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.segmented_row_topk(torch.zeros(2, 4), 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.segmented_row_topk([[1.0]], 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.topk_distill_step(torch.zeros(2, 4), torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.expert_counts(torch.zeros(2, 1, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="GPU tensor"):
        lrs.expert_balance_step(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int64))


def _distill(**kw):
    from lsd_radix_sort_amd.row_ops import _Distill
    d = dict(logits=A[0], row_stride=5000, teacher_values=A[1], teacher_stride=16, teacher_indices=A[2], index_stride=16,
             teacher_lse=None, row_weights=None, rows=4, n=5000, k=16, dtype=1, teacher_dtype=2, index_bytes=8,
             temperature=1.0)
    d.update(kw)
    return _Distill(**d)


def test_distill_workspace_sizes():
    size = lrs.load_library().topk_distill_workspace_size
    assert size(4, 5000, 16, 1, None) >= 4 * (16 + 2) * 4
    assert size(0, 5000, 16, 1, None) == 0 and size(4, 5000, 0, 1, None) == 0 and size(4, 5000, 1025, 1, None) == 0
    assert size(4, 5000, 16, 3, None) == 0 and size(4, 1 << 30, 16, 1, None) == 0


@no_gpu
def test_distill_refusals():
    lib = lrs.load_library()
    r = ctypes.byref
    loss, rl, g, ws = A[3:7]

    def step(loss=loss, rl=rl, g=g, gs=5000, ws=ws, nb=BIG, opts=None, **kw):
        return lib.topk_distill_step(r(_distill(**kw)), loss, rl, g, gs, ws, nb, None, opts)
    assert lib.topk_distill_step(None, loss, rl, g, 5000, ws, BIG, None, None) == 1
    assert step(dtype=3) == 7 and step(teacher_dtype=-1) == 7 and step(index_bytes=2) == 7
    assert step(rows=-1) == 4 and step(n=-1) == 4 and step(k=0) == 4 and step(k=1025) == 4 and step(n=1 << 30) == 4
    assert step(rows=1 << 36) == 4 and step(row_stride=-1) == 4 and step(teacher_stride=-1) == 4 and step(index_stride=-1) == 4
    assert step(gs=4999) == 4 and step(gs=-1) == 4
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert step(temperature=t) == 10
    assert step(opts=r(lrs._Options(7, 0, 0, 0, None))) == 10
    assert step(logits=None) == 1 and step(teacher_values=None) == 1 and step(teacher_indices=None) == 1
    assert step(loss=None) == 1 and step(g=None) == 1 and step(ws=None) == 1 and step(nb=64) == 6
    assert step(logits=ctypes.c_void_p(0x10000001)) == 9 and step(teacher_indices=ctypes.c_void_p(0x30000004)) == 9
    assert step(teacher_lse=ctypes.c_void_p(0x80000002)) == 9 and step(ws=ctypes.c_void_p(0x70000010)) == 9
    assert step(g=A[0]) == 5 and step(loss=A[1]) == 5 and step(rl=A[2]) == 5 and step(ws=A[0]) == 5
    assert step(g=loss) == 5 and step(rl=g) == 5 and step(ws=g) == 5
    assert step(row_weights=A[8], g=A[8]) == 5 and step(teacher_lse=A[8], rl=A[8]) == 5
    st = A[7]

    def back(stats=st, up=None, g=g, gs=5000, **kw):
        return lib.topk_distill_backward(r(_distill(**kw)), stats, up, g, gs, None, None)
    assert back(stats=None) == 1 and back(g=None) == 1 and back(gs=100) == 4 and back(dtype=9) == 7
    assert back(g=st) == 5 and back(g=A[0]) == 5 and back(up=g) == 5 and back(up=ctypes.c_void_p(0x90000001)) == 9
    assert back(rows=0) == 0
    assert lib.topk_distill_forward(r(_distill()), loss, rl, rl, ws, BIG, None, None) == 5
    assert lib.topk_distill_forward(r(_distill()), None, rl, st, ws, BIG, None, None) == 1


@no_gpu
def test_expert_refusals():
    lib = lrs.load_library()
    i, m, c, n, x, loss, g, ws = A[:8]

    def counts(i=i, stride=4, nb=8, m=m, c=c, n=n, rows=10, k=4, e=64, opts=None):
        return lib.expert_counts(i, stride, nb, m, c, n, rows, k, e, None, opts)
    assert counts(nb=2) == 7
    assert counts(rows=-1) == 4 and counts(k=-1) == 4 and counts(e=0) == 4 and counts(e=4097) == 4
    assert counts(rows=1 << 30) == 4 and counts(rows=1 << 31) == 4 and counts(stride=-1) == 4
    assert counts(i=None) == 1 and counts(c=None) == 1
    assert counts(i=ctypes.c_void_p(0x10000004)) == 9 and counts(c=ctypes.c_void_p(0x30000002)) == 9
    assert counts(c=i) == 5 and counts(c=m) == 5 and counts(n=c) == 5 and counts(n=i) == 5
    assert counts(opts=ctypes.byref(lrs._Options(7, 0, 0, 0, None))) == 10

    def bal(x=x, stride=64, c=c, n=n, m=m, rows=10, e=64, dtype=1, score=0, a=1.0, z=0.0, loss=loss, up=None, g=g, gs=64,
            ws=ws, nb=BIG):
        return lib.expert_balance(x, stride, c, n, m, rows, e, dtype, score, a, z, loss, up, g, gs, ws, nb, None, None)
    assert bal(dtype=3) == 7 and bal(score=2) == 10 and bal(score=1, z=0.1) == 10 and bal(a=float("nan")) == 10
    assert bal(z=float("inf")) == 10
    assert bal(rows=-1) == 4 and bal(e=0) == 4 and bal(e=4097) == 4 and bal(stride=-1) == 4 and bal(gs=63) == 4
    assert bal(rows=1 << 31) == 4
    assert bal(x=None) == 1 and bal(c=None) == 1 and bal(loss=None, g=None) == 1 and bal(n=None) == 1 and bal(ws=None) == 1
    assert bal(nb=4) == 6
    assert bal(x=ctypes.c_void_p(0x50000001)) == 9 and bal(ws=ctypes.c_void_p(0x80000008)) == 9
    assert bal(g=x) == 5 and bal(g=c) == 5 and bal(loss=x) == 5 and bal(ws=x) == 5 and bal(g=loss) == 5 and bal(ws=g) == 5
    assert lib.expert_balance_workspace_size(10, 64, None) > 0
    assert lib.expert_balance_workspace_size(0, 64, None) == 0 and lib.expert_balance_workspace_size(10, 4097, None) == 0


@no_gpu
def test_balance_step_refusals():
    lib = lrs.load_library()
    i, m, c, n, x, loss, g, ws = A[:8]

    def step(x=x, xs=64, i=i, istride=4, nb=8, m=m, rows=10, k=4, e=64, dtype=1, score=0, a=1.0, z=0.0, c=c, n=n, loss=loss,
             g=g, gs=64, ws=ws, wb=BIG, opts=None):
        return lib.expert_balance_step(x, xs, i, istride, nb, m, rows, k, e, dtype, score, a, z, c, n, loss, g, gs, ws, wb,
                                       None, opts)
    assert step(nb=2) == 7 and step(dtype=3) == 7
    assert step(score=2) == 10 and step(score=1, z=0.1) == 10 and step(a=float("inf")) == 10 and step(z=float("nan")) == 10
    assert step(opts=ctypes.byref(lrs._Options(7, 0, 0, 0, None))) == 10
    assert step(rows=-1) == 4 and step(k=-1) == 4 and step(e=0) == 4 and step(e=4097) == 4 and step(rows=1 << 30) == 4
    assert step(xs=-1) == 4 and step(istride=-1) == 4 and step(gs=63) == 4 and step(gs=-1) == 4
    assert step(x=None) == 1 and step(i=None) == 1 and step(c=None) == 1 and step(loss=None) == 1 and step(ws=None) == 1
    assert step(wb=lib.expert_balance_step_workspace_size(10, 4, 64, None) - 1) == 6
    assert step(x=ctypes.c_void_p(0x50000001)) == 9 and step(i=ctypes.c_void_p(0x10000004)) == 9
    assert step(c=ctypes.c_void_p(0x30000002)) == 9 and step(ws=ctypes.c_void_p(0x80000008)) == 9
    assert step(g=x) == 5 and step(g=i) == 5 and step(g=m) == 5 and step(loss=i) == 5 and step(c=i) == 5 and step(n=c) == 5
    assert step(ws=x) == 5 and step(ws=g) == 5 and step(loss=c) == 5
    size = lib.expert_balance_step_workspace_size
    assert size(-1, 4, 64, None) == 0 and size(10, 4, 4097, None) == 0 and size(0, 0, 1, None) > 0
    assert size(1 << 20, 8, 4096, None) >= 64 * 4097 * 4
