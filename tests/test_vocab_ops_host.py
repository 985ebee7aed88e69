"""Host-side checks of the vocabulary operators: sizes, refusals of the C ABI
before anything is enqueued, and refusals of the binding.  No kernel runs here."""
import ctypes
import math

import pytest
import torch

import lsd_radix_sort_amd as lrs
from lsd_radix_sort_amd.vocab_ops import _Logprobs, _TokenIds


def _gpu_present():
    try:
        return torch.cuda.is_available()
    except Exception:
        return False


# fake device addresses, passed only where validation must reject the call
A = [0x10000000000 * (i + 1) for i in range(10)]
BIG = 1 << 40
no_gpu = pytest.mark.skipif(_gpu_present(), reason="fake-pointer validation runs only without a GPU")
P = ctypes.c_void_p
BAD_OPTIONS = lrs._Options(7, 0, 0, 0, None)


def test_workspace_sizes():
    size = lrs.embedding_backward_workspace_size
    assert size(0, 1000, 64) == 0 and size(100, 0, 64) == 0 and size(100, 1000, 0) == 0
    assert size(100, 1000, 64) >= 8 * 100
    assert size(40000, 1000, 64) >= lrs.radix_sort_workspace_size(40000, 0, 10, 8, True) + 16 * 40000
    assert size(-1, 10, 10) == 0 and size(1 << 31, 10, 10) == 0 and size(10, 1 << 31, 10) == 0 and size(10, 10, 1 << 30) == 0
    assert size(1 << 20, 10, 1 << 20) == 0  # 2^40 elements
    lib = lrs.load_library()
    assert lib.embedding_backward_workspace_size(100, 1000, 64, ctypes.byref(BAD_OPTIONS)) == 0
    size = lrs.token_logprobs_workspace_size
    assert size(0, 1000) == 0 and size(4, 1000, 1001) == 0 and size(4, 2000, 1025) == 0 and size(-1, 4) == 0 and size(4, -1) == 0
    assert size(4, 1 << 30) == 0 and size(1 << 30, 2048) == 0
    assert size(2, 100_000, 20) >= 8 * 20 * 2  # pieces' words
    with pytest.raises(lrs.RadixSortArgumentError, match="float16"):
        size(4, 1000, 8, torch.float64)
    assert lib.token_logprobs_workspace_size(4, 1000, 8, 3, None) == 0
    assert lib.token_logprobs_workspace_size(4, 1000, 8, 1, ctypes.byref(BAD_OPTIONS)) == 0


@no_gpu
def test_embedding_forward_refusals():
    f = lrs.load_library().embedding_forward

    def st(weight=A[0], stride=64, ids=A[1], lines=4, length=8, id_stride=8, id_bytes=8, out=A[2], out_stride=64, vocab=100, width=64,
           dtype=1, out_dtype=1, scale=1.0, opts=None, no_ids=False):
        t = _TokenIds(ids, lines, length, id_stride, id_bytes)
        return f(P(weight), stride, None if no_ids else ctypes.byref(t), P(out), out_stride, vocab, width, dtype, out_dtype, scale, None, opts)
    assert st(dtype=3) == 7 and st(out_dtype=-1) == 7 and st(id_bytes=2) == 7
    assert st(lines=-1) == 4 and st(length=-1) == 4 and st(id_stride=-1) == 4 and st(vocab=-1) == 4 and st(width=-1) == 4
    assert st(lines=1 << 20, length=1 << 20) == 4 and st(vocab=1 << 31) == 4 and st(width=1 << 30) == 4
    assert st(lines=1 << 10, length=1 << 20, width=1 << 11, out_stride=1 << 11) == 4
    assert st(stride=-1) == 4 and st(out_stride=63) == 4
    assert st(weight=None) == 1 and st(out=None) == 1 and st(ids=None) == 1 and st(no_ids=True) == 1
    assert st(weight=A[0] + 1) == 9 and st(out=A[2] + 1) == 9 and st(ids=A[1] + 4) == 9 and st(ids=A[1] + 2, id_bytes=4) == 9
    assert st(out_dtype=2, out=A[2] + 2) == 9
    assert st(out=A[0]) == 5 and st(out=A[1]) == 5 and st(out=A[0] + 2 * (99 * 64 + 63)) == 5
    assert st(scale=math.inf) == 10 and st(scale=math.nan) == 10 and st(opts=ctypes.byref(BAD_OPTIONS)) == 10
    assert st(lines=0, out=None, ids=None) == 0 and st(width=0, out=None) == 0


@no_gpu
def test_embedding_backward_refusals():
    f = lrs.load_library().embedding_backward

    def st(grad=A[0], stride=64, ids=A[1], lines=4, length=8, id_stride=8, id_bytes=8, out=A[2], out_stride=64, vocab=100, width=64,
           dtype=1, out_dtype=2, scale=1.0, padding=-1, add=0, ws=A[3], nb=BIG, opts=None):
        t = _TokenIds(ids, lines, length, id_stride, id_bytes)
        return f(P(grad), stride, ctypes.byref(t), P(out), out_stride, vocab, width, dtype, out_dtype, scale, padding, add, P(ws), nb,
                 None, opts)
    assert st(dtype=3) == 7 and st(out_dtype=-1) == 7 and st(id_bytes=1) == 7
    assert st(lines=-1) == 4 and st(vocab=1 << 31) == 4 and st(width=1 << 30) == 4 and st(stride=-1) == 4 and st(out_stride=63) == 4
    assert st(vocab=1 << 30, width=1 << 10, out_stride=1 << 10) == 4
    assert st(grad=None) == 1 and st(out=None) == 1 and st(ids=None) == 1 and st(ws=None) == 1
    assert st(grad=A[0] + 1) == 9 and st(out=A[2] + 2) == 9 and st(ids=A[1] + 4) == 9 and st(ws=A[3] + 16) == 9
    assert st(nb=8) == 6
    assert st(out=A[0]) == 5 and st(out=A[1]) == 5 and st(ws=A[0]) == 5 and st(ws=A[1]) == 5 and st(ws=A[2]) == 5
    assert st(scale=math.nan) == 10 and st(opts=ctypes.byref(BAD_OPTIONS)) == 10
    assert st(vocab=0) == 0 and st(width=0) == 0


@no_gpu
def test_token_logprobs_refusals():
    lib = lrs.load_library()

    def arguments(logits=A[0], stride=5000, tokens=A[1], token_stride=1, token_bytes=8, dtype=1, mask=None, rows=4, n=5000, temperature=1.0):
        return _Logprobs(logits, stride, tokens, token_stride, token_bytes, dtype, mask, rows, n, temperature)

    def forward(lp=A[2], h=A[3], stats=A[4], ws=A[5], nb=BIG, opts=None, **kw):
        return lib.token_logprobs_forward(ctypes.byref(arguments(**kw)), P(lp), P(h), P(stats), P(ws), nb, None, opts)

    def topk(k=8, lp=A[2], h=A[3], ranks=A[4], top=A[6], idx=A[7], ws=A[5], nb=BIG, opts=None, **kw):
        return lib.token_logprobs_topk(ctypes.byref(arguments(**kw)), k, P(lp), P(h), P(ranks), P(top), P(idx), P(ws), nb, None, opts)

    def step(up=A[6], down=A[7], lp=A[2], h=A[3], grad=A[8], grad_stride=5000, ws=A[5], nb=BIG, opts=None, **kw):
        return lib.token_logprobs_step(ctypes.byref(arguments(**kw)), P(up), P(down), P(lp), P(h), P(grad), grad_stride, P(ws), nb, None, opts)

    def backward(stats=A[4], up=A[6], down=A[7], grad=A[8], grad_stride=5000, opts=None, **kw):
        return lib.token_logprobs_backward(ctypes.byref(arguments(**kw)), P(stats), P(up), P(down), P(grad), grad_stride, None, opts)

    for f in (forward, topk, step, backward):
        assert f(dtype=3) == 7 and f(token_bytes=2) == 7
        assert f(rows=-1) == 4 and f(n=-1) == 4 and f(n=1 << 30) == 4 and f(stride=-1) == 4 and f(token_stride=-1) == 4
        assert f(rows=1 << 30, n=2048) == 4
        for t in (0.0, -1.0, math.inf, math.nan, 1e-40):
            assert f(temperature=t) == 10
        assert f(opts=ctypes.byref(BAD_OPTIONS)) == 10
        assert f(logits=None) == 1 and f(tokens=None) == 1
        assert f(logits=A[0] + 1) == 9 and f(tokens=A[1] + 4) == 9
        assert f(rows=0) == 0
    assert forward(lp=None) == 1 and forward(h=None) == 1 and forward(ws=None) == 1
    assert forward(lp=A[2] + 2) == 9 and forward(ws=A[5] + 8) == 9 and forward(nb=0) == 6
    assert forward(lp=A[0]) == 5 and forward(h=A[2]) == 5 and forward(ws=A[1]) == 5
    assert forward(stats=A[0] + 2 * (3 * 5000 + 4999)) == 9 and forward(stats=A[0] + 2 * (3 * 5000 + 4998)) == 5
    assert forward(mask=A[2]) == 5
    assert topk(k=-1) == 4 and topk(k=5001) == 4 and topk(k=1025) == 4 and topk(mask=A[9]) == 10
    assert topk(ranks=None) == 1 and topk(top=None) == 1 and topk(idx=None) == 1 and topk(idx=A[7] + 4) == 9
    assert topk(top=A[0]) == 5 and topk(idx=A[6]) == 5 and topk(ranks=A[1]) == 5 and topk(n=100_000, stride=100_000, nb=8) == 6
    assert step(up=None, down=None) == 1 and step(grad=None) == 1 and step(grad_stride=4999) == 4 and step(grad_stride=-1) == 4
    assert step(grad=A[0]) == 5 and step(grad=A[6]) == 5 and step(lp=A[7]) == 5 and step(grad=A[8] + 1) == 9 and step(up=A[6] + 2) == 9
    assert backward(up=None, down=None) == 1 and backward(stats=None) == 1 and backward(grad=None) == 1 and backward(grad_stride=4999) == 4
    assert backward(grad=A[0]) == 5 and backward(grad=A[4]) == 5 and backward(grad=A[7]) == 5 and backward(stats=A[4] + 2) == 9
    assert backward(n=0) == 0


def test_binding_refusals():
    weight, tokens, logits = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8)
    for call in (lambda: lrs.embedding_forward(weight, tokens), lambda: lrs.embedding_lookup(weight, tokens),
                 lambda: lrs.embedding_backward(logits, tokens, 4), lambda: lrs.token_logprobs(logits, tokens),
                 lambda: lrs.token_logprobs_forward(logits, tokens), lambda: lrs.token_logprobs_topk(logits, tokens, 2),
                 lambda: lrs.token_logprobs_step(logits, tokens, torch.ones(3))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for scale in ("much", None, [1.0]):
        with pytest.raises(lrs.RadixSortArgumentError, match="scale"):
            lrs.embedding_forward(weight, tokens, scale)
    for vocab in (2.5, -1, 1 << 31, None):
        with pytest.raises(lrs.RadixSortArgumentError, match="vocab"):
            lrs.embedding_backward(logits, tokens, vocab)
    for k in (2.5, "2", None, -1, 1025, 1 << 70):
        with pytest.raises(lrs.RadixSortArgumentError, match="k must be"):
            lrs.token_logprobs_topk(logits, tokens, k)
    with pytest.raises(lrs.RadixSortArgumentError, match="temperature"):
        lrs.token_logprobs(logits, tokens, "hot")
