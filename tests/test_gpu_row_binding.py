"""The row operators' compiled binding against the Python one (which calls with
options take): the same bits, the same refusals, and autograd's manners."""
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def same(a, b):
    assert type(a) is type(b) and len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and torch.equal(x, y)


def distill_args(dtype, rows=37, n=3001, k=9, pad=3, lse=True, weights=True, wide=True):
    torch.manual_seed(rows + n)
    full = torch.randn(rows, n, device="cuda") * 2
    s = torch.zeros(rows, n + pad, device="cuda", dtype=dtype)[:, :n]
    s.copy_(full * 0.5 + torch.randn(rows, n, device="cuda"))
    v, i = lrs.segmented_row_topk(full, k)
    w = torch.rand(rows, device="cuda") / rows
    return (s, v.to(dtype), i if wide else i.int(), 1.5, torch.logsumexp(full / 1.5, 1) if lse else None, w if weights else None)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_same_as_python(dtype):
    opts = lrs.SortOptions()
    x = torch.randn(50, 1003, device="cuda").to(dtype)
    for k in (0, 1, 40):
        for descending in (True, False):
            same(lrs.segmented_row_topk(x[:, 2:], k, descending), lrs.segmented_row_topk(x[:, 2:], k, descending, options=opts))
    for lse, weights, wide in ((True, True, True), (False, False, False)):
        args = distill_args(dtype, lse=lse, weights=weights, wide=wide)
        same(lrs.topk_distill_step(*args), lrs.topk_distill_step(*args, options=opts))
        same(lrs.topk_distill_forward(*args), lrs.topk_distill_forward(*args, options=opts))
    r = torch.randn(500, 40, device="cuda").to(dtype)
    _, ids = lrs.segmented_row_topk(r, 3)
    mask = torch.rand(500, device="cuda") < 0.7
    for m in (None, mask, mask.to(torch.uint8)):
        for score in ("softmax", "sigmoid"):
            same(lrs.expert_balance_step(r, ids, 0.3, 0.0, score, m), lrs.expert_balance_step(r, ids, 0.3, 0.0, score, m, options=opts))
            same(lrs.expert_balance_forward(r, ids.int(), 0.3, 0.0, score, m),
                 lrs.expert_balance_forward(r, ids.int(), 0.3, 0.0, score, m, options=opts))


def test_refusals():
    s, v, i, t, lse, w = distill_args(torch.bfloat16)
    for call in (lrs.topk_distill_step, lrs.topk_distill_forward, lrs.topk_distill_loss):
        for bad in ((s.cpu(), v, i), (s, v[:-1], i), (s, v, i[:, :-1]), (s, v, i.float()), (s.double(), v, i), (s.T, v, i)):
            with pytest.raises(ValueError):
                call(*bad)
        with pytest.raises(ValueError):
            call(s, v, i, 0.0)
        with pytest.raises(ValueError):
            call(s, v, i, 1.0, lse[:-1])
        with pytest.raises(ValueError):
            call(s, v, i, 1.0, lse, w.double())
    r = torch.randn(20, 8, device="cuda")
    ids = torch.zeros(20, 2, dtype=torch.int64, device="cuda")
    for call in (lrs.expert_balance_step, lrs.expert_balance_forward, lrs.expert_balance_loss):
        for bad in ((r, ids[:-1]), (r, ids.float()), (r.cpu(), ids), (r.int(), ids)):
            with pytest.raises(ValueError):
                call(*bad)
        with pytest.raises(ValueError):
            call(r, ids, 1.0, 0.0, "relu")
        with pytest.raises(ValueError):
            call(r, ids, 1.0, 0.5, "sigmoid")
        with pytest.raises(ValueError):
            call(r, ids, 1.0, 0.0, "softmax", torch.ones(19, dtype=torch.bool, device="cuda"))
    for k in (-1, 9):
        with pytest.raises(ValueError):
            lrs.segmented_row_topk(r, k)


def losses():
    s, v, i, t, lse, w = distill_args(torch.float32, pad=0)
    r = torch.randn(300, 24, device="cuda")
    _, ids = lrs.segmented_row_topk(r, 2)
    return ((s, lambda x: lrs.topk_distill_loss(x, v, i, t, lse, w)), (r, lambda x: lrs.expert_balance_loss(x, ids, 0.5, 1e-2)[0]))


def test_autograd_manners():
    for x, f in losses():
        leaf = x.clone().requires_grad_(True)
        plain, = torch.autograd.grad(f(leaf), leaf)
        # a graph of the backward may be asked for, but not followed
        again, = torch.autograd.grad(f(leaf), leaf, create_graph=True)
        assert torch.equal(again.detach(), plain)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(again.sum(), leaf, retain_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            again.sum().backward()
        # what is saved may be moved by hooks
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
            loss = f(leaf)
        moved, = torch.autograd.grad(loss, leaf)
        assert torch.equal(moved, plain)
        # inside a larger program, and summed into .grad
        (3 * f(leaf * 1.0)).backward()
        f(leaf).backward()
        assert torch.allclose(leaf.grad, 4 * plain, rtol=1e-5, atol=1e-9)
        # logits changed after the forward are noticed
        y = x.clone().requires_grad_(True) * 1.0
        loss = f(y)
        y.add_(1.0)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
        with torch.no_grad():
            assert not f(leaf).requires_grad
        assert not f(x).requires_grad


def test_backward_on_another_stream():
    for x, f in losses():
        leaf = x.clone().requires_grad_(True)
        plain, = torch.autograd.grad(f(leaf), leaf)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            there, = torch.autograd.grad(f(leaf), leaf)
        side.synchronize()
        assert torch.equal(there, plain)
