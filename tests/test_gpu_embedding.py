"""The embedding lookup and its gradient by sorted tokens against the formulas in
64 bits on the CPU, over types, widths, strides, numbers of tokens and the ways
that ids can fall; the gradient also against differences."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = 2.0 ** -24  # half a step of 32-bit numbers


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half a step below the smallest normal number."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def padded(x, pad):
    if pad == 0:
        return x
    buf = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device=x.device)
    buf[:, pad // 2:pad // 2 + x.shape[1]] = x
    return buf[:, pad // 2:pad // 2 + x.shape[1]]


def make_ids(kind, shape, vocab, g):
    if kind == "same":
        ids = torch.full(shape, vocab - 1)
    elif kind == "text":  # few ids make up much of it
        ids = ((vocab + 1.0) ** torch.rand(shape, generator=g, dtype=torch.float64) - 1).long().clamp_(0, vocab - 1)
    elif kind == "runs":  # sorted already, every id as often as its neighbours
        ids = (torch.arange(shape.numel()) * vocab // max(1, shape.numel())).reshape(shape)
    elif kind == "outside":  # none that counts
        ids = torch.where(torch.rand(shape, generator=g) < 0.5, -1, vocab)
    else:
        ids = torch.randint(-1, vocab + 1, shape, generator=g)
    return ids


def lookup_reference(weight, ids, scale):
    vocab, width = weight.shape
    table = torch.zeros(vocab + 1, width, dtype=torch.float64)
    table[:vocab] = weight.double() * scale
    return table[torch.where((ids >= 0) & (ids < vocab), ids.long(), vocab)]


def gradient_reference(grad, ids, vocab, scale, padding=None):
    """The gradient, the sum of its terms' absolute values and how many there are."""
    width = grad.shape[-1]
    ids, grad = ids.reshape(-1).long(), grad.reshape(-1, width).double() * scale
    skip = (ids < 0) | (ids >= vocab)
    if padding is not None:
        skip |= ids == padding
    ids = torch.where(skip, vocab, ids)
    total, size = (torch.zeros(vocab + 1, width, dtype=torch.float64) for _ in range(2))
    total.index_add_(0, ids, grad)
    size.index_add_(0, ids, grad.abs())
    return total[:vocab], size[:vocab], torch.bincount(ids, minlength=vocab + 1)[:vocab]


def check_gradient(got, grad, ids, vocab, scale, padding=None, old=None):
    want, size, count = gradient_reference(grad, ids, vocab, scale, padding)
    if old is not None:
        want, size = want + old.double(), size + old.double().abs()
    # a sum of c terms in 32 bits is off by at most c half steps of the terms' absolute sum; one more for the scale
    # and one for what it is added to
    tol = (count[:, None] + 2) * ULP * size + half_step(got.dtype) * want.abs() * (1 + 1e-6) + smallest(got.dtype)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off - tol).max())} over the tolerance"
    none = count == 0
    assert torch.equal(got[none], torch.zeros_like(got[none]) if old is None else old[none])


WIDTHS = [1, 7, 8, 33, 64, 129, 256, 520, 1031, 4096]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_lookup(dtype, out, width):
    g = torch.Generator().manual_seed(width)
    for shape, vocab, pad, id_type, scale in (((3, 17), 101, 0, torch.int64, 1.0), ((205,), 1000, 5, torch.int32, 11.3),
                                              ((1,), 1, 0, torch.int64, -0.5), ((2, 3, 4), 50, 1, torch.int64, 2.0)):
        log(f"lookup {dtype} -> {out} width {width} tokens {shape} pad {pad}")
        weight = torch.randn(vocab, width, generator=g).to(DTYPES[dtype])
        ids = make_ids("any", torch.Size(shape), vocab, g).to(id_type)
        got = lrs.embedding_forward(padded(weight.cuda(), pad), ids.cuda(), scale, DTYPES[out]).cpu()
        want = lookup_reference(weight, ids, scale)
        assert got.shape == want.shape and got.dtype == DTYPES[out]
        tol = (half_step(got.dtype) + 2 * ULP) * want.abs() + smallest(got.dtype)
        assert bool(((got.double() - want).abs() <= tol).all())
        if scale == 1.0 and dtype == out:
            assert torch.equal(got.double(), want)


def test_lookup_of_slices_and_into_buffers():
    g = torch.Generator().manual_seed(1)
    weight = torch.randn(77, 40, generator=g).cuda()
    batch = torch.randint(-2, 80, (9, 31), generator=g)
    for ids in (batch[:, :-1], batch[:, 1:], batch[:, 3], batch[2:7, 5:9], batch[::2, :4], batch[:, :1], batch[4, ::3]):
        ids = batch.cuda().as_strided(ids.shape, ids.stride(), ids.storage_offset())
        out = torch.full((*ids.shape, 48), 5.0, device="cuda")[..., 4:44]
        want = lookup_reference(weight.cpu(), ids.cpu(), 3.0)
        assert torch.equal(lrs.embedding_forward(weight, ids, 3.0).cpu(), want.float())
        assert lrs.embedding_forward(weight, ids, 3.0, out=out) is out
        assert torch.equal(out.cpu(), want.float())
        whole = out.as_strided((out.numel() // 40, 48), (48, 1), 0)
        assert bool((whole[:, :4] == 5).all()) and bool((whole[:, 44:] == 5).all())


def test_lookup_keeps_special_values():
    for dtype in DTYPES.values():
        weight = torch.tensor([[float("inf"), -float("inf"), float("nan"), -0.0, torch.finfo(dtype).tiny / 4] * 5]).to(dtype).cuda()
        got = lrs.embedding_forward(weight, torch.tensor([0, 1, -1], device="cuda"))
        view = {2: torch.int16, 4: torch.int32}[dtype.itemsize]
        bits, kept = weight[0].view(view), got[0].view(view)
        same = ~torch.isnan(weight[0])
        assert torch.equal(bits[same], kept[same]) and bool(torch.isnan(got[0][~same]).all())
        assert not bool(got[1:].view(view).any())  # no row: zeros, whatever the table holds


@pytest.mark.parametrize("dtype,out", [("fp16", "fp16"), ("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "fp16")])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 63, 64, 65, 200, 1000, 8192, 8193, 20011])
def test_gradient(dtype, out, tokens):
    g = torch.Generator().manual_seed(tokens)
    for kind, vocab, width, pad in (("any", 97, 72, 0), ("text", 5003, 40, 3), ("same", 11, 129, 0), ("runs", 301, 64, 8),
                                    ("outside", 50, 16, 0), ("text", 40, 520, 0)):
        log(f"gradient {dtype} -> {out} tokens {tokens} {kind} vocab {vocab} width {width}")
        ids = make_ids(kind, torch.Size((tokens,)), vocab, g)
        grad = torch.randn(tokens, width, generator=g).to(DTYPES[dtype])
        args = (padded(grad.cuda(), pad), ids.cuda(), vocab, 1.7)
        got = lrs.embedding_backward(*args, dtype=DTYPES[out])
        check_gradient(got.cpu(), grad, ids, vocab, 1.7)
        assert torch.equal(got, lrs.embedding_backward(*args, dtype=DTYPES[out]))  # bit for bit


@pytest.mark.parametrize("dtype,out", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("tokens,vocab,width,pad", [(2048, 700, 128, 0), (2047, 33, 121, 5), (1000, 5003, 261, 0), (130, 40, 2015, 1),
                                                    (60, 9, 4096, 0), (2049, 500, 40, 0), (2048, 700, 129, 0), (100, 40_000, 420, 0),
                                                    (1025, 513, 250, 2), (17, 100_003, 130, 0)])
def test_gradient_of_few_tokens(dtype, out, tokens, vocab, width, pad):
    """One launch's work and what is just too much for that, added and not."""
    g = torch.Generator().manual_seed(tokens + width)
    for kind in ("any", "text", "same", "runs", "outside"):
        log(f"few {dtype} -> {out} {tokens} {vocab} {width} {kind}")
        ids = make_ids(kind, torch.Size((tokens,)), vocab, g)
        grad = torch.randn(tokens, width, generator=g).to(DTYPES[dtype])
        lines = torch.full((tokens, 3), vocab // 2)
        lines[:, 1] = ids
        ours = lines.int().cuda()[:, 1] if kind == "runs" else ids.cuda()
        args = (padded(grad.cuda(), pad), ours, vocab, 0.9)
        got = lrs.embedding_backward(*args, padding_index=vocab // 3, dtype=DTYPES[out])
        check_gradient(got.cpu(), grad, ids, vocab, 0.9, vocab // 3)
        old = torch.randn(vocab, width, generator=g).to(DTYPES[out])
        sums = [padded(old.cuda(), pad) for _ in range(2)]
        for s in sums:
            lrs.embedding_backward(*args, grad_out=s, accumulate=True)
        assert torch.equal(*sums)
        check_gradient(sums[0].cpu(), grad, ids, vocab, 0.9, old=old)


@pytest.mark.parametrize("width", WIDTHS)
def test_gradient_widths(width):
    g = torch.Generator().manual_seed(width)
    for dtype, tokens, vocab in (("bf16", 700, 60), ("fp32", 90, 1500), ("fp16", 3, 2)):
        ids = make_ids("text", torch.Size((tokens,)), vocab, g).int()
        grad = torch.randn(tokens, width, generator=g).to(DTYPES[dtype])
        check_gradient(lrs.embedding_backward(grad.cuda(), ids.cuda(), vocab).cpu(), grad, ids, vocab, 1.0)


@pytest.mark.parametrize("tokens,vocab,width,kind", [(65536, 3001, 24, "text"), (65537, 3001, 24, "text"), (140003, 40, 136, "text"),
                                                     (70001, 200_003, 8, "any"), (66000, 65536, 16, "runs"), (90000, 9, 8, "outside"),
                                                     (500, 300_001, 12, "any"), (3000, 1 << 20, 9, "text"),
                                                     (3000, (1 << 20) + 1, 9, "any"), (40, 2_000_003, 4, "any")])
def test_gradient_of_many_tokens_and_large_tables(tokens, vocab, width, kind):
    g = torch.Generator().manual_seed(tokens + vocab)
    ids = make_ids(kind, torch.Size((tokens,)), vocab, g)
    grad = torch.randn(tokens, width, generator=g).to(torch.bfloat16)
    args = (grad.cuda(), ids.cuda(), vocab, 0.3)
    got = lrs.embedding_backward(*args, dtype=torch.float32)
    check_gradient(got.cpu(), grad, ids, vocab, 0.3)
    assert torch.equal(got, lrs.embedding_backward(*args, dtype=torch.float32))


@pytest.mark.parametrize("out", DTYPES)
def test_gradient_accumulates(out):
    g = torch.Generator().manual_seed(5)
    for tokens, vocab, width, pad in ((500, 300, 36, 4), (3000, 20, 135, 1), (1, 5, 8, 0), (40, 10000, 515, 0)):
        old = torch.randn(vocab, width, generator=g).to(DTYPES[out])
        old[0, 0] = float("nan")  # no token names row 0: it stays
        ids = make_ids("text", torch.Size((tokens,)), vocab - 1, g) + 1
        grad = torch.randn(tokens, width, generator=g).to(torch.bfloat16)
        buf = padded(old.cuda(), pad)
        assert lrs.embedding_backward(grad.cuda(), ids.cuda(), vocab, 0.5, grad_out=buf, accumulate=True) is buf
        got = buf.cpu()
        assert bool(torch.isnan(got[0, 0]))
        got[0, 0] = old[0, 0] = 0
        check_gradient(got, grad, ids, vocab, 0.5, old=old)
        if pad:
            whole = buf.as_strided((vocab, width + pad), (width + pad, 1), 0)
            assert bool((whole[:, :pad // 2] == 7).all()) and bool((whole[:, pad // 2 + width:] == 7).all())


def test_gradient_into_a_buffer_and_padding():
    g = torch.Generator().manual_seed(6)
    ids = make_ids("text", torch.Size((4, 250)), 120, g)
    grad = torch.randn(4, 250, 50, generator=g)
    for padding in (None, 0, 119, int(ids[0, 0])):
        buf = torch.full((120, 64), 9.0, device="cuda", dtype=torch.bfloat16)
        got = lrs.embedding_backward(grad.cuda(), ids.cuda(), 120, 2.0, padding, grad_out=buf[:, 3:53])
        check_gradient(got.cpu(), grad, ids, 120, 2.0, padding)
        assert bool((buf[:, :3] == 9).all()) and bool((buf[:, 53:] == 9).all())


def test_nothing_to_do():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    weight = torch.randn(5, 6, device="cuda")
    assert lrs.embedding_forward(weight, none).shape == (0, 6)
    assert lrs.embedding_forward(weight[:0], torch.tensor([0, 3], device="cuda")).tolist() == [[0.0] * 6] * 2
    assert lrs.embedding_forward(weight[:, :0], torch.tensor([1], device="cuda")).shape == (1, 0)
    assert not bool(lrs.embedding_backward(torch.empty(0, 6, device="cuda"), none, 5).any())
    kept = weight.clone()
    lrs.embedding_backward(torch.empty(0, 6, device="cuda"), none, 5, grad_out=kept, accumulate=True)
    assert torch.equal(kept, weight)
    one = torch.ones(1, 6, device="cuda")
    assert lrs.embedding_backward(one, torch.tensor([0], device="cuda"), 0).shape == (0, 6)
    assert lrs.embedding_backward(one[:, :0], torch.tensor([0], device="cuda"), 5).shape == (5, 0)


def test_autograd():
    g = torch.Generator().manual_seed(7)
    ids = make_ids("text", torch.Size((6, 40)), 90, g)
    for dtype, out in ((torch.float32, None), (torch.bfloat16, None), (torch.float32, torch.bfloat16)):
        weight = torch.randn(90, 24, generator=g).to(dtype).cuda().requires_grad_(True)
        rows = lrs.embedding_lookup(weight, ids.cuda(), 3.0, padding_index=2, dtype=out)
        assert torch.equal(rows, lrs.embedding_forward(weight, ids.cuda(), 3.0, out))
        up = torch.randn(rows.shape, generator=g).to(rows.dtype)
        rows.backward(up.cuda())
        assert weight.grad.dtype == dtype
        check_gradient(weight.grad.cpu(), up, ids, 90, 3.0, 2)
        weight.grad = None
        lrs.embedding_lookup(weight, ids.cuda()).sum().backward()  # one number, expanded
        check_gradient(weight.grad.cpu(), torch.ones(6, 40, 24).to(dtype), ids, 90, 1.0)
        with pytest.raises(RuntimeError):
            first, = torch.autograd.grad(lrs.embedding_lookup(weight, ids.cuda()).float().pow(2).sum(), weight, create_graph=True)
            torch.autograd.grad(first.sum(), weight)


def test_gradient_against_differences():
    """sum(up * lookup) is linear in the table: a difference of two lookups is the gradient times the step, exactly in
    64 bits up to the roundings of the lookups."""
    g = torch.Generator().manual_seed(8)
    ids = make_ids("text", torch.Size((50,)), 12, g).cuda()
    weight, step = (torch.randn(12, 10, generator=g).cuda() for _ in range(2))
    up = torch.randn(50, 10, generator=g).cuda()
    grad = lrs.embedding_backward(up, ids, 12, 1.5)
    plus, minus = lrs.embedding_forward(weight + step, ids, 1.5).double(), lrs.embedding_forward(weight - step, ids, 1.5).double()
    change = float((up.double() * (plus - minus)).sum() / 2)
    size = float((up.double().abs() * (plus.abs() + minus.abs() + 2)).sum())
    # per element: the sums weight +- step, the products and the gradient's 50 terms each round
    assert abs(change - float((grad.double() * step.double()).sum())) <= 60 * ULP * size


def test_stream_and_graph():
    g = torch.Generator().manual_seed(9)
    weight = torch.randn(3000, 200, generator=g).to(torch.bfloat16).cuda()
    for tokens in (300, 9000):
        ids = make_ids("text", torch.Size((tokens,)), 3000, g).cuda()
        up = torch.randn(tokens, 200, generator=g).to(torch.bfloat16).cuda()
        want = lrs.embedding_forward(weight, ids, 2.0), lrs.embedding_backward(up, ids, 3000, 2.0)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = lrs.embedding_forward(weight, ids, 2.0), lrs.embedding_backward(up, ids, 3000, 2.0)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        graph = torch.cuda.CUDAGraph()
        fixed_ids, fixed_up = ids.clone(), up.clone()
        with torch.cuda.graph(graph):
            rows = lrs.embedding_forward(weight, fixed_ids, 2.0)
            grad = lrs.embedding_backward(fixed_up, fixed_ids, 3000, 2.0)
        for turn in range(3):
            new = make_ids("any", torch.Size((tokens,)), 3000, g).cuda()
            fixed_ids.copy_(new)
            fixed_up.copy_(up * (turn + 1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(rows, lrs.embedding_forward(weight, new, 2.0))
            assert torch.equal(grad, lrs.embedding_backward(up * (turn + 1), new, 3000, 2.0))


def test_rows_far_apart():
    """Rows more than 2^32 bytes from the first."""
    ids = torch.tensor([0, 65536, 3, 65536, 65535], device="cuda")
    buf = torch.zeros(65537 * 33000, dtype=torch.bfloat16, device="cuda")
    weight = buf.as_strided((65537, 16), (33000, 1))
    weight[65536] = 2.0
    weight[65535] = 3.0
    got = lrs.embedding_forward(weight, ids)
    assert got[:, 0].tolist() == [0.0, 2.0, 0.0, 2.0, 3.0]
    grad = torch.ones(5, 16, dtype=torch.bfloat16, device="cuda")
    lrs.embedding_backward(grad, ids, 65537, grad_out=weight)
    assert weight[65536, 15].item() == 2 and weight[65535, 0].item() == 1 and float(weight.sum(dtype=torch.float64)) == 80
    up = buf.as_strided((65537, 16), (33000, 1))
    up.fill_(1.0)
    assert lrs.embedding_backward(up, torch.zeros(65537, dtype=torch.int32, device="cuda"), 1, dtype=torch.float32).tolist() == [[65537.0] * 16]
