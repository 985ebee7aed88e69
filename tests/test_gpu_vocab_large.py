"""The vocabulary operators at the sizes where what is read or written passes the
caches, where rows lie more than 2^32 bytes from the first, and where one launch
does not hold a workgroup for every row or piece."""
import pytest
import torch

from test_gpu_embedding import DTYPES, ULP, half_step, make_ids, smallest
from test_gpu_token_logprobs import Reference, check_places

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def reference(grad, ids, vocab, scale):
    """The gradient, its terms' absolute sum and their number, in 64 bits on the GPU."""
    inside = (ids >= 0) & (ids < vocab)
    ids, grad = ids[inside].long(), grad[inside].double() * scale
    total, size = (torch.zeros(vocab, grad.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    return total.index_add_(0, ids, grad), size.index_add_(0, ids, grad.abs()), torch.bincount(ids, minlength=vocab)


def check(got, want, size, count):
    # c terms in 32 bits: c half steps of their absolute sum, one for the scale; the type's own rounding
    tol = (count[:, None] + 2) * ULP * size + half_step(got.dtype) * want.abs() * (1 + 1e-6) + smallest(got.dtype)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert not bool(got[count == 0].any())


# a gradient of over 512 MB from its first element to its last: dense, and with rows far apart
@pytest.mark.parametrize("dtype,out,tokens,vocab,width,pad", [
    ("bf16", "bf16", 3001, 70001, 520, 32481), ("bf16", "fp32", 8195, 131073, 1031, 0), ("fp16", "fp16", 40003, 70001, 100, 33000),
    ("fp32", "fp32", 2500, 70001, 129, 16500), ("fp32", "bf16", 33000, 65537, 4096, 8), ("bf16", "bf16", 9, 300007, 1024, 0)])
def test_gradient_past_the_caches(dtype, out, tokens, vocab, width, pad):
    print(dtype, out, tokens, vocab, width, pad, flush=True)
    g = torch.Generator().manual_seed(tokens)
    ids = make_ids("text", torch.Size((tokens,)), vocab, g)
    ids[tokens // 3:tokens // 2] = vocab - 1  # one of many runs, far from the first row
    ids[tokens // 2:tokens // 2 + 50] = vocab - 3
    grad = torch.randn(tokens, width, generator=g).to(DTYPES[dtype])
    ids, grad = ids.cuda(), grad.cuda()
    buf = torch.full((vocab, width + pad), 7.0, dtype=DTYPES[out], device="cuda")
    assert buf.numel() * buf.element_size() > 1 << 29
    got = lrs.embedding_backward(grad, ids, vocab, 0.8, grad_out=buf[:, pad // 2:pad // 2 + width])
    check(got, *reference(grad, ids, vocab, 0.8))
    assert bool((buf[:, :pad // 2] == 7).all()) and bool((buf[:, pad // 2 + width:] == 7).all())
    again = lrs.embedding_backward(grad, ids, vocab, 0.8, dtype=DTYPES[out])
    assert torch.equal(got, again)  # bit for bit, wherever its rows lie


def test_more_pieces_than_workgroups():
    """The sums' and the cleared rows' tasks take several turns of the grid."""
    g = torch.Generator().manual_seed(1)
    tokens, vocab, width = (1 << 24) + 12345, 1009, 2048
    row = torch.randn(width, generator=g).cuda()
    ids = torch.randint(-1, vocab, (tokens,), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    got = lrs.embedding_backward(row.expand(tokens, width), ids, vocab)
    count = torch.bincount(ids + 1, minlength=vocab + 1)[1:]
    want = count[:, None] * row.double()
    check(got, want, want.abs(), count)
    del got, want
    vocab = 34_000_037
    ids = make_ids("any", torch.Size((5000,)), vocab, g)
    ids[-3:] = torch.tensor([0, vocab - 1, vocab - 1])
    grad = torch.randn(5000, 3, generator=g).cuda()
    buf = torch.full((vocab, 3), 5.0, device="cuda")
    check(lrs.embedding_backward(grad, ids.cuda(), vocab, grad_out=buf), *reference(grad, ids.cuda(), vocab, 1.0))


def test_lookup_of_more_rows_than_workgroups():
    g = torch.Generator("cuda").manual_seed(2)
    for tokens, vocab, width in (((1 << 22) + 77, 1000, 264), ((1 << 26) + 5, 300, 3)):
        weight = torch.randn(vocab, width, generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        assert torch.equal(lrs.embedding_forward(weight, ids), weight[ids])


def compare(x, tokens, some, temperature, calls):
    """Rows `some` of every call's outputs against 64 bits."""
    ref = Reference(x, tokens, temperature)
    for k, out in calls.items():
        lp, h, ranks, top, indices = (t[some].cpu() for t in out)
        ref.values(lp, h)
        check_places(x, tokens, k, ranks, indices)
        want = torch.gather(ref.logp, 1, indices)
        assert bool(((top.double() - want).abs() <= ref.lse_off[:, None] + 2 * ULP * want.abs()).all())
    return ref


# logits of over 256 MB; rows alone and shared
@pytest.mark.parametrize("dtype,rows,n,pad", [("bf16", 1101, 131077, 3), ("fp16", 2050, 70001, 0), ("fp32", 300, 300001, 1),
                                              ("bf16", 520, 262145, 0), ("fp32", 20000, 4099, 0)])
def test_logits_past_the_caches(dtype, rows, n, pad):
    print(dtype, rows, n, pad, flush=True)
    g = torch.Generator("cuda").manual_seed(rows)
    buf = (torch.randn(rows, n + pad, generator=g, device="cuda") * 2.5).to(DTYPES[dtype])
    logits = buf[:, pad // 2:pad // 2 + n]
    assert rows * n * logits.element_size() > 1 << 28
    tokens = torch.randint(-1, n, (rows,), generator=g, device="cuda")
    up, down = (torch.randn(rows, generator=g, device="cuda") for _ in range(2))
    some = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1] + torch.randint(0, rows, (12,), generator=torch.Generator().manual_seed(n)).tolist())
    x, t = logits[some.cuda()].cpu(), tokens[some.cuda()].cpu()
    some = some.cuda()
    ref = compare(x, t, some, 0.9, {k: lrs.token_logprobs_topk(logits, tokens, k, 0.9) for k in (0, 7, 200)})
    logprobs, entropy, stats = lrs.token_logprobs_forward(logits, tokens, 0.9)
    ref.values(logprobs[some].cpu(), entropy[some].cpu())
    grad = lrs.token_logprobs_backward(logits, tokens, stats, up, down, 0.9)
    ref.gradient(grad[some].cpu(), up[some].cpu(), down[some].cpu())
    step = lrs.token_logprobs_step(logits, tokens, up, down, 0.9)
    ref.values(step[0][some].cpu(), step[1][some].cpu())
    ref.gradient(step[2][some].cpu(), up[some].cpu(), down[some].cpu())


@pytest.mark.parametrize("n,ks", [(9, (0, 3)), (1034, (2,))])
def test_more_rows_than_workgroups(n, ks):
    g = torch.Generator("cuda").manual_seed(n)
    rows = (1 << 20) + 1237
    logits = (torch.randn(rows, n, generator=g, device="cuda") * 2.5).to(torch.float16)
    tokens = torch.randint(-1, n, (rows,), generator=g, device="cuda")
    up, down = (torch.randn(rows, generator=g, device="cuda") for _ in range(2))
    some = torch.cat([torch.tensor([0, 1, rows - 1]), torch.arange((1 << 20) - 20, (1 << 20) + 20),
                      torch.randint(0, rows, (200,), generator=torch.Generator().manual_seed(n))]).cuda()
    x, t = logits[some].cpu(), tokens[some].cpu()
    ref = compare(x, t, some, 1.0, {k: lrs.token_logprobs_topk(logits, tokens, k) for k in ks})
    logprobs, entropy, stats = lrs.token_logprobs_forward(logits, tokens)
    ref.values(logprobs[some].cpu(), entropy[some].cpu())
    ref.gradient(lrs.token_logprobs_backward(logits, tokens, stats, up, down)[some].cpu(), up[some].cpu(), down[some].cpu())
    step = lrs.token_logprobs_step(logits, tokens, up, down)
    ref.values(step[0][some].cpu(), step[1][some].cpu())
    ref.gradient(step[2][some].cpu(), up[some].cpu(), down[some].cpu())
    # the last rows by themselves: within both calls' roundings
    last = logits[-500:].contiguous()
    alone = lrs.token_logprobs_forward(last, tokens[-500:])
    assert bool(((alone[0] - logprobs[-500:]).abs() <= 100 * ULP * (1 + logprobs[-500:].abs())).all())
