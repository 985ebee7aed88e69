"""Per-expert counts and the load balance loss against the formulas in 64 bits
on the CPU, values and gradients, with tolerances counted from the roundings;
the gradient also against differences of the 64-bit loss."""
import math
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = 2.0 ** -24
INF = math.inf


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def make(tokens, experts, k, dtype, seed, masked=False, ints=torch.int64):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, experts, generator=g) * 1.5 + torch.randn(experts, generator=g)).to(DTYPES[dtype])
    idx = torch.topk(x.float(), min(k, experts), dim=1)[1].to(ints)
    drop = torch.rand(tokens, generator=g) < 0.1
    idx[drop, -1] = -1
    mask = torch.rand(tokens, generator=g) < 0.7 if masked else None
    return x, idx, mask


def counts_of(idx, experts, mask):
    i = idx.long()
    keep = (i >= 0) & (i < experts)
    if mask is not None:
        keep &= mask[:, None]
    return torch.bincount(i[keep], minlength=experts)[:experts]


def reference(x, counts, mask, alpha, beta, score):
    x = x.double()
    tokens, experts = x.shape
    total = int(counts.sum())
    f = counts.double() * experts / total if total else torch.zeros(experts, dtype=torch.float64)
    kept = torch.ones(tokens, dtype=torch.bool) if mask is None else mask
    n = int(kept.sum())
    live = (x > -INF).any(1)
    z = torch.where(live, torch.logsumexp(torch.where(live[:, None], x, torch.zeros_like(x)), 1), torch.zeros(tokens, dtype=torch.float64))
    if score == "softmax":
        p = torch.where(live[:, None], torch.exp(x - z[:, None]), torch.zeros_like(x))
        slope = torch.ones_like(x)
    else:
        s = torch.sigmoid(x)
        p = torch.where(live[:, None], s / s.sum(1, keepdim=True), torch.zeros_like(x))
        slope = torch.sigmoid(-x)
    b = p @ f
    row = torch.where(kept, alpha * b + beta * z * z, torch.zeros_like(b))
    loss = row.sum() / n if n else torch.zeros((), dtype=torch.float64)
    d = alpha * (f - b[:, None]) + 2 * beta * z[:, None]
    terms = abs(alpha) * (f + b[:, None]) + 2 * abs(beta) * z.abs()[:, None]
    on = kept[:, None].double() / max(n, 1)
    return loss, p * slope * d * on, p * slope * terms * on, row, z, kept, n


def check(x, idx, mask, alpha=0.01, beta=0.0, score="softmax", pad=0, given=None):
    tokens, experts = x.shape
    dtype = {v: k for k, v in DTYPES.items()}[x.dtype]
    own = counts_of(idx, experts, mask)
    counts = own if given is None else given
    loss, grad, terms, row, z, kept, n = reference(x, counts, mask, alpha, beta, score)
    buf = torch.full((tokens, experts + pad), float("nan"), dtype=x.dtype)
    buf[:, :experts] = x
    gx = buf.cuda()[:, :experts]
    gi = idx.cuda()
    gm = None if mask is None else mask.cuda()
    gc = None if given is None else given.int().cuda()
    c, rows_counted = lrs.expert_counts(gi, experts, gm)
    assert torch.equal(c.cpu().long(), own) and int(rows_counted) == n
    kw = dict(balance_weight=alpha, z_weight=beta, score=score, row_mask=gm)
    got, c2, kept_dev = lrs.expert_balance_forward(gx, gi, counts=gc, **kw)
    assert torch.equal(c2.cpu().long(), counts) and int(kept_dev) == n
    back = lrs.expert_balance_backward(gx, c2, kept_dev, loss_grad=torch.tensor(1.0, device="cuda"), **kw)
    held = torch.full((tokens, experts + pad), 7.0, dtype=x.dtype, device="cuda")
    total, c3, step = lrs.expert_balance_step(gx, gi, counts=gc, grad_out=held[:, :experts], **kw)
    torch.cuda.synchronize()
    assert bool((held[:, experts:] == 7.0).all()), "wrote past a row's end"
    assert torch.equal(c3, c2)
    # a lane adds at most experts / 4 terms in 32 bits; an exponential and the products around it round some tens of times
    tol = (experts / 4 + 64) * ULP
    lim = float(((row.abs() * 2 + 2 * abs(beta) * z.abs() * (1 + 4 * z.abs())) * tol)[kept].sum()) / max(n, 1) + ULP * abs(float(loss))
    for l in (got, total):
        assert abs(float(l) - float(loss)) <= lim, (float(l), float(loss), lim)
    zf = torch.where(torch.isinf(x), torch.zeros_like(x), x).double()
    spread = (zf.max(1, keepdim=True)[0] - zf).abs() + zf.abs()
    floor = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -126, "fp32": 2.0 ** -126}[dtype]
    lim = terms * (2 * tol + 4 * ULP * (spread + 1)) + grad.abs() * (torch.finfo(x.dtype).eps / 2) + floor
    for name, g in (("backward", back), ("step", step)):
        g = g.cpu().double()
        off = (g - grad).abs()
        assert not torch.isnan(g).any() and bool((off <= lim).all()), f"{name}: gradient off by {(off - lim).max()} over its bound"


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("tokens,experts,k", [
    (1, 1, 1), (5, 2, 1), (3, 7, 3), (64, 8, 2), (100, 63, 4), (33, 64, 6), (1000, 65, 1), (777, 160, 6), (300, 256, 8),
    (50, 511, 16), (20, 1000, 10), (9, 4096, 8), (20_000, 32, 4)])
def test_sizes(dtype, score, masked, tokens, experts, k):
    log(f"balance {dtype} {score} masked={masked} {tokens}x{experts} k={k}")
    x, idx, mask = make(tokens, experts, k, dtype, 100 + experts, masked)
    check(x, idx, mask, 1.0 if dtype == "fp16" else 0.01, 1e-3 if score == "softmax" else 0.0, score)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("tokens,experts", [(50, 40), (70, 129), (31, 256), (9, 700)])
def test_strides_and_int32_ids(dtype, pad, tokens, experts):
    x, idx, mask = make(tokens, experts, 3, dtype, 200 + pad, True, torch.int32)
    check(x, idx, mask, 0.5, 0.01, "softmax", pad)
    wide = torch.full((tokens, 5), 1, dtype=torch.int32)
    wide[:, :3] = idx
    c, n = lrs.expert_counts(wide.cuda()[:, :3], experts, mask.cuda())
    assert torch.equal(c.cpu().long(), counts_of(idx, experts, mask))


def test_counts_of_all_ranks():
    x, idx, mask = make(200, 64, 4, "fp32", 300, True)
    other = torch.randint(0, 5000, (64,), generator=torch.Generator().manual_seed(1))
    check(x, idx, mask, 0.1, 1e-3, "softmax", 0, other)
    check(x, idx, None, 0.1, 1e-3, "softmax", 0, torch.zeros(64, dtype=torch.int64))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [24, 256, 600])
def test_masked_experts_and_empty_rows(score, experts):
    x, idx, _ = make(40, experts, 2, "fp32", 400)
    x[:, ::5] = -INF       # experts on a node that is down
    x[7] = -INF            # a token that may go nowhere
    beta = 1e-2 if score == "softmax" else 0.0
    check(x, idx, None, 0.3, beta, score)
    none = torch.zeros(40, dtype=torch.bool)
    check(x, idx, none, 0.3, beta, score)          # no token counts
    check(x, torch.full_like(idx, -1), None, 0.3, beta, score)  # every slot dropped
    check(x, torch.full_like(idx, experts), None, 0.3, beta, score)
    x[3] = float("nan")    # a padding token's logits do not matter
    keep = torch.ones(40, dtype=torch.bool)
    keep[3] = False
    gx, gi, gk = x.cuda(), idx.cuda(), keep.cuda()
    loss, _, grad = lrs.expert_balance_step(gx, gi, 0.3, beta, score, gk)
    assert torch.isfinite(loss) and torch.isfinite(grad).all() and bool((grad[3] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_logits(score):
    x, idx, mask = make(60, 96, 4, "fp32", 500, True)
    check(x * 40, idx, mask, 0.2, 1e-3 if score == "softmax" else 0.0, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    x, idx, mask = make(30, 40, 3, "fp32", 600, True)
    beta = 0.05 if score == "softmax" else 0.0
    _, _, grad = lrs.expert_balance_step(x.cuda(), idx.cuda(), 0.7, beta, score, mask.cuda())
    counts = counts_of(idx, 40, mask)
    g = torch.Generator().manual_seed(2)
    h = 1e-4
    for _ in range(5):
        v = torch.randn(30, 40, generator=g, dtype=torch.float64)

        def loss(y):
            return float(reference(y, counts, mask, 0.7, beta, score)[0])
        slope = (loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)
        assert abs(slope - float((grad.cpu().double() * v).sum())) < 1e-5


def test_autograd_and_streams():
    x, idx, mask = make(3000, 64, 4, "bf16", 700, True)
    gx, gi, gm = x.cuda().requires_grad_(True), idx.cuda(), mask.cuda()
    loss, counts = lrs.expert_balance_loss(gx, gi, 0.01, 1e-3, "softmax", gm)
    first, = torch.autograd.grad(loss, gx, retain_graph=True)
    two, = torch.autograd.grad(2 * loss, gx)
    ref = lrs.expert_balance_step(gx.detach(), gi, 0.01, 1e-3, "softmax", gm)
    assert torch.equal(loss.detach(), ref[0]) and torch.equal(counts, ref[1]) and torch.equal(first, ref[2])
    assert torch.allclose(two.double(), 2 * first.double(), rtol=torch.finfo(torch.bfloat16).eps, atol=0)
    given = counts * 3
    loss2, c2 = lrs.expert_balance_loss(gx, gi, 0.01, 1e-3, "softmax", gm, given)
    assert torch.equal(c2, given) and torch.allclose(loss2, loss, rtol=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = lrs.expert_balance_step(gx.detach(), gi, 0.01, 1e-3, "softmax", gm)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, again))


def test_graph_replay():
    for tokens in (50, 5000):
        x, idx, mask = make(tokens, 64, 4, "bf16", 800, True)
        gx, gi, gm = x.cuda(), idx.cuda(), mask.cuda()
        lrs.expert_balance_step(gx, gi, 0.01, 1e-3, "softmax", gm)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = lrs.expert_balance_step(gx, gi, 0.01, 1e-3, "softmax", gm)
        for seed in range(3):
            y, j, m = make(tokens, 64, 4, "bf16", 900 + seed, True)
            gx.copy_(y), gi.copy_(j), gm.copy_(m)
            g.replay()
            eager = lrs.expert_balance_step(gx, gi, 0.01, 1e-3, "softmax", gm)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_no_tokens():
    loss, counts, grad = lrs.expert_balance_step(torch.empty(0, 8, device="cuda"),
                                                 torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    assert float(loss) == 0 and counts.tolist() == [0] * 8 and grad.shape == (0, 8)
