"""Log probabilities of given tokens, entropies, ranks, alternatives and the
gradient against the formulas in 64 bits on the CPU, with tolerances counted
from the roundings; the gradient also against differences."""
import math
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = 2.0 ** -24  # half a step of 32-bit numbers
INF = math.inf


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def in_32_bits(v):
    """-inf where the nearest 32-bit number is (a lowest value over a small temperature lies beyond the lowest)."""
    return torch.where(torch.isinf(v.float()), v.float().double(), v)


class Reference:
    """Everything in 64 bits, and how far 32-bit parts may be off."""

    def __init__(self, x, tokens, temperature=1.0, mask=None):
        self.x, n = x, x.shape[1]
        z = x.double() / temperature
        rows = x.shape[0]
        m = z.max(dim=1, keepdim=True)[0] if n else z.new_full((rows, 1), -INF)
        self.empty = (m == -INF)[:, 0]
        self.z = torch.where(z == -INF, -INF, z - torch.where(m == -INF, 0.0, m))
        total = torch.exp(self.z).sum(1)
        self.lse = torch.log(total)
        self.logp = self.z - self.lse[:, None]
        self.p = torch.where(self.empty[:, None], 0.0, torch.exp(self.logp))
        self.surprise = torch.where(self.p > 0, -self.logp, 0.0)
        self.entropy = (self.p * self.surprise).sum(1)
        self.given = (tokens >= 0) & (tokens < n)
        self.at = torch.where(self.given, tokens.long(), 0)
        self.on = torch.ones(rows, dtype=torch.bool) if mask is None else mask.bool()
        self.temperature = temperature
        picked = torch.gather(self.logp, 1, self.at[:, None])[:, 0] if n else torch.zeros(rows, dtype=torch.float64)
        picked = in_32_bits(torch.where(self.empty, -INF, picked))
        self.logprobs = torch.where(self.given & self.on, picked, 0.0)
        # An exponent is off by at most 3 half steps (its difference, its factor, its product), a power by 2 more and
        # by the exponent's error; 32 terms are summed in 32 bits; a sum that is moved to a larger logit takes one more
        # such power, at most as often as the largest logit of a thread grows.
        away = torch.where(self.p > 0, -self.z, 0.0)
        s1, s2 = (self.p * away).sum(1), (self.p * away * away).sum(1)
        self.lse_off = ULP * (4 * s1 + 80)
        self.mean_off = self.lse_off + ULP * (4 * s2 + 60 * s1)
        self.logprob_off = torch.where(torch.isinf(self.logprobs), 0.0, self.lse_off + 2 * ULP * self.logprobs.abs())
        self.entropy_off = self.mean_off + self.lse_off + ULP * self.entropy

    def values(self, logprobs, entropy):
        keep = self.on
        assert logprobs.dtype == entropy.dtype == torch.float32
        want = torch.where(self.on, self.entropy, 0.0)
        fine = torch.where(torch.isinf(self.logprobs), logprobs.double() == self.logprobs,
                           (logprobs.double() - self.logprobs).abs() <= self.logprob_off)
        assert bool(fine[keep].all()), (logprobs.double() - self.logprobs).abs().max()
        assert bool(((entropy.double() - want).abs() <= self.entropy_off)[keep].all()), (entropy.double() - want).abs().max()
        assert not bool(logprobs[~keep].any()) and not bool(entropy[~keep].any())

    def gradient(self, got, up, down):
        up = torch.zeros(got.shape[0]) if up is None else up
        down = torch.zeros(got.shape[0]) if down is None else down
        live = self.on & ~self.empty
        up = torch.where(self.given & live, up, 0.0).double()[:, None]
        down = torch.where(live, down, 0.0).double()[:, None]
        away = self.entropy[:, None] - self.surprise
        inner = up + down * torch.where(self.p > 0, away, 0.0)
        want = -self.p * inner
        hot = torch.zeros_like(want)
        if got.shape[1]:
            hot.scatter_(1, self.at[:, None], up)
        want = (want + hot) / self.temperature
        far = torch.where(self.p > 0, -self.z, 0.0)
        size = self.p * (up.abs() + down.abs() * torch.where(self.p > 0, away.abs(), 0.0))
        off = size * (ULP * (3 * far + 12) + self.lse_off[:, None]) + self.p * down.abs() * (ULP * (4 * far + 4 * self.surprise + 4) + self.mean_off[:, None])
        off = (off + 3 * ULP * hot.abs()) / self.temperature
        eps, tiny = torch.finfo(got.dtype).eps, torch.finfo(got.dtype).tiny
        # a power below 2^-126 may be 0
        tol = off + eps / 2 * want.abs() * (1 + 1e-6) + tiny * eps / 2 + 2.0 ** -125 * (up.abs() + 200 * down.abs()) / self.temperature
        bad = (got.double() - want).abs() > tol
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got.double() - want).abs() - tol).max())}"


def image(x):
    """The unsigned integers whose order is the row sorts' order."""
    bits = x.contiguous().view(torch.int16 if x.dtype.itemsize == 2 else torch.int32).numpy().astype(np.int64)
    width = 8 * x.dtype.itemsize
    bits &= (1 << width) - 1
    return np.where(bits >> (width - 1), bits ^ ((1 << width) - 1), bits | (1 << (width - 1)))


def check_places(x, tokens, k, ranks, indices):
    order = np.argsort(-image(x), axis=1, kind="stable")
    assert np.array_equal(indices.numpy(), order[:, :k])
    place = np.argsort(order, axis=1, kind="stable")
    given = ((tokens >= 0) & (tokens < x.shape[1])).numpy()
    want = np.full(x.shape[0], -1)
    if x.shape[1]:
        want[given] = place[np.arange(x.shape[0])[given], tokens.numpy()[given]]
    assert ranks.dtype == torch.int32 and np.array_equal(ranks.numpy(), want)


def make(kind, rows, n, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * 2.5
    if kind == "masked":  # most are ruled out, in the last rows all
        x[torch.rand(rows, n, generator=g) < 0.9] = -INF
        x[rows // 2:, : n * 3 // 4] = -INF
        x[-1:] = -INF
    elif kind == "lowest":  # ruled out by the type's lowest value
        x = x.to(dtype).float()
        x[torch.rand(rows, n, generator=g) < 0.9] = torch.finfo(dtype).min
        x[-1:] = torch.finfo(dtype).min
    elif kind == "sure":  # nearly all mass on one
        x[:, n // 2] = 40.0
    elif kind == "levels":
        x = x.round()
    elif kind == "equal":
        x[:] = torch.randn(rows, 1, generator=g)
    elif kind == "rising":
        x = x.sort(dim=1)[0] * 8
    elif kind == "large":
        x = x * 1000 + 20000
    elif kind == "zeros":
        x = torch.where(torch.rand(rows, n, generator=g) < 0.5, 0.0, -0.0)
    x = x.to(dtype)
    tokens = torch.randint(0, max(1, n), (rows,), generator=g)
    for r in range(0, rows, 3):  # likely ones
        if n:
            tokens[r] = int(x[r].float().argmax())
    tokens[1::5] = -1
    tokens[2::7] = n
    buf = torch.zeros(rows, n + pad, dtype=dtype, device="cuda")
    buf[:, pad // 2:pad // 2 + n] = x.cuda()
    return x, tokens, buf[:, pad // 2:pad // 2 + n]


KINDS = ["any", "masked", "lowest", "sure", "levels", "equal", "rising", "large", "zeros"]
# rows, n, pad, temperature
SHAPES = [(5, 1, 0, 1.0), (9, 7, 1, 0.7), (6, 64, 0, 2.0), (7, 1000, 3, 1.0), (300, 515, 0, 1.3), (4, 8192, 0, 1.0),
          (3, 16411, 5, 0.5), (2, 50021, 0, 1.0), (1, 131072, 0, 1.0), (2, 140001, 7, 1.5), (1, 300000, 0, 1.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_values_ranks_and_gradient(dtype, kind, shape):
    rows, n, pad, temperature = shape
    log(f"{dtype} {kind} {shape}")
    x, tokens, logits = make(kind, rows, n, DTYPES[dtype], rows + n, pad)
    ref = Reference(x, tokens, temperature)
    logprobs, entropy, stats = lrs.token_logprobs_forward(logits, tokens.cuda(), temperature)
    ref.values(logprobs.cpu(), entropy.cpu())
    for k in sorted({0, min(n, 1), min(n, 5), min(n, 40), min(n, 700)}):
        lp, h, ranks, top, indices = (t.cpu() for t in lrs.token_logprobs_topk(logits, tokens.cuda().int(), k, temperature))
        ref.values(lp, h)
        check_places(x, tokens, k, ranks, indices)
        want = in_32_bits(torch.where(ref.empty[:, None], -INF, torch.gather(ref.logp, 1, indices)))
        off = (top.double() - want).abs()
        assert bool(torch.where(torch.isinf(want), top.double() == want, off <= ref.lse_off[:, None] + 2 * ULP * want.abs()).all())
    g = torch.Generator().manual_seed(n)
    scale = 1000.0 if dtype == "fp16" else 1.0
    up, down = torch.randn(rows, generator=g) * scale, torch.randn(rows, generator=g) * scale
    up[4::9] = down[4::9] = 0
    for a, b in ((up, down), (up, None), (None, down)):
        ours = [None if t is None else t.cuda() for t in (a, b)]
        grad = lrs.token_logprobs_backward(logits, tokens.cuda(), stats, *ours, temperature).cpu()
        ref.gradient(grad, a, b)
        step = lrs.token_logprobs_step(logits, tokens.cuda(), *ours, temperature)
        ref.values(step[0].cpu(), step[1].cpu())
        ref.gradient(step[2].cpu(), a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows(dtype):
    for rows, n in ((2500, 300), (700, 4099), (520, 33000)):
        x, tokens, logits = make("levels", rows, n, DTYPES[dtype], n)
        mask = torch.rand(rows, generator=torch.Generator().manual_seed(n)) < 0.7
        ref = Reference(x, tokens, 1.0, mask)
        up, down = torch.randn(rows), torch.randn(rows)
        values = lrs.token_logprobs_forward(logits, tokens.cuda(), row_mask=mask.cuda())
        ref.values(values[0].cpu(), values[1].cpu())
        step = lrs.token_logprobs_step(logits, tokens.cuda(), up.cuda(), down.cuda(), row_mask=mask.to(torch.uint8).cuda())
        ref.values(step[0].cpu(), step[1].cpu())
        ref.gradient(step[2].cpu(), up, down)
        again = lrs.token_logprobs_step(logits, tokens.cuda(), up.cuda(), down.cuda(), row_mask=mask.cuda())
        assert all(torch.equal(p, q) for p, q in zip(step, again))  # bit for bit
        for k in (8, 200):
            out = [t.cpu() for t in lrs.token_logprobs_topk(logits, tokens.cuda(), k)]
            Reference(x, tokens).values(out[0], out[1])
            check_places(x, tokens, k, out[2], out[4])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["any", "lowest", "levels", "equal", "zeros"])
@pytest.mark.parametrize("shape", [(3, 32003, 3), (130, 60001, 0), (256, 9007, 1), (257, 9007, 0)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_alternatives_of_rows_alone(dtype, kind, shape):
    """Rows that one workgroup holds: its most alternatives, and more than one batch of loads a thread."""
    rows, n, pad = shape
    log(f"{dtype} {kind} {shape}")
    x, tokens, logits = make(kind, rows, n, DTYPES[dtype], rows + n, pad)
    ref = Reference(x, tokens, 0.8)
    for k in (3, 300, 512, 513):
        lp, h, ranks, top, indices = (t.cpu() for t in lrs.token_logprobs_topk(logits, tokens.cuda(), k, 0.8))
        ref.values(lp, h)
        check_places(x, tokens, k, ranks, indices)
        want = in_32_bits(torch.where(ref.empty[:, None], -INF, torch.gather(ref.logp, 1, indices)))
        off = (top.double() - want).abs()
        assert bool(torch.where(torch.isinf(want), top.double() == want, off <= ref.lse_off[:, None] + 2 * ULP * want.abs()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["any", "masked", "levels", "zeros"])
def test_alternatives_of_many_short_rows(dtype, kind):
    """A wave a row, several batches of loads."""
    for rows, n, pad in ((2050, 2995, 1), (2048, 1027, 0)):
        x, tokens, logits = make(kind, rows, n, DTYPES[dtype], rows + n, pad)
        if kind == "any":
            x[7, 900] = x[9, n - 1] = float("nan")
            x[8, 5:1000] = INF
            logits.copy_(x)
        ref = Reference(x, tokens)
        sound = torch.ones(rows, dtype=torch.bool)
        sound[7:10] = kind != "any"
        ref.on &= sound  # the others have no values to compare
        for k in (1, 16, 17):
            lp, h, ranks, top, indices = (t.cpu() for t in lrs.token_logprobs_topk(logits, tokens.cuda(), k))
            for t in (lp, h):
                t[~sound] = 0
            ref.values(lp, h)
            check_places(x, tokens, k, ranks, indices)
            want = in_32_bits(torch.where(ref.empty[:, None], -INF, torch.gather(ref.logp, 1, indices)))[sound]
            off = (top[sound].double() - want).abs()
            allowed = ref.lse_off[sound][:, None] + 2 * ULP * want.abs()
            assert bool(torch.where(torch.isinf(want), top[sound].double() == want, off <= allowed).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows_hold_anything(dtype):
    x, tokens, logits = make("any", 6, 2003, DTYPES[dtype], 3)
    for r, v in ((0, float("nan")), (1, INF), (2, -INF)):
        logits[r] = v
    mask = torch.tensor([0, 0, 0, 1, 1, 0], dtype=torch.uint8, device="cuda")
    up = torch.ones(6, device="cuda")
    logprobs, entropy, grad = lrs.token_logprobs_step(logits, tokens.cuda(), up, up, row_mask=mask)
    off = mask == 0
    assert not bool(logprobs[off].any()) and not bool(entropy[off].any()) and not bool(grad[off].any())
    assert bool(torch.isfinite(grad).all())
    _, _, stats = lrs.token_logprobs_forward(logits, tokens.cuda(), row_mask=mask)
    assert not bool(lrs.token_logprobs_backward(logits, tokens.cuda(), stats, up, up, row_mask=mask)[off].any())
    # no derivative: no gradient, whatever the logits are
    zero = torch.zeros(6, device="cuda")
    assert not bool(lrs.token_logprobs_step(logits, tokens.cuda(), zero, zero)[2].any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [5, 700, 9001, 140001])
def test_nan_and_inf(dtype, n):
    x, tokens, logits = make("any", 7, n, DTYPES[dtype], n)
    tokens[:] = torch.arange(7) % n
    for r, (at, v) in enumerate(((0, float("nan")), (n - 1, float("nan")), (n // 2, INF), (1, INF), (n - 1, -float("nan")))):
        x[r, at] = v
    logits.copy_(x)
    up = torch.ones(7, device="cuda")
    logprobs, entropy, grad = (t.cpu() for t in lrs.token_logprobs_step(logits, tokens.cuda(), up, up))
    bad = torch.arange(7) < 5
    assert bool(torch.isnan(logprobs[bad]).all()) and bool(torch.isnan(entropy[bad]).all()) and bool(torch.isnan(grad[bad]).all())
    assert bool(torch.isfinite(logprobs[~bad]).all()) and bool(torch.isfinite(grad[~bad]).all())
    out = [t.cpu() for t in lrs.token_logprobs_topk(logits, tokens.cuda(), 3)]
    assert bool(torch.isnan(out[0][bad]).all()) and bool(torch.isnan(out[1][bad]).all()) and bool(torch.isnan(out[3][bad]).all())
    check_places(x, tokens, 3, out[2], out[4])


def test_autograd_and_differences():
    g = torch.Generator().manual_seed(11)
    x = torch.randn(6, 50, generator=g) * 2
    tokens = torch.tensor([3, -1, 49, 0, 7, 7])
    mask = torch.tensor([1, 1, 1, 0, 1, 1], dtype=torch.bool)
    for dtype in DTYPES.values():
        logits = x.to(dtype).cuda().requires_grad_(True)
        logprobs, entropy = lrs.token_logprobs(logits, tokens.cuda(), 1.5, mask.cuda())
        up, down = torch.randn(6, generator=g), torch.randn(6, generator=g)
        ref = Reference(x.to(dtype), tokens, 1.5, mask)
        for outs, ups, a, b in (((logprobs, entropy), (up, down), up, down), ((logprobs,), (up,), up, None), ((entropy,), (down,), None, down)):
            grad, = torch.autograd.grad(outs, logits, [u.cuda() for u in ups], retain_graph=True)
            ref.gradient(grad.cpu(), a, b)
        (logprobs.sum() + entropy.sum()).backward()  # upstream gradients expanded from one number
        ref.gradient(logits.grad.cpu(), torch.ones(6), torch.ones(6))
        with pytest.raises(RuntimeError):
            first, = torch.autograd.grad(lrs.token_logprobs(logits, tokens.cuda())[0].pow(2).sum(), logits, create_graph=True)
            torch.autograd.grad(first.sum(), logits)


def test_gradient_against_differences():
    """The step's gradient along a direction against a central difference of the 64-bit function."""
    g = torch.Generator().manual_seed(13)
    x = torch.randn(6, 50, generator=g) * 2
    tokens = torch.tensor([3, -1, 49, 0, 7, 7])
    up, down, step = torch.randn(6, generator=g), torch.randn(6, generator=g), torch.randn(6, 50, generator=g).double()
    grad = lrs.token_logprobs_step(x.cuda(), tokens.cuda(), up.cuda(), down.cuda(), 0.8)[2].cpu().double()

    def value(z):
        ref = Reference(z, tokens, 0.8)
        return float((ref.logprobs * up.double() + ref.entropy * down.double()).sum())
    h = 2.0 ** -14
    change = (value(x.double() + h * step) - value(x.double() - h * step)) / (2 * h)
    # the difference leaves out terms of h^2 and rounds at 2^-53 / h; the gradient's elements are off by some 100 half
    # steps of |a| + |b| (|log p| + H), logits here lying within 20 of each other
    size = float(((up.abs() + 40 * down.abs()).double()[:, None] * step.abs()).max(dim=1)[0].sum()) / 0.8
    assert abs(change - float((grad * step).sum())) <= (100 * ULP + 100 * h * h) * size


def test_strides_streams_and_graphs():
    g = torch.Generator().manual_seed(12)
    x = torch.randn(40, 9000, generator=g).cuda()
    tokens = torch.randint(0, 9000, (40, 3), generator=g).cuda()
    want = lrs.token_logprobs_topk(x, tokens[:, 1].contiguous(), 6)
    assert all(torch.equal(p, q) for p, q in zip(lrs.token_logprobs_topk(x, tokens[:, 1], 6), want))
    assert all(torch.equal(p, q) for p, q in zip(lrs.token_logprobs_topk(x[:1].expand(40, 9000), tokens[:1, 1].expand(40), 6),
                                                 [w[:1].expand(40, *w.shape[1:]) for w in want]))
    up = torch.randn(40, generator=g).cuda()
    buf = torch.full((40, 9010), 4.0, device="cuda")
    step = lrs.token_logprobs_step(x, tokens[:, 1], up, up, grad_out=buf[:, 5:9005])
    assert bool((buf[:, :5] == 4).all()) and bool((buf[:, 9005:] == 4).all())
    assert torch.equal(step[2], lrs.token_logprobs_step(x, tokens[:, 1], up, up)[2])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = lrs.token_logprobs_topk(x, tokens[:, 1], 6)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    fixed = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        top = lrs.token_logprobs_topk(fixed, tokens[:, 1], 6)
        step = lrs.token_logprobs_step(fixed, tokens[:, 1], up, up)
        values = lrs.token_logprobs_forward(fixed, tokens[:, 1])
        grad = lrs.token_logprobs_backward(fixed, tokens[:, 1], values[2], up, None)
    for turn in range(3):
        now = torch.randn(40, 9000, generator=g).cuda()
        fixed.copy_(now)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(top, lrs.token_logprobs_topk(now, tokens[:, 1], 6)))
        assert all(torch.equal(p, q) for p, q in zip(step, lrs.token_logprobs_step(now, tokens[:, 1], up, up)))
        eager = lrs.token_logprobs_forward(now, tokens[:, 1])
        assert all(torch.equal(p, q) for p, q in zip(values, eager))
        assert torch.equal(grad, lrs.token_logprobs_backward(now, tokens[:, 1], eager[2], up, None))


def test_nothing_to_do():
    logits, tokens = torch.randn(3, 8, device="cuda"), torch.tensor([1, 2, 3], device="cuda")
    up = torch.ones(3, device="cuda")
    for part in (0, 3):
        out = lrs.token_logprobs_topk(logits[:part, :0] if part else logits[:0], tokens[:part], 0)
        assert [t.shape[0] for t in out] == [part] * 5
    assert lrs.token_logprobs_step(logits[:0], tokens[:0], up[:0])[2].shape == (0, 8)
    logprobs, entropy, grad = lrs.token_logprobs_step(logits[:, :0], tokens, up)
    assert not bool(logprobs.any()) and not bool(entropy.any()) and grad.shape == (3, 0)


def test_rows_far_apart():
    """Rows and their gradient's more than 2^32 bytes from the first."""
    n, rows, stride = 1000, 40000, 60000
    buf = torch.zeros(rows * stride, dtype=torch.bfloat16, device="cuda")
    logits = buf.as_strided((rows, n), (stride, 1))
    logits[-1, 500] = 10.0
    tokens = torch.full((rows,), 500, device="cuda")
    up = torch.ones(rows, device="cuda")
    logprobs, _, _ = lrs.token_logprobs_step(logits, tokens, up, grad_out=torch.empty_like(logits))
    assert abs(float(logprobs[-1]) + math.log1p(999 * math.exp(-10))) < 1e-6 and abs(float(logprobs[0]) + math.log(1000)) < 1e-6
    far = torch.zeros(rows * stride, dtype=torch.bfloat16, device="cuda").as_strided((rows, n), (stride, 1))
    _, _, got = lrs.token_logprobs_step(logits, tokens, up, grad_out=far)
    assert got.data_ptr() == far.data_ptr() and abs(float(far[-1, 500]) - (1 - 1 / (1 + 999 * math.exp(-10)))) < 2.0 ** -8
    assert abs(float(far[-2, 500]) - 0.999) < 2.0 ** -8
