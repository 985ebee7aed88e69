"""Distillation from a teacher's top logits against the formulas in 64 bits on
the CPU, values and gradients, with tolerances counted from the roundings; the
gradient also against differences of the 64-bit loss."""
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


def lse_rows(z):
    m = z.max(dim=1, keepdim=True)[0]
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True)))[:, 0]


def reference(s, t, i, temperature, tlse, w):
    """Row losses and d loss / d s of the formulas in 64 bits, and each gradient
    element's sum of absolute terms (what a relative error of its parts scales)."""
    s, t, w = s.double(), t.double(), w.double()
    rows, n = s.shape
    # the library takes 1 / T in 32 bits
    inv_t = float(np.float32(1.0) / np.float32(temperature))
    z = s * inv_t
    ok = (i >= 0) & (i < n) & (t > -INF)
    at = torch.where(ok, i.long(), torch.full_like(i.long(), n))
    member = torch.zeros(rows, n + 1, dtype=torch.bool).scatter_(1, at, True)[:, :n]
    tz = torch.where(ok, t * inv_t, torch.full_like(t, -INF))
    if tlse is None:
        q = torch.where(ok, torch.exp(tz - lse_rows(tz)[:, None]), torch.zeros_like(t)) if t.shape[1] else t
    else:
        q = torch.exp(tz - tlse.double()[:, None])
    lse = lse_rows(z)
    lse0 = lse_rows(torch.where(member, torch.full_like(z, -INF), z)) if n else lse
    q0 = torch.zeros(rows, dtype=torch.float64)
    if tlse is not None:
        q0 = (1 - q.sum(1)).clamp_min(0)
        q0[member.all(1)] = 0
        q0[(lse0 == -INF) & (q0 <= 2.0 ** -20)] = 0
    target = torch.zeros(rows, n + 1, dtype=torch.float64).scatter_add_(1, at, q)[:, :n]
    p = torch.where(torch.isinf(z), torch.zeros_like(z), torch.exp(z - lse[:, None]))
    zt = torch.gather(torch.cat([z, torch.full((rows, 1), -INF, dtype=torch.float64)], 1), 1, at)
    part = torch.where(q > 0, q * (torch.log(q) - (zt - lse[:, None])), torch.zeros_like(q))
    part = torch.where((q > 0) & (zt == -INF), torch.full_like(q, INF), part)
    loss = part.sum(1)
    extra = torch.where(q0 > 0, q0 * (torch.log(q0) - (lse0 - lse)), torch.zeros_like(q0))
    loss = loss + torch.where((q0 > 0) & (lse0 == -INF), torch.full_like(q0, INF), extra)
    mass = q.sum(1) + q0
    rest = torch.where((q0[:, None] > 0) & ~torch.isinf(z), q0[:, None] * torch.exp(z - lse0[:, None]), torch.zeros_like(z))
    off = mass[:, None] * p - torch.where(member, target, rest)
    terms = mass[:, None] * p + torch.where(member, target, rest)
    scale = (w * inv_t)[:, None]
    dead = w == 0
    loss = torch.where(dead, torch.zeros_like(loss), loss)
    grad = torch.where(dead[:, None], torch.zeros_like(off), off * scale)
    return loss, grad, torch.where(dead[:, None], torch.zeros_like(terms), terms * scale.abs()), z


def make(rows, n, k, dtype, seed, tail=False, temperature=1.0, teacher=None, ints=torch.int64, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(rows, n, generator=g) * 2.5
    s = 0.6 * full + 1.5 * torch.randn(rows, n, generator=g)
    if kind == "masked":  # padding columns of the vocabulary, in teacher and student
        cut = n - n // 5
        full[:, cut:] = -INF
        s[:, cut:] = -INF
    kk = min(k, n)
    t, i = torch.topk(full, kk, dim=1)
    if k > kk:  # more slots than columns
        t = torch.cat([t, torch.zeros(rows, k - kk)], 1)
        i = torch.cat([i, torch.full((rows, k - kk), -1)], 1)
    tlse = torch.logsumexp(full.double() / temperature, dim=1).float() if tail else None
    return s.to(DTYPES[dtype]), t.to(DTYPES[teacher or dtype]), i.to(ints), tlse


def half_step(dtype, g):
    """Half a step of the type at g: its rounding, with the floor of its smallest numbers."""
    floor = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -126, "fp32": 2.0 ** -126}[dtype]
    return g.abs() * (torch.finfo(DTYPES[dtype]).eps / 2) + floor


def check(s, t, i, temperature=1.0, tlse=None, w=None, pad=0):
    rows, n = s.shape
    dtype = {v: k for k, v in DTYPES.items()}[s.dtype]
    wr = torch.full((rows,), 1.0 / max(rows, 1)) if w is None else w
    loss, grad, terms, z = reference(s, t, i, temperature, tlse, wr)
    buf = torch.full((rows, n + pad), float("nan"), dtype=s.dtype)
    buf[:, :n] = s
    gs = buf.cuda()[:, :n]
    gt, gi = t.cuda(), i.cuda()
    gl = None if tlse is None else tlse.cuda()
    gw = None if w is None else w.cuda()
    out = lrs.topk_distill_forward(gs, gt, gi, temperature, gl, gw)
    up = torch.tensor(1.0, device="cuda")
    back = lrs.topk_distill_backward(gs, gt, gi, out[2], temperature, gl, gw, up)
    held = torch.full((rows, n + pad), 7.0, dtype=s.dtype, device="cuda")
    total, row_loss, step = lrs.topk_distill_step(gs, gt, gi, temperature, gl, gw, grad_out=held[:, :n])
    torch.cuda.synchronize()
    assert bool((held[:, n:] == 7.0).all()), "wrote past a row's end"
    # a thread adds at most n / 256 exponentials in 32 bits; one exponential and
    # the products around it round some tens of times
    tol = (n / 256 + 64) * ULP
    for got in (out[1].cpu().double(), row_loss.cpu().double()):
        assert torch.equal(torch.isinf(got), torch.isinf(loss)) and not torch.isnan(got).any()
        fine = torch.isfinite(loss)
        off = (got - loss)[fine].abs()
        bound = tol + 2 * ULP * loss[fine].abs()
        assert bool((off <= bound).all()), f"row loss off by {off.max()}"
    fine = torch.isfinite(loss)
    if bool(fine[wr != 0].all()):
        want = (wr.double() * torch.where(wr == 0, torch.zeros_like(loss), loss)).sum()
        lim = (wr.double().abs() * (tol + 2 * ULP * loss.abs().nan_to_num(posinf=0))).sum() + 2 * ULP * want.abs()
        for got in (out[0], total):
            assert abs(float(got) - float(want)) <= float(lim)
    # an exponential's argument is up to the row's spread, and rounds twice
    zf = torch.where(torch.isinf(z), torch.zeros_like(z), z)
    spread = (zf.max(1, keepdim=True)[0] - zf).abs() if n else zf
    lim = terms * (tol + 4 * ULP * (spread + 1)) + half_step(dtype, grad)
    for name, got in (("backward", back), ("step", step)):
        got = got.cpu().double()
        off = (got - grad).abs()
        assert not torch.isnan(got).any()
        assert bool((off <= lim).all()), f"{name}: gradient off by {(off - lim).max()} over its bound"


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows,n,k,temperature", [
    (1, 1, 1, 1.0), (3, 2, 1, 2.0), (4, 7, 3, 1.0), (2, 9, 12, 1.0), (5, 64, 64, 0.7), (37, 257, 16, 1.0),
    (3, 2048, 300, 1.0), (2, 8193, 1024, 4.0), (70, 5003, 33, 2.0), (1, 131_072, 64, 1.0), (3, 70_001, 17, 1.0),
    (300, 33_000, 8, 1.0), (600, 4096, 20, 1.0)])
def test_sizes(dtype, tail, rows, n, k, temperature):
    log(f"distill {dtype} tail={tail} {rows}x{n} k={k} T={temperature}")
    s, t, i, tlse = make(rows, n, k, dtype, 1000 + n, tail, temperature)
    check(s, t, i, temperature, tlse)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,n", [(5, 4000), (3, 150_001), (320, 20_003)])
@pytest.mark.parametrize("pad", [1, 5, 8])
def test_strides_and_weights(dtype, rows, n, pad):
    log(f"distill {dtype} {rows}x{n} pad={pad}")
    s, t, i, tlse = make(rows, n, 24, dtype, 2000 + pad, True, 1.0)
    w = torch.rand(rows, generator=torch.Generator().manual_seed(3)) * 3
    w[::3] = 0
    check(s, t, i, 1.0, tlse, w, pad)
    check(s, t, i, 1.0, None, -w, pad)


@pytest.mark.parametrize("teacher", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("ints", [torch.int32, torch.int64])
def test_teacher_types_and_sliced_lists(teacher, ints):
    s, t, i, tlse = make(40, 3001, 50, "bf16", 2100, True, 1.0, teacher, ints)
    check(s, t, i, 1.0, tlse)
    # the first columns of longer lists, as a sliced row sort gives them
    gt, gi = t.cuda(), i.cuda()
    a = lrs.topk_distill_step(s.cuda(), gt[:, :9], gi[:, :9])
    b = lrs.topk_distill_step(s.cuda(), gt[:, :9].contiguous(), gi[:, :9].contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1000, 40_003, 140_000])
def test_empty_slots_and_masked_columns(dtype, n):
    for tail in (False, True):
        s, t, i, tlse = make(12, n, 20, dtype, 2200 + n, tail, 1.0, kind="masked")
        i[0] = -1            # nothing from the teacher
        i[1, 5:] = n         # out of range above
        i[2, ::2] = -7
        t[3, 10:] = -INF     # no mass
        i[4, 1:] = -1
        log(f"distill empty slots {dtype} n={n} tail={tail}")
        check(s, t, i, 1.0, tlse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tail", [False, True])
def test_columns_listed_twice(dtype, tail):
    for n, k in ((500, 12), (70_000, 200)):
        s, t, i, tlse = make(9, n, k, dtype, 2300 + n, tail)
        i[:, k // 2] = i[:, 0]
        i[3] = i[3, 1]
        if tail:  # masses that still add up to less than 1
            tlse = tlse + 3.0
        log(f"distill twice {dtype} n={n} tail={tail}")
        check(s, t, i, 1.0, tlse)


@pytest.mark.parametrize("tail", [False, True])
def test_rows_without_mass(tail):
    # the student gives a teacher's column nothing, or nothing at all: loss +inf, a finite gradient
    s, t, i, tlse = make(6, 3000, 10, "fp32", 2400, tail)
    s[0, i[0, 3]] = -INF
    s[1] = -INF
    keep = torch.zeros(3000, dtype=torch.bool)
    keep[i[2]] = True
    s[2, ~keep] = -INF     # with a tail: all the student has is on the teacher's columns
    check(s, t, i, 1.0, tlse)


@pytest.mark.parametrize("n", [700, 50_000])
def test_whole_vocabulary_listed(n):
    # the teacher lists every column that has mass: no tail is left but rounding
    k = min(n, 1024)
    g = torch.Generator().manual_seed(5)
    full = torch.full((4, n), -INF)
    full[:, :k] = torch.randn(4, k, generator=g)
    s = torch.full((4, n), -INF)
    s[:, :k] = torch.randn(4, k, generator=g)
    t, i = torch.topk(full, k, dim=1)
    check(s, t, i, 1.0, torch.logsumexp(full.double(), 1).float())


def test_weight_zero_hides_a_row_of_nan():
    for n in (300, 40_000, 135_000):
        s, t, i, tlse = make(8, n, 6, "bf16", 2500)
        w = torch.ones(8)
        w[[2, 5]] = 0
        s[2] = float("nan")
        s[5] = INF
        for l in (None, torch.full((8,), 20.0)):
            a = lrs.topk_distill_step(s.cuda(), t.cuda(), i.cuda(), row_weights=w.cuda(),
                                      teacher_lse=None if l is None else l.cuda())
            assert torch.isfinite(a[0]) and torch.isfinite(a[1]).all() and torch.isfinite(a[2].float()).all()
            assert bool((a[2][[2, 5]] == 0).all()) and bool((a[1][[2, 5]] == 0).all())
        # where such a row counts, it shows
        a = lrs.topk_distill_step(s.cuda(), t.cuda(), i.cuda())
        assert torch.isnan(a[1][[2, 5]]).all() and torch.isfinite(a[1][[0, 1, 3, 4, 6, 7]]).all()


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    s, t, i, tlse = make(4, 600, 15, "fp32", 2600, tail, 1.3)
    w = torch.tensor([0.5, 1.0, 0.25, 2.0])
    _, _, grad = lrs.topk_distill_step(s.cuda(), t.cuda(), i.cuda(), 1.3, None if tlse is None else tlse.cuda(), w.cuda())
    g = torch.Generator().manual_seed(9)
    h = 1e-4
    for _ in range(5):
        v = torch.randn(4, 600, generator=g, dtype=torch.float64)

        def loss(x):
            return float((w.double() * reference(x, t, i, 1.3, tlse, w)[0]).sum())
        slope = (loss(s.double() + h * v) - loss(s.double() - h * v)) / (2 * h)
        # third derivatives of a log-sum-exp are below 1 a coordinate; h^2 of them, and rounding
        assert abs(slope - float((grad.cpu().double() * v).sum())) < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd(dtype):
    s, t, i, tlse = make(20, 3000, 11, dtype, 2700, True)
    x = s.cuda().requires_grad_(True)
    gt, gi, gl = t.cuda(), i.cuda(), tlse.cuda()
    loss = lrs.topk_distill_loss(x, gt, gi, teacher_lse=gl)
    first, = torch.autograd.grad(loss, x, retain_graph=True)
    again, = torch.autograd.grad(loss, x, retain_graph=True)
    four, = torch.autograd.grad(4 * loss, x)
    ref = lrs.topk_distill_step(x.detach(), gt, gi, teacher_lse=gl)
    assert torch.equal(first, again) and first.dtype == s.dtype
    assert torch.equal(loss.detach(), ref[0])
    # four times the gradient, each rounded by itself; both ways of computing it round alike within their bound
    eps = torch.finfo(s.dtype).eps
    assert torch.allclose(four.double(), 4 * first.double(), rtol=eps, atol=0)
    assert torch.allclose(first.double(), ref[2].double(), rtol=eps + 200 * ULP, atol=1e-9)
    # a leaf shared by two uses, and a slice of a wider matrix
    wide = torch.zeros(20, 3008, dtype=s.dtype, device="cuda")
    wide[:, :3000] = s.cuda()
    wide.requires_grad_(True)
    (lrs.topk_distill_loss(wide[:, :3000], gt, gi, teacher_lse=gl) + wide[:, 3000:].sum()).backward()
    assert torch.equal(wide.grad[:, :3000], first) and bool((wide.grad[:, 3000:] == 1).all())


def test_same_bits_every_time_and_on_another_stream():
    for rows, n in ((3, 100_000), (400, 9000)):
        s, t, i, tlse = make(rows, n, 30, "bf16", 2800, True)
        args = (s.cuda(), t.cuda(), i.cuda(), 1.0, tlse.cuda())
        first = lrs.topk_distill_step(*args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = lrs.topk_distill_step(*args)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_graph_replay():
    for rows, n in ((4, 50_000), (300, 6000)):
        s, t, i, tlse = make(rows, n, 12, "bf16", 2900, True)
        x, gt, gi, gl = s.cuda(), t.cuda(), i.cuda(), tlse.cuda()
        lrs.topk_distill_step(x, gt, gi, 1.0, gl)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = lrs.topk_distill_step(x, gt, gi, 1.0, gl)
        for seed in range(3):
            x.copy_(make(rows, n, 12, "bf16", 3000 + seed)[0])
            g.replay()
            eager = lrs.topk_distill_step(x, gt, gi, 1.0, gl)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_rows_beyond_32_bit_offsets():
    n, stride = 5000, (1 << 31) + 8
    buf = torch.empty(stride + n, dtype=torch.bfloat16, device="cuda")
    gbuf = torch.empty(stride + n, dtype=torch.bfloat16, device="cuda")
    s, t, i, tlse = make(2, n, 16, "bf16", 3100, True)
    x = buf.as_strided((2, n), (stride, 1))
    g = gbuf.as_strided((2, n), (stride, 1))
    x.copy_(s)
    far = lrs.topk_distill_step(x, t.cuda(), i.cuda(), 1.0, tlse.cuda(), grad_out=g)
    near = lrs.topk_distill_step(s.cuda(), t.cuda(), i.cuda(), 1.0, tlse.cuda())
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    v, c = lrs.segmented_row_topk(x, 20)
    v2, c2 = lrs.segmented_row_topk(s.cuda(), 20)
    assert torch.equal(c, c2) and torch.equal(v, v2)


def test_no_rows():
    e = torch.empty(0, 100, device="cuda")
    loss, row_loss, grad = lrs.topk_distill_step(e, torch.empty(0, 3, device="cuda"),
                                                 torch.empty(0, 3, dtype=torch.int64, device="cuda"))
    assert float(loss) == 0 and row_loss.numel() == 0 and grad.shape == (0, 100)


def check_shifted(s, t, i, temperature, tlse):
    """check for logits so large that 64 bits lose log n beside them: the formulas of the rows less their largest."""
    rows, n = s.shape
    dtype = {v: k for k, v in DTYPES.items()}[s.dtype]
    wr = torch.full((rows,), 1.0 / rows)
    top = s.double().max(1, keepdim=True)[0]
    loss, grad, terms, z = reference(s.double() - top, t, i, temperature, tlse, wr)
    args = (s.cuda(), t.cuda(), i.cuda())
    gl = None if tlse is None else tlse.cuda()
    _, row_loss, stats = lrs.topk_distill_forward(*args, temperature, gl)
    back = lrs.topk_distill_backward(*args, stats, temperature, gl)
    _, row_loss2, step = lrs.topk_distill_step(*args, temperature, gl)
    tol = (n / 256 + 64) * ULP
    fine = torch.isfinite(loss)
    for got in (row_loss.cpu().double(), row_loss2.cpu().double()):
        assert torch.equal(torch.isinf(got), ~fine) and not torch.isnan(got).any()
        assert bool(((got - loss)[fine].abs() <= tol + 2 * ULP * loss[fine].abs()).all())
    # what is far below the row's largest has no share at all
    spread = torch.where(z < -1000, torch.zeros_like(z), z).abs()
    lim = terms * (tol + 4 * ULP * (spread + 1)) + half_step(dtype, grad)
    for name, got in (("backward", back), ("step", step)):
        off = (got.cpu().double() - grad).abs()
        assert bool((off <= lim).all()), f"{name}: gradient off by {(off - lim).max()} over its bound"


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("n,k", [(50, 4), (9001, 30), (70_001, 5)])
def test_lowest_values_as_masks(dtype, tail, temperature, n, k):
    """Masks of the type's lowest value: some columns, all but S, a whole row, all but one column."""
    log(f"lowest {dtype} tail={tail} T={temperature} n={n}")
    s, t, i, tlse = make(6, n, k, dtype, 700, tail, temperature)
    low = torch.finfo(s.dtype).min
    off = [next(j for j in range(n // 2, n) if j not in set(i[r].tolist())) for r in range(6)]
    # a column of S under such a mask is left out where others are not: its loss would pass 32 bits
    s[0, ::3] = low
    s[0, i[0]] = 1.0
    s[1] = low
    s[2] = low
    s[2, i[2]] = 1.5
    s[2, off[2]] = 0.5
    s[3] = low
    s[3, i[3]] = -9.0
    s[3, off[3]] = -2.0
    s[4, :n // 2] = -math.inf
    s[4, n // 2:] = low
    s[4, i[4, 0]] = low
    check_shifted(s, t, i, temperature, tlse)
    s[5] = torch.finfo(s.dtype).max / 2
    s[5, ::2] = torch.finfo(s.dtype).max / 4
    s[5, i[5]] = torch.finfo(s.dtype).max / 2
    check_shifted(s, t, i, temperature, tlse)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k", [(40, 6), (20_003, 30), (140_001, 20)])
def test_odd_teachers(dtype, n, k):
    """Rows whose teacher has no mass on S, or all of it, unused slots anywhere, and weights of either sign."""
    log(f"odd teachers {dtype} n={n} k={k}")
    s, t, i, tlse = make(8, n, k, dtype, 800, True)
    tlse[0] = math.inf
    tlse[1] = torch.logsumexp(t[1].double(), 0).float()
    t[2] = -math.inf
    i[3, ::2] = -1
    i[4, 1] = n
    t[5, 0] = -math.inf
    w = torch.tensor([0.5, -0.25, 1.0, 0.0, 2.0, -1.0, 1e-3, 0.125])
    check(s, t, i, 1.0, tlse, w)
    check(s, t, i, 1.0, None, w)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [
    (300, 5, 2), (300, 1023, 8), (270, 1025, 70), (300, 2048, 64), (257, 2051, 3), (300, 4096, 100), (258, 4099, 9),
    (300, 8192, 20), (260, 8200, 300), (265, 16_385, 33), (300, 33_000, 5)])
def test_many_rows(dtype, rows, n, k):
    """More rows than CUs: the edges between the numbers of threads that take a row."""
    log(f"many rows {dtype} {rows}x{n} k={k}")
    for tail in (False, True):
        s, t, i, tlse = make(rows, n, k, dtype, 900 + n, tail)
        check(s, t, i, 1.0, tlse, None, 1)
