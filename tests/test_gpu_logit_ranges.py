"""Row operators on finite logits of any size: masks of values in common use
(-1e4 to -1e20), whole rows at such a value, large logits that differ by little,
and temperatures that put ordinary logits there.  The oracle takes every row in
64 bits relative to its own largest logit."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = 2.0 ** -24  # half a step of 32-bit numbers
INF = float("inf")


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def half_step(dtype, g):
    """Half a step of the type at g, with the floor of its smallest numbers."""
    floor = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -126, "fp32": 2.0 ** -126}[dtype]
    return g.abs() * (torch.finfo(DTYPES[dtype]).eps / 2) + floor


# ------------------------------------------------------------- distillation

def log_softmax(s, temperature):
    """Each row's log softmax of s / temperature, and its largest logit, its log-sum-exp less the largest."""
    top = s.max(1, keepdim=True)[0]
    u = torch.where(s == -INF, s, (s - torch.where(top == -INF, 0.0, top)) / temperature)
    rest = torch.where(top == -INF, 0.0, torch.log(torch.exp(u).sum(1, keepdim=True)))  # a row without mass keeps -inf
    return u - rest, top, rest


def distill_oracle(s, t, i, temperature, tlse):
    """Row losses, the sum of their terms' sizes, the gradient (weight 1), the sum of its terms' sizes, and how far
    (in exponents) each column lies below the largest of the rows that it is weighed in."""
    s, t = s.double(), t.double()
    rows, n = s.shape
    ok = (i >= 0) & (i < n) & (t > -INF)
    at = torch.where(ok, i.long(), n)
    member = torch.zeros(rows, n + 1, dtype=torch.bool).scatter_(1, at, True)[:, :n]
    tz = torch.where(ok, t / temperature, -INF)
    logp, top, rest = log_softmax(s, temperature)
    if tlse is None:
        logq, q0 = torch.log_softmax(tz, 1), torch.zeros(rows, dtype=torch.float64)
    else:
        logq = tz - tlse.double()[:, None]
        q0 = (1 - torch.exp(logq).sum(1)).clamp_min(0)
    q = torch.exp(logq)
    zt = torch.gather(logp, 1, torch.where(ok, at, 0))
    part = torch.where(q > 0, q * (logq - zt), 0.0)
    loss = part.sum(1)
    size = torch.where(q > 0, q * (logq.abs() + zt.abs()), 0.0).sum(1)
    logp_tail, top_tail, rest_tail = log_softmax(torch.where(member, -INF, s), temperature)
    if tlse is not None:
        q0 = torch.where((top_tail[:, 0] == -INF) & (q0 <= 2.0 ** -20), 0.0, q0)
        logp0 = ((top_tail - top) / temperature + rest_tail - rest)[:, 0]
        loss = loss + torch.where(q0 > 0, q0 * (torch.log(q0) - logp0), 0.0)
        size = size + torch.where(q0 > 0, q0 * (torch.log(q0).abs() + logp0.abs()), 0.0)
    mass = q.sum(1) + q0
    target = torch.zeros(rows, n + 1, dtype=torch.float64).scatter_add_(1, at, q)[:, :n]
    tail = q0[:, None] * torch.exp(logp_tail)
    own = mass[:, None] * torch.exp(logp)
    grad = (own - torch.where(member, target, tail)) / temperature
    terms = (own + torch.where(member, target, tail)) / temperature
    # a column so far below that it has no share rounds to none
    below = torch.where(logp > -200, logp.abs(), 0.0)
    below = torch.maximum(below, torch.where(~member & (logp_tail > -200), logp_tail.abs(), 0.0))
    return loss, size, grad, terms, below


def check_distill(s, t, i, temperature=1.0, tlse=None, copies=1):
    dtype = {v: k for k, v in DTYPES.items()}[s.dtype]
    rows = s.shape[0] * copies
    loss, size, grad, terms, below = distill_oracle(s, t, i, temperature, tlse)

    def tiled(x):
        return None if x is None else x.cuda().repeat(copies, *[1] * (x.dim() - 1))
    args = (tiled(s), tiled(t), tiled(i))
    lse = tiled(tlse)
    total, row_loss, stats = lrs.topk_distill_forward(*args, temperature, lse)
    back = lrs.topk_distill_backward(*args, stats, temperature, lse)
    total2, row_loss2, step = lrs.topk_distill_step(*args, temperature, lse)
    torch.cuda.synchronize()
    # a thread adds at most 128 exponentials in 32 bits; one exponential and the products around it round some tens of times
    tol = (128 + 64) * ULP
    # log2(e) / temperature has 32 bits in 16-bit rows, rounded down, and a result is rounded once
    bound = tol + 4 * ULP * size
    for name, got in (("forward", row_loss), ("step", row_loss2)):
        off = (got.cpu().double().view(copies, -1) - loss).abs()
        assert bool((off <= bound).all()), f"{name}: row losses {got[:loss.numel()].tolist()} for {loss.tolist()}"
    for name, got in (("forward", total), ("step", total2)):
        assert abs(float(got) - float(loss.mean())) <= float(bound.mean()) + ULP * abs(float(loss.mean())), name
    # an exponent that far below rounds by its own half step, and by the factor's
    want = grad / rows
    lim = (terms / rows) * (tol + 4 * ULP * (below + 1)) + half_step(dtype, want)
    # what passes the type's largest number is an infinity
    past = want.abs() - lim > torch.finfo(s.dtype).max
    for name, got in (("backward", back), ("step", step)):
        got = got.cpu().double().view(copies, *grad.shape)
        off = torch.where(past & (got == want.sign() * INF), 0.0, (got - want).abs())
        assert bool((off <= lim).all()), f"{name}: gradient off by {(off - lim).max()} over its bound"  # NaN fails too


def rows_around(value, n, k, dtype, seed, temperature, tail):
    """Eight students and their teachers; `value` is a mask, or where all of a row lies."""
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(8, n, generator=g) * 2.5 * temperature
    full[0, n // 8:] = -INF  # the teacher may not answer there either
    t, i = torch.topk(full, k, dim=1)
    tlse = torch.logsumexp(full.double() / temperature, dim=1).float() if tail else None
    s = 0.6 * full.clamp_min(-1e4) + 1.5 * temperature * torch.randn(8, n, generator=g)
    near = (value + 2.5 * temperature * torch.randn(n, generator=g, dtype=torch.float64)).float()
    s[0, n // 8:] = value                                  # whole waves' columns masked
    s[1] = value                                           # a row masked
    s[2] = s[2].scatter(0, i[2], -INF).clamp(max=value)    # all but S
    s[2, i[2]] = torch.randn(k, generator=g)
    s[3] = near                                            # little apart, as far as the type tells
    s[4, n // 2::5] = -value                               # some as far above
    s[5, ::2] = value                                      # every other one
    s[6, ::2], s[6, 1::2] = -INF, value
    s[6, i[6]] = value
    return s.to(DTYPES[dtype]), t, i, tlse


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [0.5, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("n,k,copies", [(9001, 30, 1), (601, 6, 38), (140_001, 5, 1)])
def test_distill_masks(dtype, tail, temperature, n, k, copies):
    for value in (-1e4, -3e6, -1e9, -3e9, -1e10, -1e12, -1e20):
        log(f"distill masks {dtype} tail={tail} T={temperature} n={n} value={value}")
        s, t, i, tlse = rows_around(value, n, k, dtype, 10 + n, temperature, tail)
        check_distill(s, t, i, temperature, tlse, copies)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k,copies", [(5000, 12, 1), (4099, 20, 35), (135_001, 9, 1)])
def test_distill_large_logits_and_small_temperatures(dtype, n, k, copies):
    """Logits over a temperature of about 2^19 to 2^33, where neighbours still have shares or no longer do."""
    g = torch.Generator().manual_seed(20 + n)
    for tail in (False, True):
        for power, temperature in ((19, 1.0), (21, 1.0), (24, 0.3), (27, 1.0), (31, 1.0), (14, 1e-3), (10, 1e-5), (3, 1e-9)):
            if dtype == "fp16" and power > 14:
                continue
            log(f"distill large {dtype} tail={tail} 2^{power} T={temperature} n={n}")
            sign = torch.tensor([1.0, -1.0] * 4, dtype=torch.float64)[:, None]
            s = sign * 2.0 ** power + 2 * temperature * torch.randn(8, n, generator=g, dtype=torch.float64)
            s = s.to(DTYPES[dtype])
            t, i = torch.topk(2 * temperature * torch.randn(8, n, generator=g), k, dim=1)
            tlse = torch.logsumexp(t.double() / temperature, 1).float() + 0.5 if tail else None
            check_distill(s, t, i, temperature, tlse, copies)


# ------------------------------------------------------------- balance loss

def balance_oracle(x, counts, alpha, beta, score):
    """The loss, the sum of its terms' sizes, the gradient, the sum of its terms' sizes, and how far each element lies
    below its row's largest."""
    x = x.double()
    tokens, experts = x.shape
    load = counts.double() * experts / max(int(counts.sum()), 1)
    weight = x if score == "softmax" else torch.nn.functional.logsigmoid(x)  # p is the softmax of this
    logp, top, rest = log_softmax(weight, 1.0)
    live = top > -INF
    p = torch.where(live, torch.exp(logp), 0.0)
    z = torch.where(live, top + rest, 0.0) if score == "softmax" else torch.zeros_like(top)
    slope = torch.sigmoid(-x) if score == "sigmoid" else torch.ones_like(x)
    b = (p * load).sum(1, keepdim=True)
    row = alpha * b + beta * z * z
    size = abs(alpha) * b + abs(beta) * z * z
    grad = p * slope * (alpha * (load - b) + 2 * beta * z) / tokens
    terms = p * slope * (abs(alpha) * (load + b) + 2 * abs(beta) * z.abs()) / tokens
    below = torch.where(live & (logp > -200), logp.abs(), 0.0)
    return row.mean(), size.mean(), grad, terms, below


def check_balance(x, idx, alpha=0.3, beta=0.0, score="softmax"):
    dtype = {v: k for k, v in DTYPES.items()}[x.dtype]
    tokens, experts = x.shape
    counts = torch.bincount(idx.flatten(), minlength=experts)
    loss, size, grad, terms, below = balance_oracle(x, counts, alpha, beta, score)
    gx, gi = x.cuda(), idx.cuda()
    got, c, kept = lrs.expert_balance_forward(gx, gi, alpha, beta, score)
    back = lrs.expert_balance_backward(gx, c, kept, alpha, beta, score)
    total, _, step = lrs.expert_balance_step(gx, gi, alpha, beta, score)
    torch.cuda.synchronize()
    # a lane adds at most experts / 4 terms in 32 bits (its share of a row); an exponential and the products around it
    # round some tens of times, twice over in a sum of p f
    tol = (experts / 4 + 64) * ULP
    bound = 2 * tol * float(size) + ULP * abs(float(loss))
    for name, l in (("forward", got), ("step", total)):
        assert abs(float(l) - float(loss)) <= bound, f"{name}: loss {float(l)} for {float(loss)}, {bound}"
    lim = terms * (2 * tol + 4 * ULP * (below + 1)) + half_step(dtype, grad)
    for name, g in (("backward", back), ("step", step)):
        off = (g.cpu().double() - grad).abs()
        assert bool((off <= lim).all()), f"{name}: gradient off by {(off - lim).max()} over its bound"


def routed(tokens, experts, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(tokens, experts, generator=g, dtype=torch.float64) * 1.5, torch.randint(0, experts, (tokens, k), generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,experts", [(40, 24), (700, 256), (30, 700)])
@pytest.mark.parametrize("beta", [0.0, 1e-3])
def test_balance_softmax_large_logits(dtype, tokens, experts, beta):
    for value in (-1e4, 3e6, -3e9, -1e10, 1e10, -1e12, 1e12):
        log(f"balance {dtype} {tokens}x{experts} beta={beta} value={value}")
        x, idx = routed(tokens, experts, 4, 30 + experts)
        x[3::7] = value                       # tokens whose logits are all at it
        x[1::7] += value                      # around it
        x[2::7, ::3] = -abs(value)            # masked experts
        x[4::7, 1] = abs(value)               # one expert far above
        check_balance(x.to(DTYPES[dtype]), idx, 0.3, beta)


def test_balance_rows_do_not_depend_on_their_neighbours():
    x, idx = routed(64, 16, 2, 40)
    x = x.float().cuda()
    counts = torch.arange(1, 17, dtype=torch.int32, device="cuda")
    alone = lrs.expert_balance_backward(x, counts)
    x2 = x.clone()
    x2[::2] = -1e30
    beside = lrs.expert_balance_backward(x2, counts)
    assert torch.equal(alone[1::2], beside[1::2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("beta", [0.0, 1e-8])
def test_balance_square_of_a_large_log_sum(dtype, beta):
    """The square of a log-sum-exp passes 32 bits long before the logits do."""
    top = torch.finfo(DTYPES[dtype]).max
    for value in (-1e20, 3e22, -top, top):
        log(f"balance square {dtype} beta={beta} value={value}")
        x, idx = routed(50, 40, 3, 50)
        x[5] = value
        if beta and abs(value) > 1e23:  # the loss itself passes 32 bits
            x = x.to(DTYPES[dtype]).cuda()
            loss, _, grad = lrs.expert_balance_step(x, idx.cuda(), 0.3, beta)
            assert float(loss) == INF and not torch.isnan(grad).any()
        else:
            check_balance(x.to(DTYPES[dtype]), idx, 0.3, beta)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("tokens,experts", [(40, 24), (700, 160), (64, 256), (30, 700), (5, 4096)])
def test_balance_sigmoid_of_low_rows(dtype, tokens, experts):
    """Rows whose logits are all far below 0: sigmoids divided by their sum tend to a softmax."""
    for value in (-12.0, -60.0, -95.0, -300.0, -1e4, -3e6, -1e10, -1e20, -3e38):
        if dtype == "fp16" and value < -6e4:
            continue
        log(f"balance sigmoid {dtype} {tokens}x{experts} value={value}")
        x, idx = routed(tokens, experts, 4, 60 + experts)
        x[3::7] = value                       # tokens whose logits are all at it
        x[1::7] += value                      # around it
        x[2::7, ::3] = value                  # low experts
        x[4::7] = -INF                        # all at it but masked experts
        x[4::7, 1::2] = value
        x[0] = -INF                           # no expert at all
        check_balance(x.to(DTYPES[dtype]), idx, 0.3, 0.0, "sigmoid")


def test_balance_sigmoid_low_rows_beside_others():
    x, idx = routed(64, 16, 2, 70)
    x = x.float().cuda()
    counts = torch.arange(1, 17, dtype=torch.int32, device="cuda")
    alone = lrs.expert_balance_backward(x, counts, score="sigmoid")
    x2 = x.clone()
    x2[::2] = -100.0
    mask = torch.ones(64, dtype=torch.bool, device="cuda")
    kept = torch.tensor([64], dtype=torch.int32, device="cuda")
    beside = lrs.expert_balance_backward(x2, counts, score="sigmoid")
    assert torch.equal(alone[1::2], beside[1::2])
    # rows that do not count are not looked at
    x2[::2] = float("nan")
    mask[::2] = False
    beside = lrs.expert_balance_backward(x2, counts, kept, score="sigmoid", row_mask=mask)
    assert torch.equal(alone[1::2], beside[1::2]) and bool((beside[::2] == 0).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k,copies", [(700, 6, 1), (9001, 30, 1), (601, 6, 38), (140_001, 5, 1)])
def test_distill_temperatures_past_32_bits(dtype, n, k, copies):
    """Temperatures whose inverse is below what 32 bits hold whole, with masks."""
    for temperature in (1e30, 1e37, 2e38, 1e40, 1e46, 1e300):
        for tail in (False, True):
            log(f"distill {dtype} n={n} T={temperature} tail={tail}")
            g = torch.Generator().manual_seed(80 + n)
            s = torch.randn(5, n, generator=g).to(DTYPES[dtype])
            t, i = torch.topk(torch.randn(5, n, generator=g), k, dim=1)
            s[0, ::3] = -INF
            s[0, i[0]] = 0.5
            s[1, ::2] = torch.finfo(s.dtype).min
            s[2, ::5] = torch.finfo(s.dtype).max
            s[3] = s[3].scatter(0, i[3], -INF).clamp(max=-INF)   # all the student has is on S
            s[3, i[3]] = 1.0
            tlse = torch.full((5,), float(torch.tensor(2.0 * k).log())) if tail else None
            if tail:
                s[3, 0] = 0.25
            check_distill(s, t, i, temperature, tlse, copies)


def test_temperature_refusals():
    s, t, i = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 2, device="cuda"), torch.zeros(2, 2, dtype=torch.int64, device="cuda")
    for call in (lrs.topk_distill_step, lrs.topk_distill_forward, lrs.topk_distill_loss):
        for temperature in (0.0, -1.0, INF, float("nan"), 4e-39, 1e-320):
            with pytest.raises(ValueError):
                call(s, t, i, temperature)
        call(s, t, i, 5e-39)


@pytest.mark.parametrize("n", [300, 70_001])
@pytest.mark.parametrize("tail", [False, True])
def test_temperature_has_64_bits(n, tail):
    """Losses just below 2048, whose rounding is half that of an inverse temperature in 32 bits."""
    inverse = 1 + 1.02 * 2.0 ** -24  # 32 bits would hold 1 + 2^-23
    rows = 256
    g = torch.Generator().manual_seed(90)
    s = torch.full((rows, n), -3000.0)
    s[:, 0] = 0.0
    s[:, 5] = -2047 + 7 * torch.rand(rows, generator=g)
    t, i = torch.ones(rows, 1), torch.full((rows, 1), 5)
    tlse = torch.full((rows,), float(inverse)) if tail else None  # what its own rounding leaves over is a tail of 2^-24
    want, size, _, _, _ = distill_oracle(s, t, i, 1 / inverse, tlse)
    _, row_loss, _ = lrs.topk_distill_forward(s.cuda(), t.cuda(), i.cuda(), 1 / inverse, None if tlse is None else tlse.cuda())
    assert bool((want < 2048).all()) and bool((want > 2039).all())
    # rounded once; half a step below 2048 is 2^-14
    off = (row_loss.cpu().double() - want).abs()
    assert bool((off <= 2.0 ** -14 + 8 * ULP).all()), float(off.max())
    wrong = distill_oracle(s, t, i, 1 / (1 + 2.0 ** -23), tlse)[0]
    assert bool(((row_loss.cpu().double() - wrong).abs() > 2.0 ** -14 + 8 * ULP).any())
