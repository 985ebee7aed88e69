"""Distillation of rows over 256 KB, which several launches share: sums hold
their bits however many terms a thread adds, and every piece of a row counts."""
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


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,n", [(2048, 300_001), (3, 300_001)])
@pytest.mark.parametrize("tail", [False, True])
def test_sums_of_equal_terms(dtype, rows, n, tail):
    """Equal terms round alike in every addition, so a long sum in 32 bits would drift by its length."""
    k = 4
    t = torch.tensor([2.0, 1.0, 0.5, 0.25], device="cuda").expand(rows, k)
    i = torch.tensor([0, 17, n // 2, n - 1], device="cuda").expand(rows, k)
    q = torch.softmax(t[0].double().cpu(), 0)
    tlse = None
    if tail:
        tlse = torch.full((rows,), 3.0, device="cuda")
        q = torch.exp(t[0].double().cpu() - 3.0)
    for level in (-0.3, -0.7, -1.1, -1.9):
        log(f"long sums {dtype} {rows}x{n} tail={tail} level={level}")
        s = torch.full((1, n), level, dtype=DTYPES[dtype])
        s[0, :4096] = 0.0  # so every thread weighs the rest relative to more than their own
        v = s.double()
        lse = torch.logsumexp(v, 1)
        logp = (v - lse)[0, i[0].cpu()]
        want = float((q * (torch.log(q) - logp)).sum())
        if tail:
            off = torch.ones(n, dtype=torch.bool)
            off[i[0].cpu()] = False
            q0 = 1 - float(q.sum())
            want += q0 * float(torch.log(torch.tensor(q0, dtype=torch.float64)) - (torch.logsumexp(v[:, off], 1) - lse)[0])
        _, row_loss, _ = lrs.topk_distill_forward(s.cuda().expand(rows, n), t, i, teacher_lse=tlse)
        # 32 terms at most are added in 32 bits; an exponential and what is done once a row round some times;
        # log2(e) has 32 bits in 16-bit rows, its step twice a rounding
        bound = (32 + 8 + 4 * abs(level)) * ULP + ULP * abs(want)
        off = (row_loss.double() - want).abs().max()
        assert float(off) <= bound, f"off by {float(off)}, bound {bound}"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tail", [False, True])
def test_pieces_beyond_one_bitmap(dtype, tail):
    """So many rows that none is shared: a workgroup takes a row in several pieces of 65536 columns."""
    rows, n, k = 2050, 140_001, 40
    g = torch.Generator().manual_seed(4)
    s = (torch.randn(1, n, generator=g) * 2).to(DTYPES[dtype])
    full = torch.randn(1, n, generator=g) * 2
    t, i = torch.topk(full, k, dim=1)
    i[0, :3] = torch.tensor([65_535, 65_536, n - 1])  # either side of a piece's edge
    tlse = torch.logsumexp(full.double(), 1).float() if tail else None
    args = [s.cuda().expand(rows, n), t.cuda().expand(rows, k), i.cuda().expand(rows, k), 1.0,
            None if tlse is None else tlse.cuda().expand(rows).contiguous()]
    log(f"distill pieces {dtype} tail={tail}")
    total, row_loss, grad = lrs.topk_distill_step(*args)
    assert bool((row_loss == row_loss[0]).all()) and bool((grad == grad[0]).all())
    z, tz = s.double(), t.double()
    logp = torch.log_softmax(z, 1)
    q = torch.softmax(tz, 1) if tlse is None else torch.exp(tz - tlse.double())
    zt = torch.gather(logp, 1, i)
    want = float((q * (torch.log(q) - zt)).sum())
    own = torch.exp(logp)
    member = torch.zeros(1, n, dtype=torch.bool).scatter_(1, i, True)
    target = torch.zeros(1, n, dtype=torch.float64).scatter_(1, i, q)
    if tail:
        q0 = 1 - q.sum()
        logp0 = torch.logsumexp(torch.where(member, -torch.inf, logp), 1)
        want += float(q0 * (torch.log(q0) - logp0))
        target = torch.where(member, target, q0 * torch.exp(logp - logp0))
    tol = (32 + 64) * ULP
    spread = float(z.max() - z.min())
    assert abs(float(row_loss[0]) - want) <= tol + 2 * ULP * abs(want)
    assert abs(float(total) - want) <= tol + 4 * ULP * abs(want)
    grad64 = (own - target)[0] / rows
    lim = (own + target)[0] / rows * (tol + 4 * ULP * (spread + 1)) + grad64.abs() * (torch.finfo(s.dtype).eps / 2) + 2.0 ** -126
    assert bool(((grad[0].cpu().double() - grad64).abs() <= lim).all())
