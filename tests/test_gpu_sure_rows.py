"""Rows whose mass lies on one token: their log probabilities are never above 0
and their entropies never below, in every form of the operator."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = 2.0 ** -24  # half a step of 32-bit numbers
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


# rows alone of every number of threads, held and read twice, and shared ones
SHAPES = [(2, 5), (600, 1000), (2100, 4096), (600, 8000), (400, 16001), (48, 32000), (300, 40000), (257, 65000), (64, 131072),
          (3, 131072), (1, 300000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["one", "far", "near"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_signs(dtype, kind, shape):
    rows, n = shape
    print(dtype, kind, shape, flush=True)
    g = torch.Generator().manual_seed(rows + n)
    t = DTYPES[dtype]
    # how large the one is: around 0 up to what 16 bits hold
    top = (torch.randn(rows, generator=g) * 2.0 ** torch.randint(-3, 13, (rows,), generator=g)).to(t)
    at = torch.randint(0, n, (rows,), generator=g)
    for temperature in (1.0, 0.7):
        if kind == "one":
            x = torch.full((rows, n), -INF, dtype=t)
        else:
            x = (top[:, None].float() - (200.0 if kind == "far" else 14.0) * temperature).to(t).expand(rows, n).clone()
        x[torch.arange(rows), at] = top
        logits, tokens = x.cuda(), at.cuda()
        up = torch.ones(rows, device="cuda")
        k = min(n // 2, 4)
        forward = lrs.token_logprobs_forward(logits, tokens, temperature)
        topk = lrs.token_logprobs_topk(logits, tokens, k, temperature)
        wide = lrs.token_logprobs_topk(logits, tokens, min(n, 600), temperature)
        step = lrs.token_logprobs_step(logits, tokens, up, up, temperature)
        # A logit of x / T base 2 is held less a reference that is off by half a step of it, so a term d p of the
        # entropy by half a step of that.
        size = top.double().abs().cuda() * math.log2(math.e) / temperature
        for name, (lp, h) in dict(forward=forward[:2], topk=topk[:2], wide=wide[:2], step=step[:2]).items():
            assert bool((lp <= 0).all()), (name, float(lp.max()))
            assert bool((h >= 0).all()), (name, float(h.min()))
            if kind != "near":
                assert bool((lp == 0).all()), (name, float(lp.min()))
                assert bool((h.double() <= ULP * ULP * 2 * size + 2.0 ** -100).all()), (name, float(h.max()))
        for out in (topk, wide):
            assert bool((out[3] <= 0).all()), float(out[3].max())
            if kind != "near":
                assert bool((out[3][:, 0] == 0).all())
                # (14 less can round to the same logit: bf16 steps are 32 from 2^12 on)
                assert bool((out[2] == 0).all()) and torch.equal(out[4][:, 0], tokens)
