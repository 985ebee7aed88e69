"""The gradient of log probabilities and entropies at temperatures whose inverse
is below the normal numbers of 32 bits, under derivatives as large."""
import pytest
import torch

from test_gpu_token_logprobs import DTYPES, Reference

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("power", [120, 127, 135, 148, 152])
def test_gradient(dtype, power):
    temperature = 2.0 ** power
    g = torch.Generator().manual_seed(power)
    # held and read twice, a row's workgroup alone and several; few columns, so that each has a share that counts
    for rows, n in ((5, 3), (40, 17), (600, 1000), (2, 140001)):
        print(dtype, power, rows, n, flush=True)
        x = (torch.randn(rows, n, generator=g) * 2.5).to(DTYPES[dtype])
        tokens = torch.randint(-1, n, (rows,), generator=g)
        up, down = (torch.randn(rows, generator=g) * 2.0 ** min(power - 2, 124) for _ in range(2))
        ref = Reference(x, tokens, temperature)
        logits, ids = x.cuda(), tokens.cuda()
        stats = lrs.token_logprobs_forward(logits, ids, temperature)[2]
        for a, b in ((up, down), (up, None), (None, down)):
            ours = [None if t is None else t.cuda() for t in (a, b)]
            ref.gradient(lrs.token_logprobs_step(logits, ids, *ours, temperature)[2].cpu(), a, b)
            ref.gradient(lrs.token_logprobs_backward(logits, ids, stats, *ours, temperature).cpu(), a, b)
