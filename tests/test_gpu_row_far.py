"""Rows that lie more than 2^31 elements apart give the bits that neighbouring rows give."""
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

STRIDE = (1 << 31) + 5


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def far(rows: torch.Tensor) -> torch.Tensor:
    """The same two rows in one buffer, STRIDE elements apart."""
    n = rows.shape[1]
    buf = torch.empty(STRIDE + n, dtype=rows.dtype, device="cuda")
    out = buf.as_strided((2, n), (STRIDE, 1))
    out.copy_(rows)
    return out


@pytest.mark.parametrize("n", [40, 200, 5000, 60_000, 150_000])
def test_topk(n):
    x = torch.randn(2, n, device="cuda").bfloat16()
    near, there = lrs.segmented_row_topk(x, 20), lrs.segmented_row_topk(far(x), 20)
    assert torch.equal(near[0], there[0]) and torch.equal(near[1], there[1])


@pytest.mark.parametrize("n", [300, 50_001, 150_001])
def test_distill(n):
    x = torch.randn(2, n, device="cuda").bfloat16()
    v, i = lrs.segmented_row_topk(torch.randn(2, n, device="cuda"), 7)
    near = lrs.topk_distill_step(x, v, i)
    grad = far(torch.zeros_like(x))
    there = lrs.topk_distill_step(far(x), v, i, grad_out=grad)
    assert all(torch.equal(a, b) for a, b in zip(near, there))
    stats = lrs.topk_distill_forward(x, v, i)[2]
    back = lrs.topk_distill_backward(far(x), v, i, stats, grad_out=grad)
    assert torch.equal(back, lrs.topk_distill_backward(x, v, i, stats))


def test_balance():
    x = torch.randn(2, 96, device="cuda").bfloat16()
    _, ids = lrs.segmented_row_topk(x, 4)
    near = lrs.expert_balance_step(x, ids, 0.5, 1e-2)
    there = lrs.expert_balance_step(far(x), far(ids.int()), 0.5, 1e-2, grad_out=far(torch.zeros_like(x)))
    assert all(torch.equal(a, b) for a, b in zip(near, there))
