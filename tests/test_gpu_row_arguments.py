"""What the row operators refuse is refused as RadixSortArgumentError, by every way in, before memory is asked for."""
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def test_experts_out_of_range():
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for experts in (-5, 0, 4097, 1 << 50, 2.5):
        with pytest.raises(lrs.RadixSortArgumentError, match="experts"):
            lrs.expert_counts(ids, experts)


def test_missing_counts():
    for experts in (1, 8):
        with pytest.raises(lrs.RadixSortArgumentError, match="counts"):
            lrs.expert_balance_backward(torch.zeros(4, experts, device="cuda"), None)


def test_k_is_a_whole_number():
    x = torch.randn(3, 9, device="cuda")
    for k in (2.7, "2", None):
        with pytest.raises(lrs.RadixSortArgumentError, match="k must be"):
            lrs.segmented_row_topk(x, k)
    assert lrs.segmented_row_topk(x, torch.tensor(2))[0].shape == (3, 2)


def test_too_many_elements():
    # rows of one element each that all lie at the same place: 2^25 rows of 65536 make 2^41
    rows, n = 1 << 25, 65_536
    logits = torch.zeros(1, n, dtype=torch.float16, device="cuda").expand(rows, n)
    values = torch.zeros(1, 1, device="cuda").expand(rows, 1)
    ids = torch.zeros(1, 1, dtype=torch.int64, device="cuda").expand(rows, 1)
    for call in (lrs.topk_distill_loss, lrs.topk_distill_forward):
        with pytest.raises(lrs.RadixSortArgumentError):
            call(logits, values, ids)


def test_workspace_size_of_an_unknown_type():
    for size in (lrs.segmented_row_topk_workspace_size, lrs.topk_distill_workspace_size):
        with pytest.raises(lrs.RadixSortArgumentError, match="float16"):
            size(4, 1000, 8, torch.float64)
