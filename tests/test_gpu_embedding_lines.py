"""The table's gradient of ids that are lines of a longer batch, or a column of
one, in each of the ways to order them, set and added."""
import pytest
import torch

from test_gpu_embedding import DTYPES, check_gradient, make_ids

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


# up to 32768 tokens are ordered directly, 2, 8, 16 or 32 of them a lane; more are sorted
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("lines,length", [(3, 683), (4, 2047), (8197, 1), (7, 1171), (11, 1489), (5, 6553), (2, 16384), (3, 13337),
                                          (40, 1001), (40009, 1)])
def test_gradient(id_type, lines, length):
    g = torch.Generator().manual_seed(lines + length)
    tokens = lines * length
    for cut, vocab, width, dtype, out in ((1, 5003, 40, "bf16", "fp32"), (37, 999, 132, "fp16", "fp16")):
        batch = make_ids("text", torch.Size((lines, length + cut)), vocab, g).to(id_type)
        batch[0, 0] = -1
        ids = batch[:, cut // 2:cut // 2 + length]
        ours = batch.cuda()[:, cut // 2:cut // 2 + length]
        if length == 1 and cut == 37:  # a column
            ids, ours = ids[:, 0], ours[:, 0]
        assert not ours.is_contiguous()
        print(id_type, tuple(ours.shape), ours.stride(), vocab, width, flush=True)
        grad = torch.randn(tokens, width, generator=g).to(DTYPES[dtype])
        got = lrs.embedding_backward(grad.cuda(), ours, vocab, 1.5, 7, dtype=DTYPES[out])
        check_gradient(got.cpu(), grad, ids, vocab, 1.5, 7)
        assert torch.equal(got, lrs.embedding_backward(grad.cuda(), ours.contiguous(), vocab, 1.5, 7, dtype=DTYPES[out]))
        old = torch.randn(vocab, width, generator=g).to(DTYPES[out])
        added = lrs.embedding_backward(grad.cuda(), ours, vocab, 1.5, 7, grad_out=old.cuda(), accumulate=True)
        check_gradient(added.cpu(), grad, ids, vocab, 1.5, 7, old)
