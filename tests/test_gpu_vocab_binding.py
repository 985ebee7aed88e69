"""The vocabulary operators by every way in: the compiled binding against the
Python one (which calls with options take), refusals, streams and graphs at the
sizes where the kernels change form, and a small model that uses them together."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_same_as_python(dtype):
    opts = lrs.SortOptions()
    g = torch.Generator().manual_seed(3)
    weight = torch.randn(300, 41, generator=g).to(dtype).cuda()[:, 1:]
    batch = torch.randint(-1, 301, (6, 20), generator=g).cuda()
    for ids in (batch, batch[:, :-1], batch[2], batch[:, 3], batch.int(), batch.view(2, 3, 20), batch[0, 0]):
        for out in (None, torch.float32, torch.float16):
            same(lrs.embedding_forward(weight, ids, 1.5, out), lrs.embedding_forward(weight, ids, 1.5, out, options=opts))
            grad = torch.randn(*ids.shape, 40, generator=g).to(dtype).cuda()
            for padding in (None, 7):
                same(lrs.embedding_backward(grad, ids, 300, 1.5, padding, out),
                     lrs.embedding_backward(grad, ids, 300, 1.5, padding, out, options=opts))
            same(lrs.embedding_backward(grad.reshape(-1, 40), ids, 300), lrs.embedding_backward(grad, ids, 300, options=opts))
    logits = torch.randn(50, 1003, generator=g).to(dtype).cuda()
    tokens = torch.randint(-1, 1003, (50,), generator=g).cuda()
    up, down = torch.randn(2, 50, generator=g).cuda()
    for mask in (None, torch.rand(50, generator=g).cuda() < 0.6):
        for ids in (tokens, tokens.int()):
            args = (logits[:, 2:], ids, 0.9, mask)
            forward = lrs.token_logprobs_forward(*args)
            same(forward, lrs.token_logprobs_forward(*args, options=opts))
            same(lrs.token_logprobs(*args), forward[:2])
            for a, b in ((up, down), (up, None), (None, down)):
                same(lrs.token_logprobs_step(*args[:2], a, b, *args[2:]), lrs.token_logprobs_step(*args[:2], a, b, *args[2:], options=opts))
                same(lrs.token_logprobs_backward(*args[:2], forward[2], a, b, *args[2:]),
                     lrs.token_logprobs_backward(*args[:2], forward[2], a, b, *args[2:], options=opts))
    for k in (0, 1, 30, 600):
        same(lrs.token_logprobs_topk(logits, tokens, k), lrs.token_logprobs_topk(logits, tokens, k, options=opts))


def test_refusals():
    weight, ids = torch.randn(20, 16, device="cuda"), torch.zeros(3, 5, dtype=torch.int64, device="cuda")
    grad = torch.randn(3, 5, 16, device="cuda")
    bad = [
        lambda: lrs.embedding_forward(weight.double(), ids), lambda: lrs.embedding_forward(weight.T, ids),
        lambda: lrs.embedding_forward(weight, ids.float()), lambda: lrs.embedding_forward(weight, ids.cpu()),
        lambda: lrs.embedding_forward(weight, ids.T), lambda: lrs.embedding_forward(weight, ids, dtype=torch.float64),
        lambda: lrs.embedding_forward(weight, ids, out=grad[:, :, :15]), lambda: lrs.embedding_forward(weight, ids, out=grad.mT.contiguous().mT),
        lambda: lrs.embedding_forward(weight, ids, out=grad, dtype=torch.float16), lambda: lrs.embedding_forward(weight, ids, out=weight[:15]),
        lambda: lrs.embedding_lookup(weight, ids.float()), lambda: lrs.embedding_lookup(weight, ids, padding_index=20),
        lambda: lrs.embedding_lookup(weight, ids, padding_index=-1), lambda: lrs.embedding_lookup(weight, ids, padding_index=1.5),
        lambda: lrs.embedding_lookup(weight[0], ids), lambda: lrs.embedding_lookup(weight, ids, dtype=torch.int32),
        lambda: lrs.embedding_backward(grad[:, :4], ids, 20), lambda: lrs.embedding_backward(grad.double(), ids, 20),
        lambda: lrs.embedding_backward(grad, ids, 20, padding_index=20), lambda: lrs.embedding_backward(grad, ids, 20, accumulate=True),
        lambda: lrs.embedding_backward(grad, ids, 20, grad_out=weight[:19]), lambda: lrs.embedding_backward(grad, ids, 20, grad_out=weight.double()),
        lambda: lrs.embedding_backward(grad, ids, 20, grad_out=weight, dtype=torch.float16),
        lambda: lrs.embedding_backward(grad, ids, 20, grad_out=weight[:1].expand(20, 16)),
        lambda: lrs.embedding_backward(grad, ids, 15, grad_out=grad.view(15, 16)),
        lambda: lrs.embedding_backward(grad, ids, 20, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: lrs.embedding_backward(grad[..., ::2], ids, 20), lambda: lrs.embedding_backward(grad, ids, 20, math.nan),
    ]
    for scale in (math.inf, math.nan, 1e39):
        bad += [lambda s=scale: lrs.embedding_forward(weight, ids, s), lambda s=scale: lrs.embedding_lookup(weight, ids, s),
                lambda s=scale: lrs.embedding_backward(grad, ids, 20, s)]
    logits, tokens, up = torch.randn(4, 30, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    stats = lrs.token_logprobs_forward(logits, tokens)[2]
    mask = torch.ones(4, dtype=torch.bool, device="cuda")
    for call in (lrs.token_logprobs, lrs.token_logprobs_forward, lambda *a, **k: lrs.token_logprobs_topk(a[0], a[1], 3, *a[2:], **k),
                 lambda *a, **k: lrs.token_logprobs_step(a[0], a[1], up, up, *a[2:], **k),
                 lambda *a, **k: lrs.token_logprobs_backward(a[0], a[1], stats, up, up, *a[2:], **k)):
        bad += [lambda call=call: call(logits.double(), tokens), lambda call=call: call(logits.T, tokens),
                lambda call=call: call(logits, tokens[:3]), lambda call=call: call(logits, tokens[:, None]),
                lambda call=call: call(logits, tokens.float()), lambda call=call: call(logits, tokens.cpu()),
                lambda call=call: call(logits, tokens, 0.0), lambda call=call: call(logits, tokens, math.inf),
                lambda call=call: call(logits, tokens, 1e-40), lambda call=call: call(logits, None)]
    for call in (lrs.token_logprobs, lrs.token_logprobs_forward):
        bad += [lambda call=call: call(logits, tokens, 1.0, mask[:3]), lambda call=call: call(logits, tokens, 1.0, mask.float())]
    bad += [lambda: lrs.token_logprobs_topk(logits, tokens, 31), lambda: lrs.token_logprobs_step(logits, tokens, None),
            lambda: lrs.token_logprobs_step(logits, tokens, up.double()), lambda: lrs.token_logprobs_step(logits, tokens, up[:3]),
            lambda: lrs.token_logprobs_step(logits, tokens, up, grad_out=logits), lambda: lrs.token_logprobs_backward(logits, tokens, stats, None),
            lambda: lrs.token_logprobs_step(logits, tokens, up, grad_out=torch.empty(4, 29, device="cuda")),
            lambda: lrs.token_logprobs_backward(logits, tokens, stats[:3], up), lambda: lrs.token_logprobs_backward(logits, tokens, stats.int(), up)]
    for i, call in enumerate(bad):
        with pytest.raises(lrs.RadixSortArgumentError):
            call()
            pytest.fail(f"call {i} was taken")


def test_no_workspace_needed():
    """Where the query says 0 bytes, the workspace may be NULL."""
    from lsd_radix_sort_amd.vocab_ops import _logprob_inputs, _token_ids
    import ctypes
    lib, P = lrs.load_library(), ctypes.c_void_p
    logits, tokens = torch.randn(2, 3000, device="cuda"), torch.tensor([7, 2999], device="cuda")
    want = lrs.token_logprobs_topk(logits, tokens, 5)
    assert lrs.token_logprobs_workspace_size(2, 3000, 5, torch.float32) == 0
    out = [torch.empty_like(t) for t in want]
    d = _logprob_inputs(logits, tokens, 1.0)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.token_logprobs_topk(ctypes.byref(d), 5, *(P(t.data_ptr()) for t in out), None, 0, P(stream), None) == 0
    same(tuple(out), want)
    table, none = torch.ones(40, 8, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    assert lrs.embedding_backward_workspace_size(0, 40, 8) == 0
    assert lib.embedding_backward(None, 8, ctypes.byref(_token_ids(none, none.device)), P(table.data_ptr()), 8, 40, 8, 2, 2, 1.0, -1, 0,
                                  None, 0, P(stream), None) == 0
    assert not table.any()


def test_too_many_elements():
    rows, n = 1 << 25, 65_536  # rows that all lie at the same place
    logits = torch.zeros(1, n, dtype=torch.float16, device="cuda").expand(rows, n)
    tokens = torch.zeros(1, dtype=torch.int64, device="cuda").expand(rows)
    for call in (lrs.token_logprobs, lrs.token_logprobs_forward):
        with pytest.raises(lrs.RadixSortArgumentError):
            call(logits, tokens)
    with pytest.raises(lrs.RadixSortArgumentError):
        lrs.embedding_lookup(logits, tokens[:1])
    with pytest.raises(lrs.RadixSortArgumentError):
        lrs.embedding_backward(logits, tokens, 8)


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(4)
    work = []
    for seed in range(2):
        ids = torch.randint(0, 5000, (40_000,), generator=g).cuda()
        grad = torch.randn(40_000, 136, generator=g).to(torch.bfloat16).cuda()
        logits = torch.randn(600, 20_011, generator=g).to(torch.float16).cuda()
        tokens = torch.randint(0, 20_011, (600,), generator=g).cuda()
        work.append(lambda ids=ids, grad=grad, logits=logits, tokens=tokens: (
            lrs.embedding_backward(grad, ids, 5000), *lrs.token_logprobs_topk(logits, tokens, 12),
            *lrs.token_logprobs_topk(logits[:9], tokens[:9], 100)))
    want = [w() for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            same(out, want[i])


def test_graphs_of_many_tokens_and_long_rows():
    """Captured where the sort has several passes, rows are shared, and alternatives are selected on their own."""
    g = torch.Generator().manual_seed(5)
    ids = torch.zeros(40_000, dtype=torch.int64, device="cuda")
    grad = torch.zeros(40_000, 24, device="cuda")
    logits, tokens = torch.zeros(3, 150_000, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    def calls():
        return (lrs.embedding_backward(grad, ids, 70_000, 2.0), *lrs.token_logprobs_topk(logits, tokens, 4),
                *lrs.token_logprobs_topk(logits, tokens, 600), *lrs.token_logprobs_step(logits, tokens, up, up))
    up = torch.randn(3, generator=g).cuda()
    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for turn in range(3):
        ids.copy_(torch.randint(-1, 70_000 if turn else 40, (40_000,), generator=g))
        grad.copy_(torch.randn(40_000, 24, generator=g))
        logits.copy_(torch.randn(3, 150_000, generator=g) * (turn + 1))
        tokens.copy_(torch.randint(0, 150_000, (3,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        same(out, calls())


class Model(torch.nn.Module):
    """A tied table, a layer and a policy loss: the operators as a training program uses them."""

    def __init__(self, vocab, width, g):
        super().__init__()
        self.table = torch.nn.Parameter(torch.randn(vocab, width, generator=g) * 0.3)
        self.layer = torch.nn.Parameter(torch.randn(width, width, generator=g) * 0.2)

    def loss(self, lookup, logprobs, batch, weights, mask):
        x = lookup(self.table, batch[:, :-1], math.sqrt(self.table.size(1)))
        h = torch.tanh(x @ self.layer).reshape(-1, self.table.size(1))
        lp, entropy = logprobs(h @ self.table.T, batch[:, 1:].reshape(-1), 0.8, mask)
        return -(weights * lp).sum() - 0.02 * (entropy * mask).sum()


def test_together():
    """The gradients of a model through lookup, log probabilities and entropy, against the same model in 64 bits."""
    g = torch.Generator().manual_seed(6)
    vocab, width = 211, 24
    model = Model(vocab, width, g)
    batch = torch.randint(0, vocab, (5, 9), generator=g)
    batch[1, 4:] = 3  # padding
    weights = torch.rand(40, generator=g)
    mask = (batch[:, 1:] != 3).reshape(-1)

    def lookup64(table, ids, scale):
        return torch.where((ids == 3)[..., None], table.detach()[ids], table[ids]) * scale

    def logprobs64(logits, tokens, temperature, mask):
        logp = torch.log_softmax(logits / temperature, dim=1)
        return torch.gather(logp, 1, tokens[:, None])[:, 0] * mask, -(logp.exp() * logp).sum(1) * mask
    exact = Model(vocab, width, g).double()
    exact.load_state_dict({k: v.double() for k, v in model.state_dict().items()})
    want = exact.loss(lookup64, logprobs64, batch, weights.double(), mask)
    want.backward()
    model = model.cuda()
    got = model.loss(lambda t, i, s: lrs.embedding_lookup(t, i, s, padding_index=3), lrs.token_logprobs, batch.cuda(), weights.cuda(), mask.cuda())
    got.backward()
    # 32-bit products of 24 terms between the operators: some 100 half steps of the largest terms
    assert abs(float(got.detach().cpu()) - float(want.detach())) <= 300 * 2.0 ** -24 * float(want.detach().abs())
    for p, q in zip(model.parameters(), exact.parameters()):
        assert float((p.grad.cpu().double() - q.grad).norm() / q.grad.norm()) <= 300 * 2.0 ** -24
    # one step of serving: the next tokens' alternatives from the last places
    with torch.no_grad():
        x = lrs.embedding_forward(model.table, batch[:, -1].cuda(), math.sqrt(width))
        logits = torch.tanh(x @ model.layer) @ model.table.T
        _, indices = lrs.segmented_row_topk(logits, 5)
        lp, _, ranks, top, alternatives = lrs.token_logprobs_topk(logits, indices[:, 2].contiguous(), 5)
        assert torch.equal(alternatives, indices) and ranks.tolist() == [2] * 5 and torch.equal(lp, top[:, 2])


@pytest.mark.parametrize("tokens,width", [(200, 40), (5000, 264), (40_000, 16)])
def test_ids_that_do_not_fit(tokens, width):
    """Ids whose low 32 bits name a row are outside all the same; so is such a padding index."""
    from lsd_radix_sort_amd.vocab_ops import _token_ids
    import ctypes
    g = torch.Generator().manual_seed(tokens)
    vocab = 50
    inside = torch.randint(0, vocab, (tokens,), generator=g)
    far = torch.tensor([1 << 32, -(1 << 32), 1 << 31, -(1 << 63), (1 << 63) - vocab, 1 << 62])[torch.randint(0, 6, (tokens,), generator=g)]
    out = torch.rand(tokens, generator=g) < 0.5
    ids, only = torch.where(out, inside + far, inside).cuda(), torch.where(out, -1, inside).cuda()
    weight, grad = torch.randn(vocab, width, generator=g).cuda(), torch.randn(tokens, width, generator=g).cuda()
    same(lrs.embedding_forward(weight, ids), lrs.embedding_forward(weight, only))
    want = lrs.embedding_backward(grad, only, vocab)
    same(lrs.embedding_backward(grad, ids, vocab), want)
    lib, P = lrs.load_library(), ctypes.c_void_p
    got = torch.empty_like(want)
    ws = torch.empty(lrs.embedding_backward_workspace_size(tokens, vocab, width), dtype=torch.uint8, device="cuda")
    assert lib.embedding_backward(P(grad.data_ptr()), width, ctypes.byref(_token_ids(only, only.device)), P(got.data_ptr()), width, vocab,
                                  width, 2, 2, 1.0, (1 << 32) + 7, 0, P(ws.data_ptr()), ws.numel(),
                                  P(torch.cuda.current_stream().cuda_stream), None) == 0
    same(got, want)
    logits = torch.randn(tokens, vocab, generator=g).cuda()
    same(lrs.token_logprobs_topk(logits, ids, 3), lrs.token_logprobs_topk(logits, only, 3))
    up = torch.randn(tokens, generator=g).cuda()
    same(lrs.token_logprobs_step(logits, ids, up, up), lrs.token_logprobs_step(logits, only, up, up))


def test_backward_in_a_graph_with_its_forward():
    """Forward and backward of the autograd forms captured together, where no graph of the leaves is alive."""
    g = torch.Generator().manual_seed(8)
    weight = torch.randn(300, 40, generator=g).cuda().requires_grad_(True)
    ids = torch.randint(0, 300, (64,), generator=g).cuda()

    def step():
        logprobs, entropy = lrs.token_logprobs(lrs.embedding_lookup(weight, ids, 2.0), ids % 40)
        return torch.autograd.grad((logprobs, entropy), weight, (torch.ones_like(logprobs), torch.ones_like(entropy)))[0]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        ids.copy_(torch.randint(0, 300, (64,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        same(out, step())
