"""The operators at the two ends of a language model's vocabulary, as workloads.

Two operators: the embedding lookup with its scale and the gradient of the
table by sorted tokens (`embedding_forward`, `embedding_backward`,
`embedding_lookup`), and the log probabilities of given tokens with the rows'
entropy, the tokens' ranks, the top alternatives and the gradient
(`token_logprobs_*`).  `run` computes a case in plain torch operations in 32
bits (`own` false) or with this package's entry points (`own` true); `exact`
computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
INF = math.inf


# ------------------------------------------------------------------- cases

def listed():
    return [
        # decoding: the rows of one step's new tokens (latency counts)
        dict(name="lookup decode batch", op="lookup", lines=64, length=1, cut=0, vocab=131072, width=4096, dtype="bf16",
             out="bf16", scale=1.0, pad=0, dropped=0.0, wide=True),
        # a training batch, scaled by the square root of the width
        dict(name="lookup batch bf16", op="lookup", lines=8, length=4096, cut=0, vocab=131072, width=4096, dtype="bf16",
             out="bf16", scale=64.0, pad=0, dropped=0.0, wide=True),
        # 32-bit weights of an odd width into 16 bits; the batch is a slice that leaves out each line's last token, and
        # some tokens are places of another encoder's outputs
        dict(name="lookup odd fp32 to bf16", op="lookup", lines=7, length=1427, cut=1, vocab=50021, width=1031, dtype="fp32",
             out="bf16", scale=32.0, pad=9, dropped=0.1, wide=True),
        # the table's gradient for a training batch over a large vocabulary
        dict(name="gradient bf16", op="gradient", parts=1, lines=8, length=4096, cut=0, vocab=131072, width=4096, dtype="bf16",
             out="bf16", scale=64.0, pad=0, dropped=0.0, wide=True),
        # two micro-batches into one 32-bit gradient, as programs with 32-bit main gradients keep it
        dict(name="gradient two micro-batches", op="gradient", parts=2, lines=4, length=2047, cut=1, vocab=50021, width=1600,
             dtype="bf16", out="fp32", scale=1.0, pad=0, dropped=0.05, wide=True),
        # the smallest: a short sequence through a small model
        dict(name="gradient few tokens", op="gradient", parts=1, lines=1, length=200, cut=0, vocab=5003, width=256,
             dtype="fp32", out="fp32", scale=16.0, pad=0, dropped=0.0, wide=False),
        # the lookup inside a differentiated program, with padding tokens
        dict(name="lookup autograd fp16", op="autograd", lines=4, length=2048, cut=0, vocab=32000, width=2048, dtype="fp16",
             out="fp16", scale=1.0, pad=0, dropped=0.0, wide=True),
        # serving: a sampled token's log probability, its rank and the likeliest alternatives (latency counts)
        dict(name="alternatives one token", op="alternatives", rows=1, n=131072, k=20, dtype="bf16", temperature=1.0, pad=0,
             masked=False, wide=True),
        # the same for a batch under a grammar's mask, softened
        dict(name="alternatives decode batch", op="alternatives", rows=48, n=50021, k=5, dtype="fp16", temperature=0.7, pad=0,
             masked=True, wide=True),
        # the log probabilities of a long prompt
        dict(name="alternatives prompt", op="alternatives", rows=4096, n=131072, k=8, dtype="bf16", temperature=1.0, pad=0,
             masked=False, wide=True),
        # a training step: the log probabilities, the entropy and the gradient of a weighted sum of both
        dict(name="logprobs step bf16", op="logprobs", call="step", rows=4096, n=131072, dtype="bf16", temperature=1.0, pad=0,
             masked=False, wide=True, entropy=True),
        # policy training: forward, a loss on log probabilities and entropy, backward through autograd; padding rows
        dict(name="logprobs autograd fp32", op="logprobs", call="autograd", rows=1027, n=32768, dtype="fp32", temperature=1.0,
             pad=11, masked=True, wide=True, entropy=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["lookup", "gradient", "gradient", "autograd", "alternatives", "alternatives", "logprobs", "logprobs"])
    dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
    if op in ("lookup", "gradient", "autograd"):
        width = _log(rng, 64, 8192)
        if rng.random() < 0.6:  # widths are mostly whole multiples of 32
            width = max(64, width // 32 * 32)
        vocab = _log(rng, 1000, min(131072, (1 << 28) // width))
        tokens = _log(rng, 1, min(65536, (1 << 26) // width))
        lines = _log(rng, 1, min(tokens, 64))
        case = dict(op=op, lines=lines, length=max(1, tokens // lines), cut=rng.choice([0, 0, 1]), vocab=vocab, width=width,
                    dtype=dtype, out=rng.choice([dtype, dtype, "fp32" if op == "gradient" else "bf16"]),
                    scale=rng.choice([1.0, math.sqrt(width)]), pad=rng.choice([0, 0, 8, rng.randint(1, 63)]),
                    dropped=rng.choice([0.0, 0.0, 0.1]), wide=rng.random() < 0.7)
        if op == "gradient":
            case["parts"] = rng.choice([1, 1, 2]) if case["out"] == "fp32" else 1
        return case
    n = _log(rng, 500, 131072)
    rows = _log(rng, 1, min(8192, (1 << 27) // n))
    case = dict(op=op, rows=rows, n=n, dtype=dtype, temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
                pad=rng.choice([0, 0, 8, rng.randint(1, 63)]), masked=rng.random() < 0.4, wide=rng.random() < 0.7)
    if op == "alternatives":
        case["k"] = _log(rng, 1, 64)
    else:
        case.update(call=rng.choice(["step", "forward", "autograd"]), entropy=rng.random() < 0.6)
    return case


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _padded(values, pad):
    """The same rows inside a buffer whose rows are `pad` elements longer."""
    if pad == 0:
        return values
    buf = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device=values.device)
    buf[:, :values.shape[1]] = values
    return buf[:, :values.shape[1]]


def _text(case, g, name_of):
    """Token ids with the frequencies of text, the i-th most frequent about 1 / i as often as the first."""
    shape = (case["lines"], case["length"] + case["cut"])
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    place = (torch.exp(u * math.log(case["vocab"] + 1.0)) - 1.0).long().clamp_(0, case["vocab"] - 1)
    tokens = name_of[place]
    if case["dropped"]:
        tokens[torch.rand(shape, generator=g, device="cuda") < case["dropped"]] = -1
    return (tokens if case["wide"] else tokens.int())[:, :case["length"]]


def _prepare_embedding(case, g):
    vocab, width, dtype, out = case["vocab"], case["width"], DTYPES[case["dtype"]], DTYPES[case["out"]]
    name_of = torch.randperm(vocab, generator=g, device="cuda")
    state = dict(case=case)
    count = case["lines"] * case["length"]
    if case["op"] != "gradient":
        weight = torch.randn(vocab, width, generator=g, device="cuda").mul_(0.02).to(dtype)
        state["weight"] = _padded(weight, case["pad"])
        state["tokens"] = _text(case, g, name_of)
    if case["op"] == "autograd":
        state["weight"] = state["weight"].detach().requires_grad_(True)
        state["padding"] = int(name_of[0])  # the batch is padded with one id
        state["grad"] = torch.randn(case["lines"], case["length"], width, generator=g, device="cuda").to(out)
    if case["op"] == "gradient":
        state["parts"] = [(_padded(torch.randn(count, width, generator=g, device="cuda").to(dtype), case["pad"]), _text(case, g, name_of))
                          for _ in range(case["parts"])]
    return state


def _prepare_rows(case, g):
    rows, n, dtype = case["rows"], case["n"], DTYPES[case["dtype"]]
    logits = torch.empty(rows, n, dtype=dtype, device="cuda")
    tokens = torch.empty(rows, dtype=torch.int64, device="cuda")
    step = max(1, (1 << 26) // n)
    for r in range(0, rows, step):
        m = min(step, rows - r)
        # some rows are sure of their next token, some are not
        x = torch.randn(m, n, generator=g, device="cuda") * (1.0 + 2.0 * torch.rand(m, 1, generator=g, device="cuda"))
        if case["op"] == "alternatives" and case["masked"]:  # tokens that a grammar rules out
            x[torch.rand(m, n, generator=g, device="cuda") < 0.3] = -INF
        logits[r:r + m] = x.to(dtype)
        # the given token is drawn from the row's own distribution, and now and then any
        noise = torch.rand(m, n, generator=g, device="cuda").clamp_min_(1e-30).log_().neg_().log_()
        tokens[r:r + m] = torch.argmax(x / case["temperature"] - noise, dim=1)
        anywhere = torch.randint(0, n, (m,), generator=g, device="cuda")
        tokens[r:r + m] = torch.where(torch.rand(m, generator=g, device="cuda") < 0.1, anywhere, tokens[r:r + m])
    if rows > 8:  # positions without a token to score
        tokens[torch.rand(rows, generator=g, device="cuda") < 0.03] = -1
    state = dict(case=case, logits=_padded(logits, case["pad"]), tokens=tokens if case["wide"] else tokens.int(), mask=None)
    if case["op"] == "alternatives":
        return state
    if case["masked"]:
        state["mask"] = torch.rand(rows, generator=g, device="cuda") < 0.85
    # the loss's derivatives: a mean over rows; half precision scales its loss so that gradients stay in range
    scale = (4096.0 if dtype == torch.float16 else 1.0) / rows
    state["up"] = -scale * (0.5 + torch.rand(rows, generator=g, device="cuda"))
    state["up_entropy"] = torch.full((rows,), -0.01 * scale, device="cuda") if case["entropy"] else None
    if case["call"] == "autograd":
        state["logits"] = state["logits"].detach().requires_grad_(True)
    return state


def prepare(case, seed):
    g = _generator(seed)
    return _prepare_embedding(case, g) if case["op"] in ("lookup", "gradient", "autograd") else _prepare_rows(case, g)


# -------------------------------------------------------------- plain forms

def _plain_lookup(s):
    c = s["case"]
    weight, tokens = s["weight"].detach(), s["tokens"].long()
    inside = (tokens >= 0) & (tokens < c["vocab"])
    rows = weight[torch.where(inside, tokens, torch.zeros_like(tokens))].float() * c["scale"]
    return torch.where(inside[..., None], rows, torch.zeros_like(rows)).to(DTYPES[c["out"]])


def _add_rows(total, grad, tokens, scale, skip):
    """The rows of grad added to the rows of total that their tokens name."""
    tokens = tokens.reshape(-1).long()
    kept = (tokens >= 0) & (tokens < total.shape[0]) & (tokens != skip)
    at = torch.where(kept, tokens, torch.zeros_like(tokens))
    grad = grad.reshape(-1, total.shape[1]).float() * scale
    return total.index_add_(0, at, torch.where(kept[:, None], grad, torch.zeros_like(grad)))


def _plain_embedding(s):
    c = s["case"]
    if c["op"] == "lookup":
        return {"rows": _plain_lookup(s)}
    total = torch.zeros(c["vocab"], c["width"], device="cuda")
    if c["op"] == "autograd":
        _add_rows(total, s["grad"], s["tokens"], c["scale"], s["padding"])
        return {"rows": _plain_lookup(s), "grad": total.to(s["weight"].dtype)}
    _add_rows(total, *s["parts"][0], c["scale"], -1)
    if c["parts"] == 2:
        _add_rows(total, *s["parts"][1], c["scale"], -1)
    return {"grad": total.to(DTYPES[c["out"]])}


def _image(x):
    """The ascending order-preserving integer image of a float tensor's bit patterns."""
    if x.dtype == torch.float32:
        b = x.contiguous().view(torch.int32)
        return b ^ ((b >> 31) & 0x7FFFFFFF)
    b = x.contiguous().view(torch.int16).to(torch.int32)
    return b ^ ((b >> 31) & 0x7FFF)


def _plain_rows(s):
    c, n = s["case"], s["case"]["n"]
    logits, t = s["logits"].detach(), c["temperature"]
    tokens = s["tokens"].long()
    given = (tokens >= 0) & (tokens < n)
    at = torch.where(given, tokens, torch.zeros_like(tokens))[:, None]
    z = logits.float() / t
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    z -= m
    e = torch.exp(z)
    # long sums, and differences of what nearly cancels: in 64 bits
    total = e.sum(dim=1, dtype=torch.float64)
    low = torch.log(total)
    mean = torch.where(e > 0, e * z, torch.zeros_like(z)).sum(dim=1, dtype=torch.float64) / total
    entropy = low - mean
    logprobs = torch.gather(z, 1, at)[:, 0].double() - low
    logprobs = torch.where(given, logprobs, torch.zeros_like(logprobs))
    if c["op"] == "alternatives":
        key = _image(logits)
        mine = torch.gather(key, 1, at)
        column = torch.arange(n, device=key.device)
        ranks = ((key > mine) | ((key == mine) & (column < at))).sum(dim=1)
        indices = torch.sort(~key, dim=1, stable=True)[1][:, :c["k"]].contiguous()
        top = torch.gather(z, 1, indices).double() - low[:, None]
        return {"logprobs": logprobs.float(), "entropy": entropy.float(),
                "ranks": torch.where(given, ranks, torch.full_like(ranks, -1)).int(), "top_logprobs": top.float(),
                "top_indices": indices}
    mask = s["mask"] if s["mask"] is not None else torch.ones_like(given)
    zero = torch.zeros_like(entropy)
    out = {"logprobs": torch.where(mask, logprobs, zero).float(), "entropy": torch.where(mask, entropy, zero).float()}
    if c["call"] == "forward":
        return out
    up = torch.where(given & mask, s["up"], torch.zeros_like(s["up"]))[:, None]
    p = e / total.float()[:, None]
    grad = -up * p
    if s["up_entropy"] is not None:
        down = torch.where(mask, s["up_entropy"], torch.zeros_like(s["up_entropy"]))[:, None]
        away = z - (low - entropy).float()[:, None]
        grad -= down * torch.where(p > 0, p * away, torch.zeros_like(p))
    grad.scatter_add_(1, at, up)
    out["grad"] = (grad / t).to(logits.dtype)
    return out


# --------------------------------------------------- this package's operators

def _own_embedding(s):
    import lsd_radix_sort_amd as lrs

    c = s["case"]
    out = DTYPES[c["out"]]
    if c["op"] == "lookup":
        return {"rows": lrs.embedding_forward(s["weight"], s["tokens"], scale=c["scale"], dtype=out)}
    if c["op"] == "autograd":
        rows = lrs.embedding_lookup(s["weight"], s["tokens"], scale=c["scale"], padding_index=s["padding"], dtype=out)
        grad, = torch.autograd.grad(rows, s["weight"], s["grad"])
        return {"rows": rows.detach(), "grad": grad}
    total = lrs.embedding_backward(*s["parts"][0], c["vocab"], scale=c["scale"], dtype=out)
    if c["parts"] == 2:
        lrs.embedding_backward(*s["parts"][1], c["vocab"], scale=c["scale"], grad_out=total, accumulate=True)
    return {"grad": total}


def _own_rows(s):
    import lsd_radix_sort_amd as lrs

    c = s["case"]
    logits, tokens = s["logits"], s["tokens"]
    if c["op"] == "alternatives":
        names = ("logprobs", "entropy", "ranks", "top_logprobs", "top_indices")
        return dict(zip(names, lrs.token_logprobs_topk(logits, tokens, c["k"], temperature=c["temperature"])))
    kw = dict(temperature=c["temperature"], row_mask=s["mask"])
    if c["call"] == "step":
        return dict(zip(("logprobs", "entropy", "grad"), lrs.token_logprobs_step(logits, tokens, s["up"], s["up_entropy"], **kw)))
    if c["call"] == "forward":
        return dict(zip(("logprobs", "entropy"), lrs.token_logprobs_forward(logits, tokens, **kw)))
    logprobs, entropy = lrs.token_logprobs(logits, tokens, **kw)
    if s["up_entropy"] is None:
        grad, = torch.autograd.grad(logprobs, logits, s["up"])
    else:
        grad, = torch.autograd.grad((logprobs, entropy), logits, (s["up"], s["up_entropy"]))
    return {"logprobs": logprobs.detach(), "entropy": entropy.detach(), "grad": grad}


def run(state):
    embedding = state["case"]["op"] in ("lookup", "gradient", "autograd")
    if own:
        return _own_embedding(state) if embedding else _own_rows(state)
    return _plain_embedding(state) if embedding else _plain_rows(state)


# ------------------------------------------------------------------ the work

def _distinct(vocab, tokens):
    """How many different ids a text of so many tokens is expected to hold."""
    i = torch.arange(vocab, dtype=torch.float64)
    p = (torch.log(i + 2.0) - torch.log(i + 1.0)) / math.log(vocab + 1.0)
    return float((1.0 - torch.exp(tokens * torch.log1p(-p))).sum())


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("lookup", "gradient", "autograd"):
        o, width, vocab = BYTES[case["out"]], case["width"], case["vocab"]
        tokens = case["lines"] * case["length"]
        ids = tokens * (8 if case["wide"] else 4)
        named = _distinct(vocab, tokens * (1.0 - case["dropped"])) * width
        kept = tokens * (1.0 - case["dropped"]) * width
        lookup = {"bytes": ids + named * e + tokens * width * o, "flops": tokens * width}
        if case["op"] == "lookup":
            return lookup
        if case["op"] == "autograd":
            return {"bytes": lookup["bytes"] + kept * o + vocab * width * e, "flops": lookup["flops"] + 2 * tokens * width}
        # later parts read and write the rows that they add to
        return {"bytes": case["parts"] * (ids + kept * e) + vocab * width * o + (case["parts"] - 1) * 2 * named * o,
                "flops": case["parts"] * 2 * kept}
    rows, n = case["rows"], case["n"]
    small = rows * ((8 if case["wide"] else 4) + 8)
    if case["op"] == "alternatives":
        return {"bytes": rows * n * e + small + rows * (4 + 12 * case["k"]), "flops": rows * n * 8}
    small += rows if case["masked"] else 0
    if case["call"] == "forward":
        return {"bytes": rows * n * e + small, "flops": rows * n * 6}
    return {"bytes": 2 * rows * n * e + small + rows * (8 if case["entropy"] else 4), "flops": rows * n * 12}


# ------------------------------------------------------- in 64 bits

def _exact_lookup(s):
    c = s["case"]
    tokens = s["tokens"].long()
    table = torch.zeros(c["vocab"] + 1, c["width"], dtype=torch.float64, device="cuda")  # the last row: no id
    table[:-1] = s["weight"].detach()
    table[:-1] *= c["scale"]
    return table[torch.where((tokens >= 0) & (tokens < c["vocab"]), tokens, torch.full_like(tokens, c["vocab"]))]


def _exact_embedding(s):
    c = s["case"]
    if c["op"] == "lookup":
        return {"rows": _exact_lookup(s)}
    table = torch.zeros(c["vocab"] + 1, c["width"], dtype=torch.float64, device="cuda")
    parts = s["parts"] if c["op"] == "gradient" else [(s["grad"], s["tokens"])]
    for grad, tokens in parts:
        tokens = tokens.flatten().long()
        outside = (tokens < 0) | (tokens >= c["vocab"])
        if c["op"] == "autograd":
            outside |= tokens == s["padding"]
        table.index_add_(0, tokens.masked_fill(outside, c["vocab"]), grad.reshape(-1, c["width"]).double())
    grad = table[:-1] * c["scale"]
    return {"grad": grad} if c["op"] == "gradient" else {"rows": _exact_lookup(s), "grad": grad}


def _exact_rows(s):
    c = s["case"]
    rows, n, t = c["rows"], c["n"], c["temperature"]
    parts = {}
    step = max(1, (1 << 26) // n)
    for r in range(0, rows, step):
        part = s["logits"][r:r + step].detach()
        m = part.shape[0]
        here = torch.arange(m, device="cuda")
        tokens = s["tokens"][r:r + step].long()
        given = (tokens >= 0) & (tokens < n)
        slot = tokens.masked_fill(~given, 0)
        logp = torch.log_softmax(part.double() / t, dim=1)
        p = torch.exp(logp)
        surprise = torch.where(p > 0, -logp, torch.zeros_like(logp))
        entropy = (p * surprise).sum(dim=1)
        logprobs = logp[here, slot].masked_fill(~given, 0.0)
        found = {}
        if c["op"] == "alternatives":
            bits = part.float().view(torch.int32).long()  # widening to 32 bits keeps the order and the signs
            rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
            # one whole number holds the order and, below it, the column: no two are alike
            both = rank * (1 << 31) + ((1 << 31) - 1 - torch.arange(n, device="cuda"))
            top = torch.topk(both, c["k"], dim=1)[0]
            indices = (1 << 31) - 1 - (top & ((1 << 31) - 1))
            place = (both > both[here, slot][:, None]).sum(dim=1).masked_fill(~given, -1)
            found.update(ranks=place.int(), top_logprobs=torch.gather(logp, 1, indices), top_indices=indices)
        else:
            mask = torch.ones_like(given) if s["mask"] is None else s["mask"][r:r + step]
            logprobs = logprobs.masked_fill(~mask, 0.0)
            if c["call"] != "forward":
                up = s["up"][r:r + step].double().masked_fill(~(given & mask), 0.0)
                grad = -up[:, None] * p
                grad[here, slot] += up
                if s["up_entropy"] is not None:
                    down = s["up_entropy"][r:r + step].double().masked_fill(~mask, 0.0)
                    grad += down[:, None] * p * (surprise - entropy[:, None])
                found["grad"] = grad / t
            entropy = entropy.masked_fill(~mask, 0.0)
        for name, value in dict(logprobs=logprobs, entropy=entropy, **found).items():
            parts.setdefault(name, []).append(value)
    return {name: torch.cat(values) for name, values in parts.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_embedding(s) if case["op"] in ("lookup", "gradient", "autograd") else _exact_rows(s)
