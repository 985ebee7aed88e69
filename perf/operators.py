"""The operators on the head of a sorted row and on counts of small keys, as workloads.

Three operators: `segmented_row_topk` (the first k columns of a row sort), the
distillation loss on a teacher's top logits with its gradient, and the per-expert
counts with the balance loss and its gradient.  `run` computes a case in plain
torch operations in 32 bits (`own` false) or with this package's entry points
(`own` true); `exact` computes it in 64 bits from the definition.
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
        # sampling: the candidates of one token from its logits (latency counts)
        dict(name="topk one token", op="topk", rows=1, n=131072, k=64, dtype="bf16", descending=True, pad=0, masked=True),
        # the teacher's top logits of a batch, at the row sort's own matrix shape
        dict(name="topk rows fp16", op="topk", rows=1024, n=65536, k=64, dtype="fp16", descending=True, pad=0, masked=False),
        # a router's choice of experts for a batch of tokens
        dict(name="topk router fp32", op="topk", rows=32768, n=256, k=8, dtype="fp32", descending=True, pad=0, masked=False),
        # the least likely tokens of ragged rows cut from a padded buffer
        dict(name="topk ragged ascending", op="topk", rows=333, n=50021, k=129, dtype="fp32", descending=False, pad=27, masked=False),
        # a training step: loss and gradient in one call, the teacher renormalised over its top logits
        dict(name="distill step bf16", op="distill", call="step", rows=4096, n=131072, k=64, dtype="bf16", tail=False,
             temperature=1.0, pad=0, weighted=False),
        # a training step over an odd vocabulary in a padded buffer, padding tokens, tail mass kept, softened
        dict(name="distill step tail odd", op="distill", call="step", rows=1031, n=50021, k=33, dtype="fp16", tail=True,
             temperature=2.0, pad=43, weighted=True),
        # evaluation: the loss alone, at the row sort's own matrix shape
        dict(name="distill forward tail", op="distill", call="forward", rows=1024, n=65536, k=32, dtype="fp16", tail=True,
             temperature=1.0, pad=0, weighted=False),
        # the loss inside a differentiated program: forward, then backward through autograd
        dict(name="distill autograd fp32", op="distill", call="autograd", rows=515, n=32768, k=16, dtype="fp32", tail=False,
             temperature=1.0, pad=0, weighted=True),
        # the smallest step: the last tokens of a few sequences
        dict(name="distill few rows", op="distill", call="step", rows=4, n=32000, k=8, dtype="bf16", tail=False,
             temperature=1.0, pad=0, weighted=False),
        # a training step's router loss over a large batch
        dict(name="balance step bf16", op="balance", call="step", rows=65536, n=256, k=8, dtype="bf16", score="softmax",
             z=1e-3, masked=False, wide=True),
        # normalised sigmoid scores, padding tokens, through autograd
        dict(name="balance sigmoid autograd", op="balance", call="autograd", rows=30011, n=160, k=6, dtype="fp32",
             score="sigmoid", z=0.0, masked=True, wide=True),
        # the smallest: counts and loss of one decoded batch
        dict(name="balance few tokens", op="balance", call="forward", rows=64, n=64, k=2, dtype="bf16", score="softmax",
             z=1e-3, masked=False, wide=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["topk", "distill", "balance"])
    dtype = rng.choice(["fp16", "bf16", "fp32"])
    if op == "topk":
        if rng.random() < 0.35:  # router-like rows
            n = _log(rng, 8, 512)
            rows = _log(rng, 1, 65536)
            k = _log(rng, 1, min(n, 16))
        else:
            n = _log(rng, 513, 131072)
            rows = _log(rng, 1, min(4096, (1 << 26) // n))
            k = _log(rng, 1, min(n, 256))
        return dict(op=op, rows=rows, n=n, k=k, dtype=dtype, descending=rng.random() < 0.7,
                    pad=rng.choice([0, 0, 8, rng.randint(1, 63)]), masked=rng.random() < 0.3)
    if op == "distill":
        n = _log(rng, 500, 131072)
        rows = _log(rng, 1, min(8192, (1 << 27) // n))
        return dict(op=op, call=rng.choice(["step", "step", "forward", "autograd"]), rows=rows, n=n,
                    k=_log(rng, 1, 128), dtype=dtype, tail=rng.random() < 0.5,
                    temperature=rng.choice([1.0, 1.0, 0.7, 2.0, 4.0]), pad=rng.choice([0, 0, 8, rng.randint(1, 63)]),
                    weighted=rng.random() < 0.5)
    n = _log(rng, 8, 512)
    rows = _log(rng, 1, 65536)
    score = rng.choice(["softmax", "softmax", "sigmoid"])
    return dict(op=op, call=rng.choice(["step", "step", "forward", "autograd"]), rows=rows, n=n,
                k=_log(rng, 1, min(n, 16)), dtype=dtype, score=score, z=rng.choice([0.0, 1e-3]) if score == "softmax" else 0.0,
                masked=rng.random() < 0.5, wide=rng.random() < 0.5)


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


def prepare(case, seed):
    g = _generator(seed)
    rows, n, k, dtype = case["rows"], case["n"], case["k"], DTYPES[case["dtype"]]
    state = dict(case=case)
    if case["op"] == "topk":
        x = torch.randn(rows, n, generator=g, device="cuda") * 2.5
        if case["masked"]:  # tokens a grammar rules out
            x[torch.rand(rows, n, generator=g, device="cuda") < 0.3] = -INF
        state["x"] = _padded(x.to(dtype), case["pad"])
        return state
    if case["op"] == "distill":
        logits = torch.empty(rows, n, dtype=dtype, device="cuda")
        values = torch.empty(rows, k, device="cuda")
        indices = torch.empty(rows, k, dtype=torch.int64, device="cuda")
        lse = torch.empty(rows, device="cuda")
        t = case["temperature"]
        step = max(1, (1 << 26) // n)
        for r in range(0, rows, step):
            m = min(step, rows - r)
            teacher = torch.randn(m, n, generator=g, device="cuda") * 2.5
            values[r:r + m], indices[r:r + m] = torch.topk(teacher, k, dim=1)
            lse[r:r + m] = torch.logsumexp(teacher.double() / t, dim=1).float()
            # a student that has learned part of what the teacher knows
            logits[r:r + m] = (0.7 * teacher + 1.5 * torch.randn(m, n, generator=g, device="cuda")).to(dtype)
        if k > 2:  # a few rows for which the teacher stored fewer logits
            short = torch.rand(rows, generator=g, device="cuda") < 0.05
            indices[short, k - 1] = -1
        state.update(logits=_padded(logits, case["pad"]), values=values.to(dtype), indices=indices,
                     lse=lse if case["tail"] else None)
        # the mean over rows; half precision scales its loss so that gradients stay in range
        weights = torch.full((rows,), (4096.0 if dtype == torch.float16 else 1.0) / rows, device="cuda")
        if case["weighted"]:  # padding tokens weigh nothing
            weights = (torch.rand(rows, generator=g, device="cuda") < 0.8).float() * weights
        state["weights"] = weights
        if case["call"] == "autograd":
            state["logits"] = state["logits"].detach().requires_grad_(True)
        return state
    # router logits with a preference for some experts, so that the load is uneven
    x = torch.randn(rows, n, generator=g, device="cuda") * 1.5 + torch.randn(n, generator=g, device="cuda") * 0.5
    x = x.to(dtype)
    indices = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :k].contiguous()
    dropped = torch.rand(rows, generator=g, device="cuda") < 0.02  # over capacity
    indices[dropped, k - 1] = -1
    state.update(logits=x, indices=indices if case["wide"] else indices.int(), mask=None)
    if case["masked"]:
        state["mask"] = torch.rand(rows, generator=g, device="cuda") < 0.85
    if case["call"] == "autograd":
        state["logits"] = state["logits"].detach().requires_grad_(True)
    return state


def _coefficients(case):
    """The loss's coefficients; half precision scales its loss so that gradients stay in range."""
    scale = 65536.0 if case["dtype"] == "fp16" else 1.0
    return 0.01 * scale, case["z"] * scale


# -------------------------------------------------------------- plain forms

def _image(x):
    """The ascending order-preserving integer image of a float tensor's bit patterns."""
    if x.dtype == torch.float32:
        b = x.contiguous().view(torch.int32)
        return b ^ ((b >> 31) & 0x7FFFFFFF)
    b = x.contiguous().view(torch.int16).to(torch.int32)
    return b ^ ((b >> 31) & 0x7FFF)


def _plain_topk(s):
    c, x = s["case"], s["x"]
    key = _image(x)
    if c["descending"]:
        key = ~key
    indices = torch.sort(key, dim=1, stable=True)[1][:, :c["k"]].contiguous()
    return {"values": torch.gather(x, 1, indices), "indices": indices}


def _lse(z):
    """log sum exp of each row, summed in 64 bits (it is a long sum, and what is left
    of two such logarithms may be small); -inf for a row without mass."""
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    return m.squeeze(1).double() + torch.log(torch.exp(z - m).sum(dim=1, dtype=torch.float64))


def _plain_distill(s):
    c = s["case"]
    t, rows, n = c["temperature"], c["rows"], c["n"]
    logits = s["logits"].detach()
    z = logits.float() / t
    counted = (s["indices"] >= 0) & (s["indices"] < n) & (s["values"].float() > -INF)
    at = torch.where(counted, s["indices"], torch.zeros_like(s["indices"]))
    # what there is once a row or a slot stays in 64 bits: the terms of a loss
    # nearly cancel, and 1 - sum q loses what a small tail holds
    tv = torch.where(counted, s["values"].double() / t, torch.full_like(s["values"].double(), -INF))
    zt = torch.gather(logits, 1, at).double() / t
    lse = _lse(z)
    q0 = None
    if c["tail"]:
        q = torch.exp(tv - s["lse"].double()[:, None])
        q0 = (1.0 - q.sum(dim=1)).clamp_min(0.0)
        rest = z.clone()
        r, j = torch.nonzero(counted, as_tuple=True)
        rest[r, at[r, j]] = -INF
        lse0 = _lse(rest)
        q0 = torch.where(counted.sum(dim=1) == n, torch.zeros_like(q0), q0)
        q0 = torch.where((lse0 == -INF) & (q0 <= 2.0 ** -20), torch.zeros_like(q0), q0)
    else:
        q = torch.exp(tv - _lse(tv)[:, None])
        q = torch.where(counted, q, torch.zeros_like(q))
    part = torch.where(q > 0, q * (torch.log(q) - (zt - lse[:, None])), torch.zeros_like(q))
    row_loss = part.sum(dim=1)
    if q0 is not None:
        row_loss = row_loss + torch.where(q0 > 0, q0 * (torch.log(q0) - (lse0 - lse)), torch.zeros_like(q0))
    w = s["weights"]
    row_loss = torch.where(w == 0, torch.zeros_like(row_loss), row_loss)
    out = {"loss": (w.double() * row_loss).sum().float(), "row_loss": row_loss.float()}
    if c["call"] == "forward":
        return out
    a = q.sum(dim=1)
    if q0 is not None:
        a = a + q0
    lse32 = lse.float()[:, None]
    top = a[:, None] * torch.exp(zt - lse[:, None]) - q
    grad = torch.exp(z - lse32)
    if q0 is None:
        grad *= a.float()[:, None]
    else:
        grad -= q0.float()[:, None] * torch.exp(z - lse0.float()[:, None])
    r, j = torch.nonzero(counted, as_tuple=True)
    grad[r, at[r, j]] = top[r, j].float()
    grad *= (w / t)[:, None]
    out["grad"] = grad.to(logits.dtype)
    return {"loss": out["loss"], "grad": out["grad"]} if c["call"] == "autograd" else out


def _plain_balance(s):
    c = s["case"]
    alpha, beta = _coefficients(c)
    rows, n = c["rows"], c["n"]
    logits = s["logits"].detach()
    x = logits.float()
    mask = s["mask"] if s["mask"] is not None else torch.ones(rows, dtype=torch.bool, device=x.device)
    idx = s["indices"]
    keep = (idx >= 0) & (idx < n) & mask[:, None]
    counts = torch.bincount(idx[keep].long(), minlength=n)
    total = counts.sum()
    f = torch.where(total > 0, n * counts.float() / total.clamp_min(1).float(), torch.zeros_like(counts, dtype=torch.float32))
    kept = mask.sum().float()
    inv = torch.where(kept > 0, 1.0 / kept.clamp_min(1.0), torch.zeros_like(kept))
    if c["score"] == "softmax":
        lse = _lse(x).float()
        p = torch.exp(x - lse[:, None])
    else:
        sig = 1.0 / (1.0 + torch.exp(-x))
        p = sig / sig.sum(dim=1, keepdim=True)
    b = (p * f).sum(dim=1)
    row = alpha * b
    if beta:
        row = row + beta * lse * lse
    out = {"loss": torch.where(mask, row, torch.zeros_like(row)).sum(dtype=torch.float64).float() * inv, "counts": counts.int()}
    if c["call"] == "forward":
        return out
    if c["score"] == "softmax":
        d = alpha * (f - b[:, None])
        if beta:
            d = d + 2.0 * beta * lse[:, None]
        grad = p * d * inv
    else:
        grad = alpha * p * (1.0 - sig) * (f - b[:, None]) * inv
    out["grad"] = torch.where(mask[:, None], grad, torch.zeros_like(grad)).to(logits.dtype)
    return out


# --------------------------------------------------- this package's operators

def _own(s):
    import lsd_radix_sort_amd as lrs

    c = s["case"]
    if c["op"] == "topk":
        values, indices = lrs.segmented_row_topk(s["x"], c["k"], descending=c["descending"])
        return {"values": values, "indices": indices}
    if c["op"] == "distill":
        args = (s["logits"], s["values"], s["indices"])
        kw = dict(temperature=c["temperature"], teacher_lse=s["lse"], row_weights=s["weights"])
        if c["call"] == "autograd":
            loss = lrs.topk_distill_loss(*args, **kw)
            grad, = torch.autograd.grad(loss, s["logits"])
            return {"loss": loss.detach(), "grad": grad}
        if c["call"] == "forward":
            loss, row_loss, _ = lrs.topk_distill_forward(*args, **kw)
            return {"loss": loss, "row_loss": row_loss}
        loss, row_loss, grad = lrs.topk_distill_step(*args, **kw)
        return {"loss": loss, "row_loss": row_loss, "grad": grad}
    args = (s["logits"], s["indices"])
    alpha, beta = _coefficients(c)
    kw = dict(balance_weight=alpha, z_weight=beta, score=c["score"], row_mask=s["mask"])
    if c["call"] == "autograd":
        loss, counts = lrs.expert_balance_loss(*args, **kw)
        grad, = torch.autograd.grad(loss, s["logits"])
        return {"loss": loss.detach(), "counts": counts, "grad": grad}
    if c["call"] == "forward":
        loss, counts, _ = lrs.expert_balance_forward(*args, **kw)
        return {"loss": loss, "counts": counts}
    loss, counts, grad = lrs.expert_balance_step(*args, **kw)
    return {"loss": loss, "counts": counts, "grad": grad}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_topk(state) if op == "topk" else _plain_distill(state) if op == "distill" else _plain_balance(state)


# ------------------------------------------------------------------ the work

def work(case):
    rows, n, k, e = case["rows"], case["n"], case["k"], BYTES[case["dtype"]]
    if case["op"] == "topk":
        return {"bytes": rows * n * e + rows * k * (e + 8), "flops": 2 * rows * n}
    gradient = case["call"] != "forward"
    if case["op"] == "distill":
        small = rows * k * (e + 8) + rows * 4 + (rows * 4 if case["tail"] else 0)
        outs = 4 if case["call"] == "autograd" else rows * 4 + 4
        return {"bytes": rows * n * e * (2 if gradient else 1) + small + outs, "flops": rows * n * (8 if gradient else 4)}
    small = rows * k * (8 if case["wide"] else 4) + n * 4 + 4 + (rows if case["masked"] else 0)
    return {"bytes": rows * n * e * (2 if gradient else 1) + small, "flops": rows * n * (12 if gradient else 6)}


# ------------------------------------------------------- in 64 bits

def _exact_topk(s):
    c, x = s["case"], s["x"]
    rows, n, k = c["rows"], c["n"], c["k"]
    values = torch.empty(rows, k, dtype=torch.float64, device="cuda")
    indices = torch.empty(rows, k, dtype=torch.int64, device="cuda")
    column = torch.arange(n, device="cuda")
    step = max(1, (1 << 24) // n)
    for r in range(0, rows, step):
        part = x[r:r + step]
        bits = part.float().view(torch.int32).long()  # widening to 32 bits keeps the order and the signs
        rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
        if not c["descending"]:
            rank = -1 - rank
        # one whole number holds the order and, below it, the column: no two are alike
        both = rank * (1 << 31) + ((1 << 31) - 1 - column)
        top = torch.topk(both, k, dim=1)[0]
        at = (1 << 31) - 1 - (top & ((1 << 31) - 1))
        indices[r:r + step] = at
        values[r:r + step] = torch.gather(part, 1, at).double()
    return {"values": values, "indices": indices}


def _exact_distill(s):
    c = s["case"]
    t, rows, n, k = c["temperature"], c["rows"], c["n"], c["k"]
    row_loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    full = c["call"] != "forward"
    grad = torch.zeros(rows, n, dtype=torch.float64, device="cuda") if full else None
    weights = s["weights"].double()
    step = max(1, (1 << 26) // n)
    for r in range(0, rows, step):
        u = s["logits"][r:r + step].detach().double() / t
        m = u.shape[0]
        idx, tv = s["indices"][r:r + step], s["values"][r:r + step].double() / t
        ok = (idx >= 0) & (idx < n)
        # the teacher's mass spread over the columns
        target = torch.zeros(m, n + 1, dtype=torch.float64, device="cuda")
        member = torch.zeros(m, n + 1, dtype=torch.bool, device="cuda")
        slot = torch.where(ok, idx, torch.full_like(idx, n))
        if c["tail"]:
            mass = torch.exp(tv - s["lse"][r:r + step].double()[:, None]) * ok
        else:
            mass = torch.softmax(torch.where(ok, tv, torch.full_like(tv, -INF)), dim=1)
            mass = torch.nan_to_num(mass, nan=0.0)
        target.scatter_add_(1, slot, mass)
        member.scatter_(1, slot, True)
        target, member = target[:, :n], member[:, :n]
        logp = torch.log_softmax(u, dim=1)
        kl = torch.special.xlogy(target, target).sum(1) - torch.where(target > 0, target * logp, torch.zeros_like(logp)).sum(1)
        p = torch.exp(logp)
        if c["tail"]:
            q0 = (1.0 - target.sum(1)).clamp_min(0.0) * (~member).any(1)
            logp0 = torch.logsumexp(torch.where(member, torch.full_like(logp, -INF), logp), dim=1)
            kl = kl + torch.special.xlogy(q0, q0) - torch.where(q0 > 0, q0 * logp0, torch.zeros_like(q0))
            d = torch.where(member, p - target, p - q0[:, None] * torch.exp(logp - logp0[:, None]))
        else:
            d = target.sum(1, keepdim=True) * p - target
        w = weights[r:r + step]
        row_loss[r:r + step] = torch.where(w == 0, torch.zeros_like(kl), kl)
        if full:
            grad[r:r + step] = d * (w / t)[:, None]
    out = {"loss": (weights * row_loss).sum()}
    if c["call"] != "autograd":
        out["row_loss"] = row_loss
    if full:
        out["grad"] = grad
    return out


def _exact_balance(s):
    c = s["case"]
    alpha, beta = _coefficients(c)
    rows, n = c["rows"], c["n"]
    x = s["logits"].detach().double().requires_grad_(c["call"] != "forward")
    mask = torch.ones(rows, device="cuda", dtype=torch.bool) if s["mask"] is None else s["mask"]
    idx = s["indices"].long()
    idx = torch.where((idx >= 0) & (idx < n) & mask[:, None], idx, torch.full_like(idx, n))
    counts = torch.zeros(n + 1, dtype=torch.int64, device="cuda").scatter_add_(0, idx.flatten(), torch.ones_like(idx).flatten())[:n]
    load = counts.double() * n / max(int(counts.sum()), 1)
    if c["score"] == "softmax":
        p = torch.softmax(x, dim=1)
    else:
        p = torch.sigmoid(x)
        p = p / p.sum(dim=1, keepdim=True)
    row = alpha * (p @ load)
    if beta:
        row = row + beta * torch.logsumexp(x, dim=1) ** 2
    loss = row[mask].sum() / max(int(mask.sum()), 1)
    out = {"loss": loss.detach(), "counts": counts.int()}
    if c["call"] != "forward":
        out["grad"] = torch.autograd.grad(loss, x)[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_topk(s) if case["op"] == "topk" else _exact_distill(s) if case["op"] == "distill" else _exact_balance(s)
