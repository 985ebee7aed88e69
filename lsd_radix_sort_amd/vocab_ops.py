"""Operators at the two ends of a language model's vocabulary.

    embedding_forward / _backward / embedding_lookup(weight, tokens, ...)
    token_logprobs_forward / _backward / _step / token_logprobs(logits, tokens, ...)
    token_logprobs_topk(logits, tokens, k, ...)

The entry points of the C ABI (include/lsd_radix_sort.h), with the checks,
streams, outputs and errors of the package's sorts.  Regular calls go through
the compiled binding, as in row_ops.  The table's gradient is a
stable sort of the tokens' ids and a sum over equal ones; a
token's rank and the top alternatives are places in the descending row sort.
embedding_lookup and token_logprobs differentiate through torch autograd; the
other calls do not record a graph.
"""
from __future__ import annotations

import ctypes
import math

import torch

import lsd_radix_sort_amd as _lrs
from . import row_ops as _rows
from .row_ops import _ID_BYTES, _dtype_code, _grad_out, _mask, _matrix, _whole


_MAX_TOPK = 1024  # LRS_MAX_TOPK


class _TokenIds(ctypes.Structure):
    # mirrors struct lrs_token_ids
    _fields_ = [("ids", ctypes.c_void_p), ("lines", ctypes.c_int64), ("length", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("id_bytes", ctypes.c_int)]


class _Logprobs(ctypes.Structure):
    # mirrors struct lrs_logprobs
    _fields_ = [("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("tokens", ctypes.c_void_p),
                ("token_stride", ctypes.c_int64), ("token_bytes", ctypes.c_int), ("dtype", ctypes.c_int),
                ("row_mask", ctypes.c_void_p), ("rows", ctypes.c_int64), ("n", ctypes.c_int64),
                ("temperature", ctypes.c_double)]


# ---------------------------------------------------------------- embedding

def _token_ids(tokens, device) -> _TokenIds:
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda:
        _lrs._bad("tokens must be a GPU tensor")
    _lrs._same_device(tokens, "tokens", device)
    size = _ID_BYTES.get(tokens.dtype)
    if size is None:
        _lrs._bad(f"tokens must be int32 or int64, got {tokens.dtype}")
    if tokens.is_contiguous():
        lines, length, stride = 1, tokens.numel(), 0
    elif tokens.dim() == 1:
        lines, length, stride = tokens.size(0), 1, tokens.stride(0)
    elif tokens.dim() == 2 and (tokens.stride(1) == 1 or tokens.size(1) <= 1):
        (lines, length), stride = tokens.shape, tokens.stride(0)
    else:
        _lrs._bad("tokens must be contiguous, 1-D, or 2-D with contiguous rows")
    return _TokenIds(tokens.data_ptr(), lines, length, stride, size)


def _rows_of(t, name: str, tokens, width: int, device) -> int:
    """Checks a [*tokens.shape, width] tensor whose rows are contiguous and lie evenly apart; returns their stride."""
    _lrs._same_device(t, name, device)
    _dtype_code(t.dtype, name)
    if t.dim() == 0 or t.size(-1) != width or (t.shape[:-1] != tokens.shape and t.shape[:-1] != (tokens.numel(),)):
        _lrs._bad(f"{name} must have shape {(*tokens.shape, width)}, got {tuple(t.shape)}")
    try:
        rows = t.detach().view(tokens.numel(), width)
    except RuntimeError:
        rows = None
    if rows is None or (width > 1 and rows.stride(1) != 1):
        _lrs._bad(f"{name} must have contiguous rows that lie evenly apart")
    return rows.stride(0)


def _number(v, name: str) -> float:
    try:
        return float(v)
    except (TypeError, ValueError, OverflowError):
        _lrs._bad(f"{name} must be a number, got {v!r}")


def _finite(scale) -> float:
    scale = _number(scale, "scale")
    if not math.isfinite(ctypes.c_float(scale).value):
        _lrs._bad(f"scale must be finite in 32 bits, got {scale}")
    return scale


def embedding_forward(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, dtype: torch.dtype | None = None,
                      out: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None) -> torch.Tensor:
    """Rows of a [vocab, width] table times scale: [*tokens.shape, width] of `dtype` (the table's), 0 for tokens
    outside [0, vocab).  tokens: int32 or int64, contiguous, 1-D with any stride, or 2-D with contiguous rows."""
    if out is None and options is None:
        fast = (_rows._fast or _rows._binding()).embedding_forward(weight, tokens, _finite(scale), dtype)
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    code = _matrix(weight, "weight")
    vocab, width = weight.shape
    ids = _token_ids(tokens, weight.device)
    scale = _finite(scale)
    if out is None:
        out_code = _dtype_code(weight.dtype if dtype is None else dtype, "dtype")
        out = torch.empty((*tokens.shape, width), dtype=weight.dtype if dtype is None else dtype, device=weight.device)
        stride = width
    else:
        if dtype is not None and isinstance(out, torch.Tensor) and out.dtype != dtype:
            _lrs._bad(f"out is {out.dtype}, dtype {dtype}")
        stride = _rows_of(out, "out", tokens, width, weight.device)
        out_code = _dtype_code(out.dtype, "out")
    with torch.cuda.device(weight.device):
        _lrs._check(lib.embedding_forward(weight.data_ptr(), weight.stride(0), ctypes.byref(ids), out.data_ptr(), stride, vocab,
                                          width, code, out_code, scale, _lrs._stream(weight), _lrs._opt(options)),
                    "embedding_forward")
    return out


def embedding_backward_workspace_size(tokens: int, vocab: int, width: int, options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().embedding_backward_workspace_size(tokens, vocab, width, _lrs._opt(options)))


def embedding_backward(grad: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                       padding_index: int | None = None, dtype: torch.dtype | None = None,
                       grad_out: torch.Tensor | None = None, accumulate: bool = False,
                       workspace: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None) -> torch.Tensor:
    """The gradient of embedding_forward's table from that of its output: [vocab, width] of `dtype` (grad's).

    grad: [*tokens.shape, width] or [tokens.numel(), width].  Tokens outside [0, vocab) and those equal to
    padding_index count for nothing.  accumulate: the gradient is added to grad_out, whose rows without a token
    stay as they are.  The sums are in 32 bits, in an order that the ids and sizes alone decide: equal calls
    give equal bits."""
    vocab = _whole(vocab, "vocab")
    if not 0 <= vocab < 2 ** 31 - 1:
        _lrs._bad(f"vocab must be in [0, 2^31 - 1), got {vocab}")
    if workspace is None and options is None:
        fast = (_rows._fast or _rows._binding()).embedding_backward(grad, tokens, vocab, _finite(scale), padding_index, dtype,
                                                                    grad_out, bool(accumulate))
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda:
        _lrs._bad("grad must be a GPU tensor")
    device = grad.device
    ids = _token_ids(tokens, device)
    if grad.dim() == 0:
        _lrs._bad("grad must have a last dimension, the table's width")
    width = grad.size(-1)
    stride = _rows_of(grad, "grad", tokens, width, device)
    code = _dtype_code(grad.dtype, "grad")
    scale = _finite(scale)
    padding = -1
    if padding_index is not None:
        padding = _whole(padding_index, "padding_index")
        if not 0 <= padding < vocab:
            _lrs._bad(f"padding_index must be in [0, {vocab}), got {padding}")
    if grad_out is None:
        if accumulate:
            _lrs._bad("accumulate needs the grad_out to add to")
        dtype = grad.dtype if dtype is None else dtype
        _dtype_code(dtype, "dtype")
        grad_out = torch.empty((vocab, width), dtype=dtype, device=device)
    else:
        _lrs._same_device(grad_out, "grad_out", device)
        if _matrix(grad_out, "grad_out") is not None and grad_out.shape != (vocab, width):
            _lrs._bad(f"grad_out must have shape {(vocab, width)}, got {tuple(grad_out.shape)}")
        if dtype is not None and grad_out.dtype != dtype:
            _lrs._bad(f"grad_out is {grad_out.dtype}, dtype {dtype}")
    opt = _lrs._opt(options)
    need = lib.embedding_backward_workspace_size(tokens.numel(), vocab, width, opt)
    with torch.cuda.device(device):
        workspace = _lrs._workspace(workspace, need, device)
        _lrs._check(lib.embedding_backward(grad.data_ptr(), stride, ctypes.byref(ids), grad_out.data_ptr(), grad_out.stride(0),
                                           vocab, width, code, _dtype_code(grad_out.dtype, "grad_out"), scale, padding,
                                           int(bool(accumulate)), workspace.data_ptr(), workspace.numel(),
                                           _lrs._stream(grad), opt), "embedding_backward")
    return grad_out


def embedding_lookup(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, padding_index: int | None = None,
                     dtype: torch.dtype | None = None) -> torch.Tensor:
    """embedding_forward, differentiable in the table; rows of padding_index get no gradient.

    Inside a graph capture use embedding_forward and embedding_backward: a backward pass of torch's autograd may
    wait there for streams of graphs that were built outside it."""
    if padding_index is not None:
        padding_index = _whole(padding_index, "padding_index")
        if isinstance(weight, torch.Tensor) and weight.dim() == 2 and not 0 <= padding_index < weight.size(0):
            _lrs._bad(f"padding_index must be in [0, {weight.size(0)}), got {padding_index}")
    out = (_rows._fast or _rows._binding()).embedding_lookup(weight, tokens, _finite(scale), padding_index, dtype)
    if out is None:
        embedding_forward(weight, tokens, scale, dtype)  # says what is wrong
        _lrs._bad("embedding_lookup does not take these arguments")
    return out


# --------------------------------------- log probabilities of given tokens

def _logprob_inputs(logits, tokens, temperature, row_mask=None) -> _Logprobs:
    dtype = _matrix(logits, "logits")
    rows, n = logits.shape
    _lrs._same_device(tokens, "tokens", logits.device)
    size = _ID_BYTES.get(tokens.dtype)
    if size is None:
        _lrs._bad(f"tokens must be int32 or int64, got {tokens.dtype}")
    if tokens.dim() != 1 or tokens.size(0) != rows:
        _lrs._bad(f"tokens must be a 1-D tensor of {rows} tokens, got {tuple(tokens.shape)}")
    return _Logprobs(logits.data_ptr(), logits.stride(0), tokens.data_ptr(), tokens.stride(0), size, dtype,
                     _mask(row_mask, rows, logits.device), rows, n, _number(temperature, "temperature"))


def _by_row(t, name: str, rows: int, device) -> int | None:
    if t is None:
        return None
    _lrs._same_device(t, name, device)
    if t.dtype != torch.float32 or t.shape != (rows,) or not t.is_contiguous():
        _lrs._bad(f"{name} must be a contiguous float32 tensor of shape ({rows},)")
    return t.data_ptr()


def token_logprobs_workspace_size(rows: int, n: int, k: int = 0, dtype: torch.dtype = torch.bfloat16,
                                  options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().token_logprobs_workspace_size(rows, n, k, _dtype_code(dtype, "dtype"), _lrs._opt(options)))


def _logprob_workspace(lib, workspace, d: _Logprobs, k: int, opt, device) -> torch.Tensor:
    return _lrs._workspace(workspace, lib.token_logprobs_workspace_size(d.rows, d.n, k, d.dtype, opt), device)


def token_logprobs_forward(logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0,
                           row_mask: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                           options: "_lrs.SortOptions | None" = None):
    """Log probabilities of one given token a row, and the rows' entropy, of logits [rows, n] / temperature.

    A token outside [0, n), such as -1, has log probability 0; rows whose row_mask is not set have entropy 0, too.
    Returns (logprobs [rows] float32, entropy [rows] float32, row_stats for the backward)."""
    if workspace is None and options is None:
        fast = (_rows._fast or _rows._binding()).logprobs_forward(logits, tokens, _number(temperature, "temperature"), row_mask)
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    d = _logprob_inputs(logits, tokens, temperature, row_mask)
    opt = _lrs._opt(options)
    device = logits.device
    with torch.cuda.device(device):
        workspace = _logprob_workspace(lib, workspace, d, 0, opt, device)
        logprobs, entropy = (torch.empty(d.rows, dtype=torch.float32, device=device) for _ in range(2))
        stats = torch.empty((d.rows, 3), dtype=torch.float32, device=device)
        _lrs._check(lib.token_logprobs_forward(ctypes.byref(d), logprobs.data_ptr(), entropy.data_ptr(), stats.data_ptr(),
                                               workspace.data_ptr(), workspace.numel(), _lrs._stream(logits), opt),
                    "token_logprobs_forward")
    return logprobs, entropy, stats


def token_logprobs_topk(logits: torch.Tensor, tokens: torch.Tensor, k: int, temperature: float = 1.0,
                        workspace: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """token_logprobs_forward's values, up to their last bits (the sums are taken in another order), with the tokens'
    ranks (0: the likeliest) and the k likeliest alternatives.

    Ranks and alternatives are places in the row's descending stable sort, so top_indices[r, ranks[r]] is the
    token where ranks[r] < k; a token outside [0, n) has rank -1.
    Returns (logprobs, entropy, ranks [rows] int32, top_logprobs [rows, k] float32, top_indices [rows, k] int64)."""
    k = _whole(k, "k")
    if not 0 <= k <= _MAX_TOPK:
        _lrs._bad(f"k must be between 0 and {_MAX_TOPK}, got {k}")
    if workspace is None and options is None:
        fast = (_rows._fast or _rows._binding()).logprobs_topk(logits, tokens, k, _number(temperature, "temperature"))
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    d = _logprob_inputs(logits, tokens, temperature)
    if not 0 <= k <= d.n:
        _lrs._bad(f"k must be between 0 and the row length {d.n}, got {k}")
    opt = _lrs._opt(options)
    device = logits.device
    with torch.cuda.device(device):
        workspace = _logprob_workspace(lib, workspace, d, k, opt, device)
        logprobs, entropy = (torch.empty(d.rows, dtype=torch.float32, device=device) for _ in range(2))
        ranks = torch.empty(d.rows, dtype=torch.int32, device=device)
        top = torch.empty((d.rows, k), dtype=torch.float32, device=device)
        indices = torch.empty((d.rows, k), dtype=torch.int64, device=device)
        _lrs._check(lib.token_logprobs_topk(ctypes.byref(d), k, logprobs.data_ptr(), entropy.data_ptr(), ranks.data_ptr(),
                                            top.data_ptr(), indices.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                            _lrs._stream(logits), opt), "token_logprobs_topk")
    return logprobs, entropy, ranks, top, indices


def _derivatives(logprob_grad, entropy_grad, d: _Logprobs, device):
    if logprob_grad is None and entropy_grad is None:
        _lrs._bad("one of logprob_grad and entropy_grad must be given")
    return _by_row(logprob_grad, "logprob_grad", d.rows, device), _by_row(entropy_grad, "entropy_grad", d.rows, device)


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, row_stats: torch.Tensor,
                            logprob_grad: torch.Tensor | None, entropy_grad: torch.Tensor | None = None,
                            temperature: float = 1.0, row_mask: torch.Tensor | None = None,
                            grad_out: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None) -> torch.Tensor:
    """The gradient in the logits of a loss whose derivatives in token_logprobs_forward's log probabilities and
    entropies are logprob_grad and entropy_grad ([rows] float32, None: 0), from the same inputs and the row_stats
    that the forward returned."""
    if grad_out is None and options is None:
        fast = (_rows._fast or _rows._binding()).logprobs_backward(logits, tokens, row_stats, logprob_grad, entropy_grad,
                                                                   _number(temperature, "temperature"), row_mask)
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    d = _logprob_inputs(logits, tokens, temperature, row_mask)
    device = logits.device
    _lrs.check_output(row_stats, "row_stats", device, 4, (d.rows, 3))
    if row_stats.dtype != torch.float32:
        _lrs._bad("row_stats must be float32, as token_logprobs_forward returned them")
    up, up_entropy = _derivatives(logprob_grad, entropy_grad, d, device)
    with torch.cuda.device(device):
        grad_out = _grad_out(grad_out, logits)
        _lrs._check(lib.token_logprobs_backward(ctypes.byref(d), row_stats.data_ptr(), up, up_entropy, grad_out.data_ptr(),
                                                grad_out.stride(0), _lrs._stream(logits), _lrs._opt(options)),
                    "token_logprobs_backward")
    return grad_out


def token_logprobs_step(logits: torch.Tensor, tokens: torch.Tensor, logprob_grad: torch.Tensor | None,
                        entropy_grad: torch.Tensor | None = None, temperature: float = 1.0,
                        row_mask: torch.Tensor | None = None, grad_out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """token_logprobs_forward and _backward in one call, for derivatives that are known beforehand (such as those of
    a weighted sum of log probabilities): returns (logprobs, entropy, grad), the first two up to their last bits."""
    if grad_out is None and workspace is None and options is None:
        fast = (_rows._fast or _rows._binding()).logprobs_step(logits, tokens, logprob_grad, entropy_grad,
                                                               _number(temperature, "temperature"), row_mask)
        if fast is not None:
            return fast
    lib = _lrs.load_library()
    d = _logprob_inputs(logits, tokens, temperature, row_mask)
    opt = _lrs._opt(options)
    device = logits.device
    up, up_entropy = _derivatives(logprob_grad, entropy_grad, d, device)
    with torch.cuda.device(device):
        workspace = _logprob_workspace(lib, workspace, d, 0, opt, device)
        logprobs, entropy = (torch.empty(d.rows, dtype=torch.float32, device=device) for _ in range(2))
        grad_out = _grad_out(grad_out, logits)
        _lrs._check(lib.token_logprobs_step(ctypes.byref(d), up, up_entropy, logprobs.data_ptr(), entropy.data_ptr(),
                                            grad_out.data_ptr(), grad_out.stride(0), workspace.data_ptr(), workspace.numel(),
                                            _lrs._stream(logits), opt), "token_logprobs_step")
    return logprobs, entropy, grad_out


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0, row_mask: torch.Tensor | None = None):
    """token_logprobs_forward's (logprobs, entropy), differentiable in the logits.

    Inside a graph capture use token_logprobs_forward and _backward, or _step, as with embedding_lookup."""
    out = (_rows._fast or _rows._binding()).logprobs_autograd(logits, tokens, _number(temperature, "temperature"), row_mask)
    if out is None:
        token_logprobs_forward(logits, tokens, temperature, row_mask)  # says what is wrong
        _lrs._bad("token_logprobs does not take these arguments")
    return out
