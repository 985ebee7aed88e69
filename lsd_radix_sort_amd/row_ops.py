"""Operators on the head of a sorted row and on counts of small keys.

    segmented_row_topk(x, k, descending=True)
    topk_distill_forward / _backward / _step(logits, teacher_values, teacher_indices, ...)
    expert_counts(indices, experts)
    expert_balance_forward / _backward / _step(logits, indices, ...)

The entry points of the C ABI (include/lsd_radix_sort.h), with the checks,
streams, outputs and errors of the package's sorts.  Matrices may have any row
stride (a slice of a wider buffer); the elements of a row are contiguous.
topk_distill_loss and expert_balance_loss are the same losses for programs that
differentiate through torch autograd; the `_step` calls return loss and
gradient at once, without it.

Calls that leave outputs and workspaces to the package go through a compiled
binding (csrc/row_binding.cpp); it takes them only when every argument is in
order, and the code here takes the others and names what is wrong with them.
"""
from __future__ import annotations

import ctypes
import operator

import torch

import lsd_radix_sort_amd as _lrs

_fast = None


def _binding():
    """The compiled binding of regular calls, bound to the loaded library's entry points."""
    global _fast
    if _fast is None:
        lib = _lrs.load_library()
        try:
            from lsd_radix_sort_amd import _row_binding as fast
        except ImportError as e:
            raise ImportError("lsd_radix_sort_amd/_row_binding.so is missing or of another torch: build it with "
                              "`python -m lsd_radix_sort_amd.build`") from e
        names = ("segmented_row_topk_workspace_size", "segmented_row_topk", "topk_distill_workspace_size",
                 "topk_distill_forward", "topk_distill_backward", "topk_distill_step",
                 "expert_balance_step_workspace_size", "expert_balance_step", "expert_balance")
        fast.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names})
        _fast = fast
    return _fast


_DTYPES = {torch.float16: _lrs.LRS_DTYPE_FP16, torch.bfloat16: _lrs.LRS_DTYPE_BF16,
           torch.float32: _lrs.LRS_DTYPE_FP32}


_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _dtype_code(dtype, name: str) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        _lrs._bad(f"{name} must be float16, bfloat16 or float32, got {dtype}")
    return code


def _whole(n, name: str) -> int:
    try:
        return operator.index(n)
    except TypeError:
        _lrs._bad(f"{name} must be a whole number, got {n!r}")


def _matrix(x, name: str) -> int:
    """Check a float matrix with contiguous rows; returns its LRS_DTYPE code."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _lrs._bad(f"{name} must be a GPU tensor")
    code = _dtype_code(x.dtype, name)
    if x.dim() != 2:
        _lrs._bad(f"{name} must be a 2-D tensor")
    if x.stride(1) != 1 and x.size(1) > 1:
        _lrs._bad(f"{name} must have contiguous rows (stride 1 along the last dimension)")
    return code


# ------------------------------------------------------------------- top k

def segmented_row_topk_workspace_size(rows: int, n: int, k: int, dtype: torch.dtype = torch.float16,
                                      options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().segmented_row_topk_workspace_size(rows, n, k, _dtype_code(dtype, "dtype"),
                                                                     _lrs._opt(options)))


def segmented_row_topk(x: torch.Tensor, k: int, descending: bool = True, values_out: torch.Tensor | None = None,
                       indices_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       options: "_lrs.SortOptions | None" = None):
    """The k largest (or smallest) elements of every row of a 2-D fp16/bf16/fp32 GPU tensor, in order:
    the first k columns of a stable row sort.  Returns (values, int64 column indices).

    Under autograd the values carry no gradient: torch.gather(x, 1, indices) are the same values with one."""
    k = _whole(k, "k")
    if values_out is None and indices_out is None and workspace is None and options is None:
        out = (_fast or _binding()).topk(x, k, bool(descending))
        if out is not None:
            return out
    lib = _lrs.load_library()
    dtype = _matrix(x, "x")
    rows, n = x.shape
    if not 0 <= k <= n:
        _lrs._bad(f"k must be between 0 and the row length {n}, got {k}")
    values_out = _lrs._output(values_out, "values_out", x, shape=(rows, k))
    indices_out = _lrs._output(indices_out, "indices_out", x, element_size=8, shape=(rows, k), dtype=torch.int64)
    opt = _lrs._opt(options)
    need = lib.segmented_row_topk_workspace_size(rows, n, k, dtype, opt)
    if need or workspace is not None:
        workspace = _lrs._workspace(workspace, need, x.device)
    _lrs._check(lib.segmented_row_topk(x.data_ptr(), x.stride(0), values_out.data_ptr(), indices_out.data_ptr(),
                                       rows, n, k, dtype, int(descending), _lrs._ptr(workspace), need,
                                       _lrs._stream(x), opt), "segmented_row_topk")
    return values_out, indices_out


# -------------------------------------------- distillation from top logits

class _Distill(ctypes.Structure):
    # mirrors struct lrs_distill
    _fields_ = [("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("teacher_values", ctypes.c_void_p), ("teacher_stride", ctypes.c_int64),
                ("teacher_indices", ctypes.c_void_p), ("index_stride", ctypes.c_int64),
                ("teacher_lse", ctypes.c_void_p), ("row_weights", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("teacher_dtype", ctypes.c_int), ("index_bytes", ctypes.c_int),
                ("temperature", ctypes.c_double)]


def _by_row(t, name: str, rows: int, device) -> int | None:
    if t is None:
        return None
    _lrs._same_device(t, name, device)
    if t.dtype is not torch.float32 or t.dim() != 1 or t.size(0) != rows or not t.is_contiguous():
        _lrs._bad(f"{name} must be a contiguous float32 tensor of shape ({rows},)")
    return t.data_ptr()


def _ids(t, name: str, rows: int, device) -> int:
    """Check a rows x k integer matrix; returns its element size."""
    _lrs._same_device(t, name, device)
    size = _ID_BYTES.get(t.dtype)
    if size is None:
        _lrs._bad(f"{name} must be int32 or int64, got {t.dtype}")
    if t.dim() != 2 or t.size(0) != rows:
        _lrs._bad(f"{name} must be a 2-D tensor of {rows} rows")
    if t.stride(1) != 1 and t.size(1) > 1:
        _lrs._bad(f"{name} must have contiguous rows (stride 1 along the last dimension)")
    return size


def _distill_inputs(logits, teacher_values, teacher_indices, temperature, teacher_lse, row_weights) -> _Distill:
    dtype = _matrix(logits, "logits")
    rows, n = logits.shape
    device = logits.device
    teacher_dtype = _matrix(teacher_values, "teacher_values")
    _lrs._same_device(teacher_values, "teacher_values", device)
    index_bytes = _ids(teacher_indices, "teacher_indices", rows, device)
    k = teacher_values.size(1)
    if teacher_values.size(0) != rows or teacher_indices.size(1) != k:
        _lrs._bad(f"teacher_values {tuple(teacher_values.shape)} and teacher_indices {tuple(teacher_indices.shape)} differ")
    return _Distill(logits.data_ptr(), logits.stride(0), teacher_values.data_ptr(), teacher_values.stride(0),
                    teacher_indices.data_ptr(), teacher_indices.stride(0),
                    _by_row(teacher_lse, "teacher_lse", rows, device),
                    _by_row(row_weights, "row_weights", rows, device), rows, n, k, dtype,
                    teacher_dtype, index_bytes, temperature)


def _grad_out(t, like: torch.Tensor) -> torch.Tensor:
    """A gradient like the logits: new and contiguous, or the caller's with contiguous rows."""
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _lrs._same_device(t, "grad_out", like.device)
    if t.dtype != like.dtype or t.shape != like.shape or (t.shape[1] > 1 and t.stride(1) != 1):
        _lrs._bad(f"grad_out must be a {like.dtype} tensor of shape {tuple(like.shape)} with contiguous rows")
    return t


def _scale(t, device) -> int | None:
    """The upstream gradient of a scalar loss."""
    if t is None:
        return None
    _lrs._same_device(t, "loss_grad", device)
    if t.dtype != torch.float32 or t.numel() != 1:
        _lrs._bad("loss_grad must be one float32 number")
    return t.data_ptr()


def topk_distill_workspace_size(rows: int, n: int, k: int, dtype: torch.dtype = torch.bfloat16,
                                options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().topk_distill_workspace_size(rows, n, k, _dtype_code(dtype, "dtype"),
                                                               _lrs._opt(options)))


def _distill_workspace(lib, workspace, d: _Distill, opt, device) -> torch.Tensor:
    return _lrs._workspace(workspace, lib.topk_distill_workspace_size(d.rows, d.n, d.k, d.dtype, opt), device)


def _distill_forward(d: _Distill, logits, row_loss, workspace, options):
    lib = _lrs.load_library()
    opt = _lrs._opt(options)
    workspace = _distill_workspace(lib, workspace, d, opt, logits.device)
    loss = torch.empty((), dtype=torch.float32, device=logits.device)
    stats = torch.empty((d.rows, d.k + 3), dtype=torch.float32, device=logits.device)
    _lrs._check(lib.topk_distill_forward(ctypes.byref(d), loss.data_ptr(), _lrs._ptr(row_loss), stats.data_ptr(),
                                         workspace.data_ptr(), workspace.numel(), _lrs._stream(logits), opt),
                "topk_distill_forward")
    return loss, stats


def _distill_backward(d: _Distill, logits, stats, loss_grad, grad_out, options):
    lib = _lrs.load_library()
    grad_out = _grad_out(grad_out, logits)
    _lrs._check(lib.topk_distill_backward(ctypes.byref(d), stats.data_ptr(), _scale(loss_grad, logits.device),
                                          grad_out.data_ptr(), grad_out.stride(0), _lrs._stream(logits),
                                          _lrs._opt(options)), "topk_distill_backward")
    return grad_out


def topk_distill_forward(logits: torch.Tensor, teacher_values: torch.Tensor, teacher_indices: torch.Tensor,
                         temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                         row_weights: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         options: "_lrs.SortOptions | None" = None):
    """KL divergence of a student's rows of logits from a teacher's top logits.

    teacher_values, teacher_indices: [rows, k], the teacher's top logits and their columns (slots with a
    column outside the row, such as -1, are unused).  With teacher_lse ([rows] float32, the log-sum-exp of
    the teacher's whole row over the temperature) the rest of the teacher's mass counts against the rest of
    the student's; without it the teacher's top logits are renormalised.  row_weights: [rows] float32, default
    1 / rows; a row of weight 0 is left out.  Returns (loss, row_loss [rows], row_stats for the backward)."""
    if workspace is None and options is None:
        out = (_fast or _binding()).distill_forward(logits, teacher_values, teacher_indices, float(temperature), teacher_lse,
                                                    row_weights)
        if out is not None:
            return out
    d = _distill_inputs(logits, teacher_values, teacher_indices, temperature, teacher_lse, row_weights)
    row_loss = torch.empty(d.rows, dtype=torch.float32, device=logits.device)
    loss, stats = _distill_forward(d, logits, row_loss, workspace, options)
    return loss, row_loss, stats


def topk_distill_backward(logits: torch.Tensor, teacher_values: torch.Tensor, teacher_indices: torch.Tensor,
                          row_stats: torch.Tensor, temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                          row_weights: torch.Tensor | None = None, loss_grad: torch.Tensor | None = None,
                          grad_out: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """The gradient of topk_distill_forward's loss in the logits, times loss_grad, from the same inputs
    and the row_stats that the forward returned."""
    d = _distill_inputs(logits, teacher_values, teacher_indices, temperature, teacher_lse, row_weights)
    _lrs.check_output(row_stats, "row_stats", logits.device, 4, (d.rows, d.k + 3))
    return _distill_backward(d, logits, row_stats, loss_grad, grad_out, options)


def topk_distill_step(logits: torch.Tensor, teacher_values: torch.Tensor, teacher_indices: torch.Tensor,
                      temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                      row_weights: torch.Tensor | None = None, grad_out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """topk_distill_forward and its gradient in one call: returns (loss, row_loss, grad)."""
    if grad_out is None and workspace is None and options is None:
        out = (_fast or _binding()).distill_step(logits, teacher_values, teacher_indices, float(temperature), teacher_lse,
                                                 row_weights)
        if out is not None:
            return out
    lib = _lrs.load_library()
    d = _distill_inputs(logits, teacher_values, teacher_indices, temperature, teacher_lse, row_weights)
    opt = _lrs._opt(options)
    workspace = _distill_workspace(lib, workspace, d, opt, logits.device)
    loss = torch.empty((), dtype=torch.float32, device=logits.device)
    row_loss = torch.empty(d.rows, dtype=torch.float32, device=logits.device)
    grad_out = _grad_out(grad_out, logits)
    _lrs._check(lib.topk_distill_step(ctypes.byref(d), loss.data_ptr(), row_loss.data_ptr(), grad_out.data_ptr(),
                                      grad_out.stride(0), workspace.data_ptr(), workspace.numel(),
                                      _lrs._stream(logits), opt), "topk_distill_step")
    return loss, row_loss, grad_out


def _once(gradient):
    """`gradient` as the backward of a Function that cannot be differentiated again: the check for that is
    made only where a graph of the backward is wanted."""
    checked = torch.autograd.function.once_differentiable(gradient)

    def backward(ctx, *grads):
        return (checked if torch.is_grad_enabled() else gradient)(ctx, *grads)
    return staticmethod(backward)


def topk_distill_loss(logits: torch.Tensor, teacher_values: torch.Tensor, teacher_indices: torch.Tensor,
                      temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                      row_weights: torch.Tensor | None = None) -> torch.Tensor:
    """topk_distill_forward's loss, differentiable in the logits (the teacher and the weights are constants).

    Inside a graph capture use topk_distill_step: a backward pass of torch's autograd may wait there for
    streams of graphs that were built outside it."""
    out = (_fast or _binding()).distill_loss(logits, teacher_values, teacher_indices, float(temperature), teacher_lse,
                                             row_weights)
    if out is None:
        topk_distill_forward(logits, teacher_values, teacher_indices, temperature, teacher_lse, row_weights)  # says what is wrong
        _lrs._bad("topk_distill_loss does not take these arguments")
    return out


# ------------------------------------------ expert counts and balance loss

_SCORES = {"softmax": 0, "sigmoid": 1}
_MAX_EXPERTS = 4096  # LRS_MAX_EXPERTS


def _mask(t, rows: int, device) -> int | None:
    if t is None:
        return None
    _lrs._same_device(t, "row_mask", device)
    if t.dtype not in (torch.bool, torch.uint8) or t.shape != (rows,) or not t.is_contiguous():
        _lrs._bad(f"row_mask must be a contiguous bool or uint8 tensor of shape ({rows},)")
    return t.data_ptr()


def expert_counts(indices: torch.Tensor, experts: int, row_mask: torch.Tensor | None = None,
                  options: "_lrs.SortOptions | None" = None):
    """How often each expert occurs in a [tokens, k] matrix of expert ids, over the tokens whose row_mask is
    set; ids outside [0, experts) are dropped slots.  Returns (counts int32 [experts], rows_counted int32 [1])."""
    lib = _lrs.load_library()
    if not isinstance(indices, torch.Tensor) or not indices.is_cuda:
        _lrs._bad("indices must be a GPU tensor")
    index_bytes = _ids(indices, "indices", indices.shape[0] if indices.dim() else 0, indices.device)
    rows, k = indices.shape
    experts = _whole(experts, "experts")
    if not 1 <= experts <= _MAX_EXPERTS:
        _lrs._bad(f"experts must be between 1 and {_MAX_EXPERTS}, got {experts}")
    both = torch.empty(experts + 1, dtype=torch.int32, device=indices.device)
    at = both.data_ptr()
    _lrs._check(lib.expert_counts(indices.data_ptr(), indices.stride(0), index_bytes,
                                  _mask(row_mask, rows, indices.device), at, at + 4 * experts, rows, k, experts,
                                  _lrs._stream(indices), _lrs._opt(options)), "expert_counts")
    return both[:experts], both[experts:]


def expert_balance_workspace_size(rows: int, experts: int, options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().expert_balance_workspace_size(rows, experts, _lrs._opt(options)))


def _balance(logits, counts, rows_counted, balance_weight, z_weight, score, row_mask, want_loss, loss_grad, want_grad,
             grad_out, workspace, options):
    lib = _lrs.load_library()
    dtype = _matrix(logits, "logits")
    rows, experts = logits.shape
    device = logits.device
    if score not in _SCORES:
        _lrs._bad(f"score must be one of {sorted(_SCORES)}")
    for t, name, size in ((counts, "counts", experts), (rows_counted, "rows_counted", 1)):
        if t is None and name == "rows_counted":
            continue
        _lrs._same_device(t, name, device)
        if t.dtype != torch.int32 or t.shape != (size,) or not t.is_contiguous():
            _lrs._bad(f"{name} must be a contiguous int32 tensor of shape ({size},)")
    opt = _lrs._opt(options)
    loss, grad, nbytes, ws = None, None, 0, None
    if want_loss:
        loss = torch.empty((), dtype=torch.float32, device=device)
        workspace = _lrs._workspace(workspace, lib.expert_balance_workspace_size(rows, experts, opt), device)
        ws, nbytes = workspace.data_ptr(), workspace.numel()
    if want_grad:
        grad = _grad_out(grad_out, logits)
    _lrs._check(lib.expert_balance(logits.data_ptr(), logits.stride(0), counts.data_ptr(), _lrs._ptr(rows_counted),
                                   _mask(row_mask, rows, device), rows, experts, dtype, _SCORES[score],
                                   balance_weight, z_weight, _lrs._ptr(loss), _scale(loss_grad, device),
                                   _lrs._ptr(grad), 0 if grad is None else grad.stride(0), ws, nbytes,
                                   _lrs._stream(logits), opt), "expert_balance")
    return loss, grad


def expert_balance_step_workspace_size(rows: int, k: int, experts: int,
                                       options: "_lrs.SortOptions | None" = None) -> int:
    """Workspace bytes of expert_balance_forward and _step on these tokens' own counts."""
    return int(_lrs.load_library().expert_balance_step_workspace_size(rows, k, experts, _lrs._opt(options)))


def _step(logits, indices, balance_weight, z_weight, score, row_mask, counts, want_kept, want_grad, grad_out, workspace,
          options):
    """Loss, counts, rows counted (if wanted) and gradient (if wanted), on these tokens' counts or the given ones."""
    if counts is None and grad_out is None and workspace is None and options is None and score in _SCORES:
        out = (_fast or _binding()).balance_step(logits, indices, float(balance_weight), float(z_weight), _SCORES[score],
                                                 row_mask, want_kept, want_grad)
        if out is not None:
            return out
    lib = _lrs.load_library()
    dtype = _matrix(logits, "logits")
    rows, experts = logits.shape
    device = logits.device
    index_bytes = _ids(indices, "indices", rows, device)
    if counts is not None:
        _, kept = expert_counts(indices, experts, row_mask, options)
        loss, grad = _balance(logits, counts, kept, balance_weight, z_weight, score, row_mask, True, None, want_grad,
                              grad_out, workspace, options)
        return loss, counts, kept, grad
    if score not in _SCORES:
        _lrs._bad(f"score must be one of {sorted(_SCORES)}")
    opt = _lrs._opt(options)
    k = indices.shape[1]
    need = lib.expert_balance_step_workspace_size(rows, k, experts, opt)
    workspace = _lrs._workspace(workspace, need, device)
    counts = torch.empty(experts, dtype=torch.int32, device=device)
    kept = torch.empty(1, dtype=torch.int32, device=device) if want_kept else None
    loss = torch.empty((), dtype=torch.float32, device=device)
    grad = _grad_out(grad_out, logits) if want_grad else None
    _lrs._check(lib.expert_balance_step(logits.data_ptr(), logits.stride(0), indices.data_ptr(), indices.stride(0),
                                        index_bytes, _mask(row_mask, rows, device), rows, k, experts, dtype,
                                        _SCORES[score], balance_weight, z_weight, counts.data_ptr(), _lrs._ptr(kept),
                                        loss.data_ptr(), _lrs._ptr(grad), 0 if grad is None else grad.stride(0),
                                        workspace.data_ptr(), need, _lrs._stream(logits), opt), "expert_balance_step")
    return loss, counts, kept, grad


def expert_balance_forward(logits: torch.Tensor, indices: torch.Tensor, balance_weight: float = 1.0,
                           z_weight: float = 0.0, score: str = "softmax", row_mask: torch.Tensor | None = None,
                           counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                           options: "_lrs.SortOptions | None" = None):
    """The load balance loss of [tokens, experts] router logits whose tokens chose `indices` [tokens, k].

    loss = mean over the tokens of row_mask of balance_weight * sum_e f_e p_e + z_weight * logsumexp^2, with
    f_e = experts * counts_e / sum(counts) and p the softmax (or normalised sigmoid) of the token's logits.
    counts: int32 [experts] to use in place of these tokens' own, such as their sum over ranks.
    Returns (loss, counts, rows_counted)."""
    return _step(logits, indices, balance_weight, z_weight, score, row_mask, counts, True, False, None, workspace,
                 options)[:3]


def expert_balance_backward(logits: torch.Tensor, counts: torch.Tensor, rows_counted: torch.Tensor | None = None,
                            balance_weight: float = 1.0, z_weight: float = 0.0, score: str = "softmax",
                            row_mask: torch.Tensor | None = None, loss_grad: torch.Tensor | None = None,
                            grad_out: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """The gradient of expert_balance_forward's loss in the logits, times loss_grad."""
    return _balance(logits, counts, rows_counted, balance_weight, z_weight, score, row_mask, False, loss_grad, True,
                    grad_out, None, options)[1]


def expert_balance_step(logits: torch.Tensor, indices: torch.Tensor, balance_weight: float = 1.0,
                        z_weight: float = 0.0, score: str = "softmax", row_mask: torch.Tensor | None = None,
                        counts: torch.Tensor | None = None, grad_out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, options: "_lrs.SortOptions | None" = None):
    """expert_balance_forward and its gradient from one read of the logits: returns (loss, counts, grad)."""
    loss, counts, _, grad = _step(logits, indices, balance_weight, z_weight, score, row_mask, counts, False, True,
                                  grad_out, workspace, options)
    return loss, counts, grad


def _balance_gradient(ctx, loss_grad, _):
    logits, counts, kept, row_mask = ctx.saved_tensors
    grad = expert_balance_backward(logits, counts, kept, *ctx.how, row_mask, loss_grad)
    return grad, None, None, None, None, None, None


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, indices, balance_weight, z_weight, score, row_mask, counts):
        loss, counts, kept = expert_balance_forward(logits, indices, balance_weight, z_weight, score, row_mask, counts)
        ctx.save_for_backward(logits, counts, kept, row_mask)
        ctx.how = (balance_weight, z_weight, score)
        ctx.mark_non_differentiable(counts)
        return loss, counts

    backward = _once(_balance_gradient)


def expert_balance_loss(logits: torch.Tensor, indices: torch.Tensor, balance_weight: float = 1.0,
                        z_weight: float = 0.0, score: str = "softmax", row_mask: torch.Tensor | None = None,
                        counts: torch.Tensor | None = None):
    """expert_balance_forward's loss, differentiable in the logits, and the counts: (loss, counts).

    Inside a graph capture use expert_balance_step, as with topk_distill_loss."""
    if counts is None and score in _SCORES:
        out = (_fast or _binding()).balance_loss(logits, indices, float(balance_weight), float(z_weight), _SCORES[score],
                                                 row_mask)
        if out is not None:
            return out
    return _BalanceLoss.apply(logits, indices, balance_weight, z_weight, score, row_mask, counts)
