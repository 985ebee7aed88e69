"""Operators on the head of a sorted row and on counts of small keys.

    segmented_row_topk(x, k, descending=True)

The entry points of the C ABI under the same names (include/lsd_radix_sort.h),
with the checks, streams, outputs and errors of the package's sorts.  Matrices
may have any row stride (a slice of a wider buffer); the elements of a row are
contiguous.
"""
from __future__ import annotations

import torch

import lsd_radix_sort_amd as _lrs

_DTYPES = {torch.float16: _lrs.LRS_DTYPE_FP16, torch.bfloat16: _lrs.LRS_DTYPE_BF16,
           torch.float32: _lrs.LRS_DTYPE_FP32}


def _matrix(x, name: str) -> int:
    """Check a float matrix with contiguous rows; returns its LRS_DTYPE code."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _lrs._bad(f"{name} must be a GPU tensor")
    if x.dtype not in _DTYPES:
        _lrs._bad(f"{name} must be float16, bfloat16 or float32, got {x.dtype}")
    if x.dim() != 2:
        _lrs._bad(f"{name} must be a 2-D tensor")
    if x.shape[1] > 1 and x.stride(1) != 1:
        _lrs._bad(f"{name} must have contiguous rows (stride 1 along the last dimension)")
    return _DTYPES[x.dtype]


# ------------------------------------------------------------------- top k

def segmented_row_topk_workspace_size(rows: int, n: int, k: int, dtype: torch.dtype = torch.float16,
                                      options: "_lrs.SortOptions | None" = None) -> int:
    return int(_lrs.load_library().segmented_row_topk_workspace_size(rows, n, k, _DTYPES[dtype],
                                                                     _lrs._opt(options)))


def segmented_row_topk(x: torch.Tensor, k: int, descending: bool = True, values_out: torch.Tensor | None = None,
                       indices_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       options: "_lrs.SortOptions | None" = None):
    """The k largest (or smallest) elements of every row of a 2-D fp16/bf16/fp32 GPU tensor, in order:
    the first k columns of a stable row sort.  Returns (values, int64 column indices)."""
    lib = _lrs.load_library()
    dtype = _matrix(x, "x")
    rows, n = x.shape
    k = int(k)
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
