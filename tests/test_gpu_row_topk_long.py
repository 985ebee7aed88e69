"""segmented_row_topk of rows that several workgroups share, streamed or held,
and of many rows by the largest workgroups: every order of elements, ties
across the pieces of a row, more rows than are shared finely."""
import numpy as np
import pytest
import torch

from test_gpu_row_topk import check, log, make_bits

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

KINDS = ["normal", "levels", "rising", "falling", "equal", "masked", "special", "patterns"]


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


@pytest.mark.parametrize("dtype,rows,n,k", [
    ("fp16", 1, 700_001, 1024), ("bf16", 2, 700_001, 1024), ("fp32", 1, 300_001, 1024), ("fp32", 3, 300_001, 1000),
    ("bf16", 1, 2_000_003, 300), ("fp32", 1, 1_000_001, 300)])
@pytest.mark.parametrize("kind", KINDS)
def test_streamed(dtype, rows, n, k, kind):
    """So many are wanted that shares of 256 KB would not fit the merge."""
    log(f"topk streamed {dtype} {kind} {rows}x{n} k={k}")
    bits = make_bits(kind, rows, n, dtype, 400 + n)
    check(bits, dtype, k, True)
    check(bits, dtype, k, False, pad=3, offset=1)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("n,k", [(1_300_001, 700), (300_001, 1024)])
def test_streamed_rows_of_the_largest_pattern(dtype, n, k):
    """Nothing can follow the largest image of all; few others lie between."""
    log(f"topk largest patterns {dtype} n={n} k={k}")
    t = np.uint32 if dtype == "fp32" else np.uint16
    for descending in (True, False):
        last = (np.iinfo(t).max >> 1) if descending else np.iinfo(t).max
        bits = np.full((2, n), last, dtype=t)
        bits[1, ::7] = 0
        check(bits, dtype, k, descending)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [(3, 200_003, 64), (70, 140_001, 40), (2, 132_001, 1024)])
@pytest.mark.parametrize("kind", KINDS)
def test_shared_and_merged(dtype, rows, n, k, kind):
    log(f"topk shared {dtype} {kind} {rows}x{n} k={k}")
    bits = make_bits(kind, rows, n, dtype, 500 + n)
    check(bits, dtype, k, True)
    check(bits, dtype, k, False, pad=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "levels", "equal", "masked"])
@pytest.mark.parametrize("k", [64, 700])
def test_many_rows_of_the_largest_workgroups(dtype, kind, k):
    rows, n = 258, 66_001 if dtype == "bf16" else 33_001
    log(f"topk many {dtype} {kind} {rows}x{n} k={k}")
    check(make_bits(kind, rows, n, dtype, 600), dtype, k, True, pad=1)


def test_more_shared_rows_than_one_launch_joins():
    """2^22 rows and more, each shared: one row of 256 KB and 4 bytes, seen that often."""
    n, rows = 65_537, (1 << 22) + 3
    x = torch.randn(n, generator=torch.Generator().manual_seed(7)).cuda()
    log(f"topk {rows} shared rows")
    values, indices = lrs.segmented_row_topk(x.expand(rows, n), 1)
    best = x.argmax()
    torch.cuda.synchronize()
    assert bool((indices == best).all()) and bool((values == x[best]).all())
