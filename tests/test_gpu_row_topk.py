"""GPU parity of segmented_row_topk with a stable sort of every row on the CPU:
values bit for bit and int64 columns, tolerance 0, over types, directions,
strides, alignments, lengths and the element orders that stress the selection
(sorted either way, all equal, few levels, special patterns)."""
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

lrs = pytest.importorskip("lsd_radix_sort_amd")

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SPECIAL16 = np.array([0xFFFF, 0xFC01, 0xFC00, 0xFF80, 0xFBFF, 0x8001, 0x8000, 0x0000, 0x0001, 0x7BFF, 0x7C00, 0x7F80,
                      0x7FFF], dtype=np.uint16)
SPECIAL32 = np.array([0xFFFFFFFF, 0xFFC00000, 0xFF800000, 0xFF7FFFFF, 0x80000001, 0x80000000, 0x00000000, 0x00000001,
                      0x7F7FFFFF, 0x7F800000, 0x7FC00000, 0x7FFFFFFF], dtype=np.uint32)


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lrs.load_library()


def image(bits: np.ndarray) -> np.ndarray:
    """The unsigned integers whose order is the row sorts' order of these patterns."""
    width = 8 * bits.itemsize
    b = bits.astype(np.int64)
    sign, ones = 1 << (width - 1), (1 << width) - 1
    return np.where(b & sign, b ^ ones, b | sign)


def expected(bits: np.ndarray, k: int, descending: bool):
    key = image(bits)
    order = np.argsort(-key if descending else key, axis=1, kind="stable")[:, :k]
    return np.take_along_axis(bits, order, axis=1), order


def make_bits(kind: str, rows: int, n: int, dtype: str, seed: int) -> np.ndarray:
    rng = np.random.default_rng(seed)
    if kind == "patterns":  # any bits at all
        bits = rng.integers(0, 1 << (32 if dtype == "fp32" else 16), size=(rows, n), dtype=np.uint64)
        return bits.astype(np.uint32 if dtype == "fp32" else np.uint16)
    x = rng.standard_normal((rows, n)).astype(np.float32) * 2.5
    if kind == "levels":
        x = np.round(x)
    elif kind == "rising":
        x = np.sort(x, axis=1)
    elif kind == "falling":
        x = -np.sort(-x, axis=1)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "masked":
        x[rng.random((rows, n)) < 0.5] = -np.inf
        x[0] = -np.inf
    t = torch.from_numpy(x).to(DTYPES[dtype])
    bits = t.view(torch.int32 if dtype == "fp32" else torch.int16).numpy()
    bits = bits.view(np.uint32 if dtype == "fp32" else np.uint16).copy()
    if kind == "special":
        s = SPECIAL32 if dtype == "fp32" else SPECIAL16
        at = rng.integers(0, n, size=(rows, max(1, n // 7)))
        np.put_along_axis(bits, at, s[rng.integers(0, s.size, size=at.shape)], axis=1)
    return bits


def to_gpu(bits: np.ndarray, dtype: str, pad: int = 0, offset: int = 0) -> torch.Tensor:
    """The matrix on the GPU, rows `pad` elements apart, the first one `offset` elements into its buffer."""
    rows, n = bits.shape
    signed = bits.view(np.int32 if dtype == "fp32" else np.int16)
    buf = np.full(offset + rows * (n + pad), -1, dtype=signed.dtype)
    buf[offset:].reshape(rows, n + pad)[:, :n] = signed
    g = torch.from_numpy(buf).cuda().view(DTYPES[dtype])
    return g[offset:].view(rows, n + pad)[:, :n]


def check(bits, dtype, k, descending, pad=0, offset=0, **kw):
    x = to_gpu(bits, dtype, pad, offset)
    values, indices = lrs.segmented_row_topk(x, k, descending=descending, **kw)
    torch.cuda.synchronize()
    ev, ei = expected(bits, k, descending)
    assert values.dtype == x.dtype and indices.dtype == torch.int64
    assert np.array_equal(indices.cpu().numpy(), ei)
    got = values.view(torch.int32 if dtype == "fp32" else torch.int16).cpu().numpy()
    assert np.array_equal(got.view(bits.dtype), ev)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,n,k", [
    (1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 8, 8), (70, 64, 6), (9, 255, 17), (300, 256, 8), (65, 257, 1), (4, 513, 512),
    (7, 1024, 1024), (2, 2049, 1000), (5, 4097, 64), (1, 8191, 129), (260, 8200, 33), (3, 16385, 1024),
    (1, 65536, 64), (2, 131075, 50), (1, 300_001, 1024), (257, 20_000, 5)])
def test_sizes(dtype, rows, n, k):
    log(f"topk {dtype} {rows}x{n} k={k}")
    bits = make_bits("normal", rows, n, dtype, 100 + n)
    check(bits, dtype, k, True)
    check(bits, dtype, k, False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("kind", ["levels", "rising", "falling", "equal", "masked", "special", "patterns"])
@pytest.mark.parametrize("rows,n,k", [(2, 50_000, 100), (270, 20_011, 64), (40, 300, 9), (300, 48, 16)])
def test_orders(dtype, kind, rows, n, k):
    log(f"topk {dtype} {kind} {rows}x{n} k={k}")
    bits = make_bits(kind, rows, n, dtype, 200 + n)
    check(bits, dtype, k, True)
    check(bits, dtype, k, False)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (63, 7)])
@pytest.mark.parametrize("rows,n,k", [(3, 70_001, 40), (260, 9_003, 12), (100, 160, 6)])
def test_strides(dtype, pad, offset, rows, n, k):
    log(f"topk {dtype} {rows}x{n} pad={pad} offset={offset}")
    check(make_bits("levels", rows, n, dtype, 300 + pad), dtype, k, True, pad, offset)


def test_broadcast_rows_and_empty():
    row = torch.randn(1000, device="cuda").half()
    values, indices = lrs.segmented_row_topk(row.expand(5, 1000), 10)
    v0, i0 = lrs.segmented_row_topk(row[None], 10)
    assert torch.equal(indices, i0.expand(5, 10)) and torch.equal(values, v0.expand(5, 10))
    for rows, n, k in ((0, 10, 3), (4, 10, 0), (4, 0, 0)):
        v, i = lrs.segmented_row_topk(torch.empty(rows, n, device="cuda"), k)
        assert v.shape == i.shape == (rows, k)


def test_head_of_the_row_sort():
    x = (torch.randn(300, 5000, device="cuda") * 4).round().bfloat16()
    for descending in (True, False):
        sv, si = lrs.segmented_row_sort(x, descending)
        v, i = lrs.segmented_row_topk(x, 77, descending)
        same = torch.equal(i, si[:, :77]) and torch.equal(v.view(torch.int16), sv[:, :77].contiguous().view(torch.int16))
        assert same


def test_given_outputs_workspace_stream_and_timer():
    bits = make_bits("normal", 3, 150_000, "bf16", 400)
    x = to_gpu(bits, "bf16")
    need = lrs.segmented_row_topk_workspace_size(3, 150_000, 20, torch.bfloat16)
    assert need > 0 and lrs.segmented_row_topk_workspace_size(3, 50_000, 20, torch.bfloat16) == 0
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    v = torch.empty(3, 20, dtype=torch.bfloat16, device="cuda")
    i = torch.empty(3, 20, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    timer = lrs.KernelTimer()
    with torch.cuda.stream(side):
        out = lrs.segmented_row_topk(x, 20, values_out=v, indices_out=i, workspace=ws,
                                     options=lrs.SortOptions(timer=timer))
    side.synchronize()
    assert out[0] is v and out[1] is i
    ms, launches = timer.read()
    assert launches["resident"] == 2 and ms["resident"] > 0
    ev, ei = expected(bits, 20, True)
    assert np.array_equal(i.cpu().numpy(), ei)
    with pytest.raises(ValueError, match="workspace holds"):
        lrs.segmented_row_topk(x, 20, workspace=ws[:-1])


def test_graph_replay():
    for rows, n, k in ((2, 60_000, 30), (2, 160_000, 30), (300, 200, 8)):
        x = torch.randn(rows, n, device="cuda").half()
        v, i = lrs.segmented_row_topk(x, k)
        ws = torch.empty(max(1, lrs.segmented_row_topk_workspace_size(rows, n, k, x.dtype)), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lrs.segmented_row_topk(x, k, values_out=v, indices_out=i, workspace=ws)
        for seed in range(3):
            x.copy_(torch.randn(rows, n, device="cuda"))
            g.replay()
            ev, ei = lrs.segmented_row_topk(x, k)
            assert torch.equal(i, ei) and torch.equal(v, ev)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "equal", "masked", "patterns", "falling"])
@pytest.mark.parametrize("rows,n,k", [
    (1, 9, 9), (131, 16, 5), (77, 17, 17), (500, 31, 3), (5, 33, 33), (9, 63, 63), (6, 64, 64), (3, 65, 64), (5, 66, 65),
    (1000, 129, 1), (33, 512, 64), (8, 1023, 40), (7, 1025, 64), (5, 2048, 64), (5, 2047, 2), (3, 2049, 64), (4, 4095, 33),
    (4, 4096, 64), (2, 4097, 64)])
def test_short_rows(dtype, kind, rows, n, k):
    """Rows held by one wave or part of one, at the edges of each form."""
    log(f"topk {dtype} {kind} {rows}x{n} k={k}")
    bits = make_bits(kind, rows, n, dtype, 300 + n)
    check(bits, dtype, k, True)
    check(bits, dtype, k, False, pad=3, offset=1)
