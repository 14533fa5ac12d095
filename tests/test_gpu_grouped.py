"""The grouped matrix products (forward bf16 and FP8, dx, dw) and the dense FP8 product on the GPU
against 64-bit evaluations of their definitions, with derived element bounds."""

import pytest
import torch

from moe_layer_top_b200 import ops
from tests.operator_helpers import (assert_within, offsets_of, product_bound, quantize_rows, quantize_weight,
                                    row_values, weight_values)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_layer_top_b200 import build
    build.build()


def _randn(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std


def _rows(seed, M, n, std=1.0, pad=0):
    return _randn(seed, M, n + pad, std=std)[:, :n]


def _blocks(off):
    o = off.tolist()
    return [(g, o[g], o[g + 1]) for g in range(len(o) - 1) if o[g + 1] > o[g]]


SIZES = [
    [1], [5], [127], [128], [129], [300],
    [0, 1], [1, 0, 2], [0, 0, 0, 3, 0], [16, 17, 15], [130, 0, 1, 260],
    [7] * 20, [64, 1, 64, 200, 33, 0, 0, 5],
]
# enough tiles for the kernels that pair two SMs
# and few tiles with long reductions for those that share one
LONG = [([3], 136, 2048), ([40, 0, 2], 264, 1104), ([130], 128, 4096)]
LARGE = [([700, 0, 300, 33, 513, 1000], 2056, 528), ([1, 2048, 31, 257, 256, 255], 2304, 464)]
SHAPES = [(8, 8), (64, 64), (128, 128), (136, 72), (256, 1024), (264, 328), (1000, 200), (56, 520)]


def _cases():
    """Every row pattern with two shapes, every shape with several patterns."""
    out = []
    for i, sizes in enumerate(SIZES):
        for j in (i, i + 3):
            out.append((sizes, *SHAPES[j % len(SHAPES)]))
    return out + LARGE + LONG + [(sizes, K, N) for sizes, N, K in LARGE + LONG] + [([2000], 136, 72), ([700, 900], 264, 56)]


def _forward(x, w, off, N, M, **kw):
    y = torch.full((M, N), 7.0, dtype=kw.pop("dtype", torch.bfloat16), device="cuda")
    ops.grouped_matmul(x, w, off, out=y, **kw)
    return y


def _check_rows(y, ref_of, off, M, terms, fp8=False):
    """Rows of groups within their bounds, others left as they were."""
    covered = torch.zeros((M,), dtype=torch.bool, device="cuda")
    for g, a, b in _blocks(off):
        ref, mag = ref_of(g, a, b)
        assert_within(y[a:b], ref, product_bound(ref, mag, terms, y.dtype, fp8))
        covered[a:b] = True
    assert (y[~covered] == 7).all()


@pytest.mark.parametrize("sizes,N,K", _cases())
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_forward(sizes, N, K, dtype):
    off = offsets_of(sizes, start=2)                      # rows before the first and behind the last group
    M, G = int(off[-1]) + 3, len(sizes)
    x, w = _rows(1, M, K, pad=8), _randn(2, G, N, K, std=0.1)
    y = _forward(x, w, off, N, M, dtype=dtype)
    _check_rows(y, lambda g, a, b: (x[a:b].double() @ w[g].double().t(),
                                    x[a:b].double().abs() @ w[g].double().abs().t()), off, M, K)


@pytest.mark.parametrize("sizes,N,K", _cases())
def test_forward_fp8(sizes, N, K):
    K = (K + 15) // 16 * 16
    off = offsets_of(sizes, start=1)
    M, G = int(off[-1]) + 2, len(sizes)
    x, xs = quantize_rows(_rows(3, M, K))
    w, ws = quantize_weight(_randn(4, G, N, K, std=0.1))
    xv, wv = row_values(x, xs), weight_values(w, ws)
    for dtype in (torch.bfloat16, torch.float32):
        y = _forward(x, w, off, N, M, dtype=dtype, x_scale=xs, w_scale=ws)
        _check_rows(y, lambda g, a, b: (xv[a:b] @ wv[g].t(), xv[a:b].abs() @ wv[g].abs().t()), off, M, K, fp8=True)


@pytest.mark.parametrize("sizes,N,K", _cases())
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_dx(sizes, N, K, dtype):
    off = offsets_of(sizes, start=2)
    M, G = int(off[-1]) + 3, len(sizes)
    dy, w = _rows(5, M, N, pad=16), _randn(6, G, N, K, std=0.1)
    dx = torch.full((M, K), 7.0, dtype=dtype, device="cuda")
    ops.grouped_matmul_dx(dy, w, off, out=dx)
    _check_rows(dx, lambda g, a, b: (dy[a:b].double() @ w[g].double(), dy[a:b].double().abs() @ w[g].double().abs()),
                off, M, N)


@pytest.mark.parametrize("tiles", [10, 18, 20, 24, 29, 37, 49, 74])
@pytest.mark.parametrize("M", [5, 77])
def test_every_number_of_parts_of_a_reduction(tiles, M):
    """Few tiles with long reductions, shared by 8, 7, 6, 5, 4, 3 and 2 CTAs (or fewer, where a GPU holds fewer
    clusters of that size at once)."""
    n, k = 128 * tiles - 40, 2072
    off = offsets_of([M])
    x, w = _rows(11, M, k), _randn(12, 1, n, k, std=0.1)
    y = _forward(x, w, off, n, M)
    _check_rows(y, lambda g, a, b: (x[a:b].double() @ w[g].double().t(),
                                    x[a:b].double().abs() @ w[g].double().abs().t()), off, M, k)
    dy, wt = _rows(13, M, k), _randn(14, 1, k, n, std=0.1)
    dx = torch.full((M, n), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.grouped_matmul_dx(dy, wt, off, out=dx)
    _check_rows(dx, lambda g, a, b: (dy[a:b].double() @ wt[g].double(), dy[a:b].double().abs() @ wt[g].double().abs()),
                off, M, k)
    a, b = _rows(15, 27 * M + 2000, n), _rows(16, 27 * M + 2000, 120)
    dw = ops.grouped_matmul_dw(a, b, None, out_dtype=torch.float32)
    ref, mag = a.double().t() @ b.double(), a.double().abs().t() @ b.double().abs()
    assert_within(dw[0], ref, product_bound(ref, mag, a.shape[0], torch.float32))
    k = 4112
    (q, qs), (c, cs) = quantize_rows(_rows(17, M, k)), quantize_weight(_randn(18, n, k, std=0.1))
    y = ops.matmul_fp8(q, qs, c, cs)
    xv, wv = row_values(q, qs), weight_values(c, cs)
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    assert_within(y, ref, product_bound(ref, mag, k, torch.bfloat16, True))


@pytest.mark.parametrize("sizes,N,K", [([200], 4872, 4112), ([450], 4104, 4480), ([150, 0, 301], 2056, 4240),
                                       ([1, 500, 40], 2120, 4096)])
def test_fp8_tiles_whose_reduction_two_pairs_share(sizes, N, K):
    off = offsets_of(sizes, start=1)
    M, G = int(off[-1]) + 2, len(sizes)
    x, xs = quantize_rows(_rows(21, M, K))
    w, ws = quantize_weight(_randn(22, G, N, K, std=0.1))
    xv, wv = row_values(x, xs), weight_values(w, ws)
    for dtype in (torch.bfloat16, torch.float32):
        y = _forward(x, w, off, N, M, dtype=dtype, x_scale=xs, w_scale=ws)
        _check_rows(y, lambda g, a, b: (xv[a:b] @ wv[g].t(), xv[a:b].abs() @ wv[g].abs().t()), off, M, K, fp8=True)
        assert torch.equal(y, _forward(x, w, off, N, M, dtype=dtype, x_scale=xs, w_scale=ws))


@pytest.mark.parametrize("sizes,N,K", _cases())
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)],
                         ids=["bf16", "fp32", "accumulate"])
def test_dw(sizes, N, K, dtype, accumulate):
    off = offsets_of(sizes, start=2)
    M, G = int(off[-1]) + 3, len(sizes)
    dy, x = _rows(7, M, N, pad=8), _rows(8, M, K, pad=24)
    # rows of no group must not reach any gradient
    dy, x = dy.clone(), x.clone()
    dy[:2], x[:2], dy[-3:], x[-3:] = float("nan"), float("inf"), float("inf"), float("nan")
    dw = torch.randn((G, N, K), device="cuda").to(dtype)
    before = dw.clone()
    ops.grouped_matmul_dw(dy, x, off, out=dw, accumulate=accumulate)
    o = off.tolist()
    for g in range(G):
        a, b = dy[o[g]:o[g + 1]].double(), x[o[g]:o[g + 1]].double()
        ref, mag = a.t() @ b, a.abs().t() @ b.abs()
        bound = product_bound(ref, mag, max(1, sizes[g]), dtype)
        if accumulate:
            ref = ref + before[g].double()
            bound = bound + 2.0 ** -24 * ref.abs() * 2
        assert_within(dw[g], ref, bound)
        if sizes[g] == 0:
            assert torch.equal(dw[g], before[g] if accumulate else torch.zeros_like(dw[g]))


@pytest.mark.parametrize("N,K", [(136, 72), (1160, 2312)])
def test_a_groups_gradient_does_not_see_its_neighbours(N, K):
    """NaN in one group's rows stays in that group, for every tail length of a 64-row stage."""
    for n in (1, 15, 16, 17, 48, 63, 64, 65, 100):
        off = offsets_of([n, 40])
        dy, x = _randn(9, n + 40, N), _randn(10, n + 40, K)
        clean = ops.grouped_matmul_dw(dy, x, off)
        dy[n:], x[n:] = float("nan"), float("nan")
        got = ops.grouped_matmul_dw(dy, x, off)
        assert torch.equal(got[0], clean[0]) and torch.isnan(got[1]).all()
        y = ops.grouped_matmul(x, _randn(11, 2, N, K), off)
        assert torch.isfinite(y[:n]).all() and torch.isnan(y[n:]).all()


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 4096, 7168), (2, 128, 128), (16, 264, 144), (17, 1536, 4096),
                                   (130, 520, 1616), (333, 2056, 1616), (1000, 1024, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_dense_fp8(M, N, K, dtype):
    x = _randn(12, M, K, std=0.5)
    codes, scales = ops.quantize_rows_fp8(x)
    w, ws = quantize_weight(_randn(13, N, K, std=0.02))
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    y = ops.matmul_fp8(codes, scales, w, ws, out_dtype=dtype, status=status)
    xv, wv = row_values(codes, scales), weight_values(w, ws)
    ref = xv @ wv.t()
    assert_within(y, ref, product_bound(ref, xv.abs() @ wv.abs().t(), K, dtype, fp8=True))
    assert int(status) == 0
    wide = torch.full((M, N + 8), 7.0, dtype=dtype, device="cuda")
    ops.matmul_fp8(codes, scales, w, ws, out=wide[:, :N])
    assert torch.equal(wide[:, :N], y) and (wide[:, N:] == 7).all()


def test_dense_fp8_takes_the_layers_quantised_weights():
    N, K, M = 256, 384, 40
    w = _randn(14, N, K, std=0.02)
    q, s = ops.quantize_weights_fp8(w)
    rq, rs = quantize_weight(w)
    assert torch.equal(q, rq) and torch.equal(s, rs)
    codes, scales = ops.quantize_rows_fp8(_randn(15, M, K))
    y = ops.matmul_fp8(codes, scales, q, s, out_dtype=torch.float32)
    xv, wv = row_values(codes, scales), weight_values(q, s)
    assert_within(y, xv @ wv.t(), product_bound(xv @ wv.t(), xv.abs() @ wv.abs().t(), K, torch.float32, fp8=True))


@pytest.mark.parametrize("sizes,N,K", [([5, 3, 140], 264, 272), LARGE[0]])
def test_fp8_rows_with_nan_stay_their_own(sizes, N, K):
    """A NaN code spoils its own row; a NaN in a group's weights only that group's column."""
    off = offsets_of(sizes)
    M = int(off[-1])
    codes, scales = quantize_rows(_randn(33, M, K))
    w, ws = quantize_weight(_randn(34, len(sizes), N, K, std=0.1))
    clean = ops.grouped_matmul(codes, w, off, x_scale=scales, w_scale=ws)
    bad_rows = [0, int(off[-1]) - 1, int(off[1])]
    for r in bad_rows:
        codes[r, r % K] = 0x7F
    w[-1, 9, 7] = 0xFF
    got = ops.grouped_matmul(codes, w, off, x_scale=scales, w_scale=ws)
    want = clean.clone()
    want[bad_rows] = float("nan")
    want[int(off[-2]):, 9] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(got)], clean[~torch.isnan(got)])


def test_one_group_without_offsets():
    x, w = _randn(16, 200, 256), _randn(17, 1, 136, 256, std=0.1)
    y = ops.grouped_matmul(x, w, None)
    assert torch.equal(y, ops.grouped_matmul(x, w, offsets_of([200])))
    dy = _randn(18, 200, 136)
    assert torch.equal(ops.grouped_matmul_dx(dy, w, None), ops.grouped_matmul_dx(dy, w, offsets_of([200])))
    assert torch.equal(ops.grouped_matmul_dw(dy, x, None), ops.grouped_matmul_dw(dy, x, offsets_of([200])))


def test_no_rows():
    w = _randn(19, 3, 64, 128)
    off = offsets_of([0, 0, 0])
    x, dy = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 64), dtype=torch.bfloat16,
                                                                                    device="cuda")
    assert ops.grouped_matmul(x, w, off).shape == (0, 64)
    assert ops.grouped_matmul_dx(dy, w, off).shape == (0, 128)
    dw = ops.grouped_matmul_dw(dy, x, off)
    assert torch.equal(dw, torch.zeros_like(dw)) and dw.shape == (3, 64, 128)
    acc = torch.ones((3, 64, 128), device="cuda")
    ops.grouped_matmul_dw(dy, x, off, out=acc, accumulate=True)
    assert (acc == 1).all()


def test_many_groups():
    """1024 groups, most of them empty or of a single row."""
    sizes = [(i * 7919) % 3 for i in range(1024)]
    off = offsets_of(sizes)
    M, N, K = int(off[-1]), 136, 72
    x, w = _randn(20, M, K), _randn(21, 1024, N, K, std=0.1)
    g = torch.repeat_interleave(torch.arange(1024, device="cuda"), torch.tensor(sizes, device="cuda"))
    y = ops.grouped_matmul(x, w, off)
    ref = torch.einsum("mk,mnk->mn", x.double(), w.double()[g])
    mag = torch.einsum("mk,mnk->mn", x.double().abs(), w.double().abs()[g])
    assert_within(y, ref, product_bound(ref, mag, K, torch.bfloat16))
    dy = _randn(22, M, N)
    dx = ops.grouped_matmul_dx(dy, w, off)
    ref = torch.einsum("mn,mnk->mk", dy.double(), w.double()[g])
    mag = torch.einsum("mn,mnk->mk", dy.double().abs(), w.double().abs()[g])
    assert_within(dx, ref, product_bound(ref, mag, N, torch.bfloat16))


def test_gradients_against_differences():
    """dx and dw of sum(c * y) for y = x w^T, by differences in double (the function is linear in each)."""
    sizes, N, K = [3, 0, 4], 24, 16
    off = offsets_of(sizes)
    x, w, c = _randn(23, 7, K), _randn(24, 3, N, K), _randn(25, 7, N)
    dx, dw = ops.grouped_matmul_dx(c, w, off, out_dtype=torch.float32), ops.grouped_matmul_dw(c, x, off,
                                                                                              out_dtype=torch.float32)
    g = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sizes, device="cuda"))

    def loss(xd, wd):
        return (c.double() * torch.einsum("mk,mnk->mn", xd, wd[g])).sum()

    xd, wd = x.double(), w.double()
    for r, k in [(0, 0), (3, 15), (6, 7)]:
        e = torch.zeros_like(xd)
        e[r, k] = 1.0
        assert abs((loss(xd + e, wd) - loss(xd - e, wd)) / 2 - dx[r, k].double()) <= 1e-4
    for i, n, k in [(0, 0, 0), (1, 5, 5), (2, 23, 15)]:
        e = torch.zeros_like(wd)
        e[i, n, k] = 1.0
        assert abs((loss(xd, wd + e) - loss(xd, wd - e)) / 2 - dw[i, n, k].double()) <= 1e-4


@pytest.mark.parametrize("offs", [[-5, 20, 1000, 60], [40, 10, 30, 20], [2 ** 31 - 1, -2 ** 31, 50, 0], [7, 7, 3, 90]])
def test_offsets_out_of_range_or_order(offs):
    """They count as clamped to [0, M] and, where one is below an earlier one, as that one."""
    M, N, K = 50, 64, 128
    x, w, dy = _randn(26, M, K), _randn(27, 3, N, K), _randn(28, M, N)
    good = torch.tensor(offs, dtype=torch.int64).clamp(0, M).cummax(0).values.to(torch.int32).cuda()
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    guard = torch.full((M + 20, N), 7.0, dtype=torch.bfloat16, device="cuda")
    want = guard.clone()
    ops.grouped_matmul(x, w, off, out=guard[10:10 + M])
    ops.grouped_matmul(x, w, good, out=want[10:10 + M])
    assert torch.equal(guard, want) and (guard[:10] == 7).all() and (guard[10 + M:] == 7).all()
    assert torch.equal(ops.grouped_matmul_dw(dy, x, off), ops.grouped_matmul_dw(dy, x, good))


def test_repeated_calls_agree_bit_for_bit():
    off = offsets_of([70, 0, 300, 5, 129])
    x, w = _randn(29, 504, 520), _randn(30, 5, 264, 520)
    dy = _randn(31, 504, 264)
    first = [ops.grouped_matmul(x, w, off), ops.grouped_matmul_dx(dy, w, off), ops.grouped_matmul_dw(dy, x, off)]
    for _ in range(3):
        again = [ops.grouped_matmul(x, w, off), ops.grouped_matmul_dx(dy, w, off), ops.grouped_matmul_dw(dy, x, off)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
