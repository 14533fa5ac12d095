"""The kernels that many rows, narrow rows and many small groups take, against the definitions (64 bits, or the row
format's rule in plain torch).  The reciprocal deviations that the backward pass reads come from the definition too.

Bounds of the norm: a sum of squares has only positive terms, at most 17 additions per thread and 10 levels of tree,
so it is off by less than 32 x 2^-24 relative, its root by half of that and three roundings; two more products: 2^-18.
Then half a step of the output type."""

import pytest
import torch

from moe_layer_top_b200 import ops
from tests.operator_helpers import (HALF_STEP, assert_within, offsets_of, product_bound, quantize_rows,
                                    quantize_weight, row_values, weight_values)

pytestmark = pytest.mark.gpu

EPS = 1e-6
FP32 = 2.0 ** -18


@pytest.fixture(autouse=True, scope="module")
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_layer_top_b200 import build
    build.build()


def _rows(seed, T, H, std=1.0, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((T, H + pad), generator=g, device="cuda", dtype=torch.bfloat16) * std)[:, :H]


def _weight(H):
    return (1 + 0.1 * _rows(99, 1, H)[0]).to(torch.bfloat16).contiguous()


def _rstd(s):
    return (s.double().square().mean(-1) + EPS).rsqrt()


# ----------------------------------------------------------------------------- norm
@pytest.mark.parametrize("T", [297, 300, 1037])
@pytest.mark.parametrize("H", [8, 256, 264, 512, 520, 4104, 7168, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_many_rows(T, H, residual):
    x, w = _rows(1, T, H, pad=8), _weight(H)
    r = _rows(2, T, H, std=3.0) if residual else None
    wide = torch.full((T, H + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    res = ops.rms_norm(x, w, EPS, residual=r, y=wide[:, :H], rstd=True)
    s = (x.double() + r.double()).to(torch.bfloat16) if residual else x
    if residual:
        assert torch.equal(res["residual"], s)
    rstd = _rstd(s)
    y = s.double() * rstd[:, None] * w.double()
    assert_within(res["rstd"], rstd, rstd * FP32)
    assert_within(wide[:, :H], y, y.abs() * (HALF_STEP[torch.bfloat16] + FP32))
    assert (wide[:, H:] == 7).all()


@pytest.mark.parametrize("T,H", [(297, 16), (300, 272), (1037, 512), (300, 528), (1037, 4112), (1037, 7168), (297, 16384)])
def test_fp8_norm_of_many_rows(T, H):
    x, w, r = _rows(3, T, H), _weight(H), _rows(4, T, H)
    res = ops.rms_norm(x, w, EPS, residual=r, fp8=True, rstd=True)
    s = (x.double() + r.double()).to(torch.bfloat16)
    rstd = _rstd(s)
    y = s.double() * rstd[:, None] * w.double()
    assert torch.equal(res["residual"], s)
    assert_within(res["y"], y, y.abs() * (HALF_STEP[torch.bfloat16] + FP32))
    codes, scales = quantize_rows(res["y"])
    assert torch.equal(res["scales"], scales) and torch.equal(res["codes"], codes)
    only = ops.rms_norm(x, w, EPS, residual=r, y=False, fp8=True)
    assert torch.equal(only["codes"], codes) and torch.equal(only["scales"], scales)


@pytest.mark.parametrize("T,H", [(T, H) for T in (4737, 9500) for H in (8, 256, 264, 512)] +
                         [(4736 * 8 + 3, 16), (1037, 4096), (1800, 5128), (300, 16384)])
@pytest.mark.parametrize("dres", [False, True])
def test_norm_backward_of_many_rows(T, H, dres):
    """Narrow rows: a warp holds a row, and here takes several."""
    dy, s, w = _rows(5, T, H, 0.01, pad=8), _rows(6, T, H, 2.0, pad=16), _weight(H)
    d = _rows(7, T, H, 0.01) if dres else None
    r = _rstd(s).float()
    dx, dw = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
    D, S, R = dy.double(), s.double(), r.double()[:, None]
    n, a = S * R, D * w.double()
    rx = R * (a - n * (a * n).mean(-1, keepdim=True))
    mag = R * (a.abs() + n.abs() * (a * n).abs().mean(-1, keepdim=True))
    if dres:
        rx, mag = rx + d.double(), mag + d.double().abs()
    # dx: some 30 fp32 roundings of terms of size `mag` in the sums, then half a step
    assert_within(dx, rx, rx.abs() * HALF_STEP[torch.bfloat16] + mag * FP32)
    # dw: T terms, each with two roundings, added one by one
    assert_within(dw, (D * n).sum(0), (D * n).abs().sum(0) * (T + 2) * 2.0 ** -23)
    again = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


# ----------------------------------------------------------------------------- FP8 rows
@pytest.mark.parametrize("rows,cols", [(8192, 7168), (40000, 272), (80003, 144), (75776, 128), (75777, 16),
                                       (9473, 1024), (5000, 2064), (2500, 4112)])
def test_many_rows_round_trip(rows, cols):
    """From 75776 scale groups on a thread takes several; narrow rows share a block, the last one cut."""
    x = _rows(8, rows, cols, 0.5, pad=8)
    x[-1, -1] = 448.0   # a scale border: amax / 448 is a power of two
    codes, scales = ops.quantize_rows_fp8(x)
    rc, rs = quantize_rows(x)
    assert torch.equal(scales, rs) and torch.equal(codes, rc)
    assert torch.equal(ops.dequantize_rows_fp8(codes, scales).double(), row_values(codes, scales))


# ----------------------------------------------------------------------------- FP8 products
def _check_fp8(sizes, N, K, dtype, seed):
    off = offsets_of(sizes, start=1)
    M, G = int(off[-1]) + 2, len(sizes)
    x, xs = quantize_rows(_rows(seed, M, K))
    w, ws = quantize_weight(_rows(seed + 1, G * N, K, 0.1).reshape(G, N, K))
    xv = row_values(x, xs)
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    ops.grouped_matmul(x, w, off, x_scale=xs, w_scale=ws, out=y)
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        wv = weight_values(w[g], ws[g])
        ref, mag = xv[a:b] @ wv.t(), xv[a:b].abs() @ wv.abs().t()
        assert_within(y[a:b], ref, product_bound(ref, mag, K, dtype, fp8=True))
    assert (y[:1] == 7).all() and (y[-2:] == 7).all()
    again = torch.full_like(y, 7.0)
    ops.grouped_matmul(x, w, off, x_scale=xs, w_scale=ws, out=again)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("sizes,N,K", [
    ([1, 17, 40, 70, 100, 128, 0, 3] * 8, 1032, 2064),         # every box, one behind the other
    ([128, 1] * 30 + [97, 16, 0, 33, 65], 904, 4112),          # large and small blocks in turn
    ([(i * 7919) % 61 for i in range(150)], 264, 1552),
    ([1] * 200 + [128] * 20, 136, 3088),                       # many small blocks, then large ones
])
def test_few_rows_per_group_in_tiles_of_many_sizes(sizes, N, K, dtype):
    """Many more tiles than SMs and many K blocks: the ring of bytes wraps with gaps of blocks of another size, and a
    large block waits for several small ones."""
    _check_fp8(sizes, N, K, dtype, 21)


@pytest.mark.parametrize("kind", ["normal", "positive", "mixed"])
@pytest.mark.parametrize("M,N,K", [(40, 264, 512), (40, 264, 4096), (300, 520, 4096), (1000, 1024, 512), (1, 4096, 7168),
                                   (2048, 2048, 2048), (77, 2056, 144)])
def test_fp8_sums_are_those_of_fp32(M, N, K, kind):
    """The products of E4M3 numbers are exact in fp32; 128 of them are added in the tensor core, each addition off by
    at most one step (2^-23) of the running magnitude, then ceil(K / 128) sums and up to eight parts of a shared
    reduction: (128 + ceil(K / 128) + 8) 2^-23 of the magnitude in all, 2^-15.5 at most here.  (An accumulator of 14
    bits that truncates is off by 2^-14 of the block's largest term in the mean, per term: 2^-12 of the magnitude of
    positive data whose largest term is four times the mean one.)"""
    x, w = _rows(31, M, K).contiguous(), _rows(32, N, K, 0.1)
    if kind == "positive":
        x, w = x.abs(), w.abs()
    elif kind == "mixed":
        g = torch.Generator(device="cuda")
        g.manual_seed(33)
        x = x * torch.exp2(torch.randint(-8, 1, x.shape, generator=g, device="cuda")).to(torch.bfloat16)
        w = w * torch.exp2(torch.randint(-8, 1, w.shape, generator=g, device="cuda")).to(torch.bfloat16)
    (x, xs), (w, ws) = quantize_rows(x), quantize_weight(w)
    y = ops.matmul_fp8(x, xs, w, ws, out_dtype=torch.float32)
    xv, wv = row_values(x, xs), weight_values(w, ws)
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    assert_within(y, ref, ref.abs() * HALF_STEP[torch.float32] + mag * (128 + -(-K // 128) + 8) * 2.0 ** -23)
