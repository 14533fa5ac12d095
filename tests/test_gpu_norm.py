"""The RMS norm (forward, FP8 output, backward) and the E4M3 row format on the GPU against 64-bit
evaluations of their definitions.

Bounds: a row's sum of squares has only positive terms, at most 16 per thread and 10 levels of
tree, so it is off by less than 32 x 2^-24 relative and rstd by half of that and three roundings;
the products add two more: 2^-18 covers them.  Then half a step of the output type."""

import pytest
import torch

from moe_layer_top_b200 import ops
from tests.operator_helpers import HALF_STEP, assert_within, quantize_rows, row_values

pytestmark = pytest.mark.gpu

EPS = 1e-6
FP32 = 2.0 ** -18


@pytest.fixture(autouse=True, scope="module")
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_layer_top_b200 import build
    build.build()


def _rows(seed, T, H, std=1.0, stride=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, stride or H), generator=g, device="cuda", dtype=torch.bfloat16) * std
    return x[:, :H]


def _weight(H):
    return (1 + 0.1 * _rows(99, 1, H)[0]).to(torch.bfloat16).contiguous()


def _reference(s, w):
    s = s.double()
    r = (s.square().mean(-1) + EPS).rsqrt()
    return s * r[:, None] * w.double(), r


def _check_forward(res, s, w):
    y, r = _reference(s, w)
    assert_within(res["rstd"], r, r * FP32)
    if res["y"] is not None:
        assert_within(res["y"], y, y.abs() * (HALF_STEP[torch.bfloat16] + FP32))


@pytest.mark.parametrize("T,H", [(1, 8), (1, 16), (3, 128), (9, 136), (17, 256), (5, 264), (2, 1000), (257, 4096),
                                 (33, 4104), (64, 7168), (3, 8192), (4, 8200), (2, 16384), (1, 16376)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, H, residual):
    x, w = _rows(1, T, H), _weight(H)
    r = _rows(2, T, H, std=3.0) if residual else None
    x0 = x.clone()
    res = ops.rms_norm(x, w, EPS, residual=r, rstd=True)
    s = (x.float() + r.float()).to(torch.bfloat16) if residual else x
    if residual:
        assert torch.equal(res["residual"], s)
    assert torch.equal(x, x0)
    _check_forward(res, s, w)


@pytest.mark.parametrize("T,H", [(1, 16), (1, 7168), (7, 128), (5, 144), (130, 1616), (33, 2048), (16, 8208), (3, 16384)])
def test_fp8_rows_are_those_of_the_rounded_output(T, H):
    x, w, r = _rows(3, T, H), _weight(H), _rows(4, T, H)
    res = ops.rms_norm(x, w, EPS, residual=r, fp8=True, rstd=True)
    _check_forward(res, res["residual"], w)
    codes, scales = quantize_rows(res["y"])
    assert torch.equal(res["scales"], scales) and torch.equal(res["codes"], codes)
    only = ops.rms_norm(x, w, EPS, residual=r, y=False, fp8=True)
    assert only["y"] is None and only["rstd"] is None
    assert torch.equal(only["codes"], codes) and torch.equal(only["scales"], scales)


def test_strided_rows_and_aliases():
    T, H = 37, 512
    x, r = _rows(5, T, H, stride=640), _rows(6, T, H, stride=520)
    w = _weight(H)
    s = (x.float() + r.float()).to(torch.bfloat16)
    wide = torch.full((T, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    res = ops.rms_norm(x, w, EPS, residual=r, residual_out=r, y=wide[:, :H], rstd=True)   # in place
    assert torch.equal(r, s) and torch.equal(wide[:, H:], torch.full_like(wide[:, H:], 7.0))
    _check_forward(res, s, w)
    x2 = s.clone()
    ops.rms_norm(x2, w, EPS, y=x2)                                                         # y over x
    assert torch.equal(x2, wide[:, :H])


def test_rows_of_zeros_and_of_large_and_small_values():
    H = 256
    x = torch.zeros((4, H), dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 7] = 300.0
    w = torch.ones((H,), dtype=torch.bfloat16, device="cuda")
    res = ops.rms_norm(x, w, EPS, rstd=True, fp8=True)
    _check_forward(res, x, w)
    codes, scales = quantize_rows(res["y"])
    assert torch.equal(res["codes"], codes) and torch.equal(res["scales"], scales)


def test_non_finite_rows_stay_their_own():
    H = 512
    x = _rows(7, 4, H).contiguous()
    clean = ops.rms_norm(x, _weight(H), EPS)["y"]
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    res = ops.rms_norm(x, _weight(H), EPS, fp8=True)
    assert torch.equal(res["y"][0], clean[0]) and torch.equal(res["y"][3], clean[3])
    assert torch.isnan(res["y"][1]).all()
    assert torch.isnan(res["y"][2, 5]) and (res["y"][2, :5] == 0).all()
    codes, scales = quantize_rows(res["y"])
    nan = (codes & 127) == 127
    assert torch.equal((res["codes"] & 127) == 127, nan)
    assert torch.equal(res["codes"][~nan], codes[~nan]) and torch.equal(res["scales"], scales)


def test_no_rows():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    res = ops.rms_norm(x, _weight(256), EPS, fp8=True, rstd=True)
    assert res["y"].shape == (0, 256) and res["scales"].shape == (2, 0)
    dx, dw = ops.rms_norm_backward(x, x, _weight(256), torch.empty((0,), device="cuda"))
    assert dx.shape == (0, 256) and torch.equal(dw, torch.zeros_like(dw))


# ----------------------------------------------------------------------------- backward
def _backward_reference(dy, s, w, r, dres):
    dy, s, w, r = dy.double(), s.double(), w.double(), r.double()[:, None]
    n, a = s * r, dy * w
    dx = r * (a - n * (a * n).mean(-1, keepdim=True))
    mag = r * (a.abs() + n.abs() * (a * n).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    return dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 4096), (2, 136), (37, 256), (295, 1000), (296, 1024), (297, 264),
                                 (1037, 4096), (900, 7168), (5, 8200), (3, 16384)])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(T, H, dres):
    dy, s, w = _rows(11, T, H, 0.01), _rows(12, T, H, 2.0), _weight(H)
    d = _rows(13, T, H, 0.01) if dres else None
    r = ops.rms_norm(s, w, EPS, rstd=True)["rstd"]
    dx, dw = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
    rx, mag, rw, wmag = _backward_reference(dy, s, w, r, d)
    # dx: some 30 fp32 roundings of terms of size `mag` in the sums, then half a step
    assert_within(dx, rx, rx.abs() * HALF_STEP[torch.bfloat16] + mag * FP32)
    # dw: T terms, each with two roundings, added one by one
    assert_within(dw, rw, wmag * (T + 2) * 2.0 ** -23)
    again = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("T,H", [(1776, 5120), (1775, 5120), (1800, 5128), (14300, 520), (3552, 4096), (149, 8200),
                                 (300, 12288), (1, 10240), (447, 16384)])
def test_backward_with_rows_under_way(T, H):
    """Where rows are copied ahead: one and two vectors per thread, blocks with equal and unequal numbers of rows,
    every number of rows ahead, outputs in place."""
    dy, s, w = _rows(14, T, H, 0.01, stride=H + 8), _rows(15, T, H, 2.0, stride=H + 16), _weight(H)
    r = ops.rms_norm(s, w, EPS, rstd=True)["rstd"]
    for d in (None, _rows(16, T, H, 0.01)):
        dx, dw = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
        rx, mag, rw, wmag = _backward_reference(dy, s, w, r, d)
        assert_within(dx, rx, rx.abs() * HALF_STEP[torch.bfloat16] + mag * FP32)
        assert_within(dw, rw, wmag * (T + 2) * 2.0 ** -23)
        place = dy.clone() if d is None else d
        again = ops.rms_norm_backward(dy if d is not None else place, s, w, r, dresidual=d, dx=place)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_against_differences():
    """The gradient of sum(c * y) in double, by central differences of the definition."""
    T, H, h = 3, 24, 1e-5
    s, c, w = _rows(21, T, H, 2.0), _rows(22, T, H), _weight(H)
    r = ops.rms_norm(s, w, EPS, rstd=True)["rstd"]
    dx, dw = ops.rms_norm_backward(c, s, w, r)

    def loss(sd, wd):
        return (c.double() * sd * (sd.square().mean(-1, keepdim=True) + EPS).rsqrt() * wd).sum()

    sd, wd = s.double(), w.double()
    for t, i in [(0, 0), (1, 5), (2, 23)]:
        e = torch.zeros_like(sd)
        e[t, i] = h
        num = (loss(sd + e, wd) - loss(sd - e, wd)) / (2 * h)
        # bf16 half step, and h^2 times a third derivative of order 1
        assert abs(dx[t, i].double() - num) <= 2.0 ** -8 * abs(num) + 1e-5
    for i in (0, 11):
        e = torch.zeros_like(wd)
        e[i] = h
        num = (loss(sd, wd + e) - loss(sd, wd - e)) / (2 * h)
        assert abs(dw[i].double() - num) <= 1e-5


def test_backward_in_place_and_strided():
    T, H = 300, 520
    dy, s, w = _rows(31, T, H, 0.01, stride=528), _rows(32, T, H, 2.0, stride=640), _weight(H)
    r = ops.rms_norm(s, w, EPS, rstd=True)["rstd"]
    d = _rows(33, T, H, 0.01, stride=520).contiguous()
    want, want_w = ops.rms_norm_backward(dy, s, w, r, dresidual=d)
    got, got_w = ops.rms_norm_backward(dy, s, w, r, dresidual=d, dx=d)
    assert got is d and torch.equal(d, want) and torch.equal(got_w, want_w)
    got, got_w = ops.rms_norm_backward(dy, s, w, r, dx=dy)
    assert torch.equal(got_w, want_w)


# ----------------------------------------------------------------------------- rows
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (130, 7168), (7, 2064), (1000, 256), (1, 20000)])
def test_rows_round_trip(rows, cols):
    x = _rows(41, rows, cols, 0.5, stride=cols + 8)
    x[0, 0] = 448.0    # a scale border: amax / 448 is a power of two
    codes, scales = ops.quantize_rows_fp8(x)
    rc, rs = quantize_rows(x)
    assert torch.equal(scales, rs) and torch.equal(codes, rc)
    back = ops.dequantize_rows_fp8(codes, scales)
    assert torch.equal(back.double(), row_values(codes, scales))
    wide = torch.full((rows, cols + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    ops.dequantize_rows_fp8(codes, scales, out=wide[:, :cols])
    assert torch.equal(wide[:, :cols], back) and (wide[:, cols:] == 3).all()


def test_rows_with_non_finite_tiny_and_huge_values():
    x = torch.zeros((6, 256), dtype=torch.bfloat16, device="cuda")
    x[1, 0], x[1, 1] = float("nan"), 2.0
    x[2, 0], x[2, 1] = float("inf"), -3.0
    x[3, 0] = torch.finfo(torch.bfloat16).max
    x[4, 130] = 1e-30
    x[5, :] = -torch.finfo(torch.bfloat16).tiny
    codes, scales = ops.quantize_rows_fp8(x)
    rc, rs = quantize_rows(x)
    assert torch.equal(scales, rs)
    nan = (rc & 127) == 127
    assert int(nan.sum()) == 2 and torch.equal((codes & 127) == 127, nan)
    assert torch.equal(decode_sign_free(codes[~nan]), decode_sign_free(rc[~nan]))
    back = ops.dequantize_rows_fp8(codes, scales)
    assert torch.isnan(back[1, 0]) and back[1, 1] == 2 and torch.isnan(back[2, 0]) and back[2, 1] == -3


def decode_sign_free(c):
    """Codes with -0 and +0 alike."""
    return torch.where((c & 127) == 0, torch.zeros_like(c), c)


def test_scale_layout_is_the_layers_own():
    """The rows that the layer quantises inside its pipeline have these codes and scales."""
    from moe_layer_top_b200 import inputs
    cfg = inputs.make_custom_config("rows", E=4, topk=1, H=512, I=128, fp8=True, routing="logits")
    T = 24
    w13, w2 = inputs.make_weights(cfg, 0, device="cuda")
    q13, s13 = ops.quantize_weights_fp8(w13)
    q2, s2 = ops.quantize_weights_fp8(w2)
    x = inputs.make_tokens(cfg, T, 0, device="cuda")
    logits = inputs.make_routing(cfg, T, 0, device="cuda")["logits"]
    p = ops.problem(T, cfg.E, 1, cfg.H, cfg.I, fp8=True, mode=ops.MODE_NORMAL)
    ws = ops.alloc_workspace(p)
    ops.fused_forward(p, x, q13, q2, logits=logits, w13_scale=s13, w2_scale=s2, ws=ws)
    v = ops.workspace_views(p, ws)
    pos = v["pos_of_flat"].long()
    codes, scales = ops.quantize_rows_fp8(x)
    assert torch.equal(v["a1"][pos], codes)
    assert torch.equal(v["a1_scale_t"][:, pos], scales)
