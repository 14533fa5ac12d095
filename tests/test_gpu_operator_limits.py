"""The stand-alone operators at the ends of what they document, on the GPU."""

import pytest
import torch

from moe_layer_top_b200 import ops
from tests.operator_helpers import assert_within, product_bound, row_values

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


def test_a_reduction_that_takes_longer_than_the_limit_of_a_wait():
    """One group with nearly all of 2^30 rows, whose one tile takes one SM seconds: the limit of the waits for it
    counts from the last progress.  All but a few rows are zeros, which add nothing, so the sum has as many terms."""
    M, N, K, G, g = 1 << 30, 8, 8, 80, 3
    if torch.cuda.mem_get_info()[0] < (44 << 30):
        pytest.skip("not enough free memory")
    rows = torch.tensor([5, 63, 64, 1 << 20, (1 << 29) + 1, M - 70, M - 6], device="cuda")
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    dy[rows], x[rows] = _randn(1, len(rows), N), _randn(2, len(rows), K)
    off = torch.zeros((G + 1,), dtype=torch.int32, device="cuda")
    off[g + 1:] = M - 5
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    dw = ops.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32, status=status)
    a, b = dy[rows].double(), x[rows].double()
    assert int(status) == 0
    assert_within(dw[g], a.t() @ b, product_bound(a.t() @ b, a.abs().t() @ b.abs(), len(rows), torch.float32))
    assert not dw[:g].any() and not dw[g + 1:].any()


@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 127, 3.0e38])
def test_codes_past_bf16_are_read_back_finite(scale):
    """Every code at the largest scales: the bf16 value, or bf16's largest finite number; NaN codes stay NaN."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 128)
    scales = torch.full((1, 2), scale, device="cuda")
    want = row_values(codes, scales)
    most = torch.finfo(torch.bfloat16).max
    back = ops.dequantize_rows_fp8(codes, scales).double()
    nan = torch.isnan(want)
    assert int(nan.sum()) == 2 and torch.equal(torch.isnan(back), nan)
    assert torch.equal(back[~nan], want[~nan].clamp(-most, most).to(torch.bfloat16).double())


def test_the_largest_rows_read_back_finite():
    """x / 2^120 = 248 .. 255 rounds to the code of 256, which is 2^128."""
    x = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    most = torch.finfo(torch.bfloat16).max
    x[0, 3], x[1, 200], x[2, 7] = most, -248 * 2.0 ** 120, 247 * 2.0 ** 120
    back = ops.dequantize_rows_fp8(*ops.quantize_rows_fp8(x))
    assert back[0, 3] == most and back[1, 200] == -most and back[2, 7] == 240 * 2.0 ** 120
    assert torch.isfinite(back).all()
