"""The stand-alone operators at the ends of what they document, on the GPU."""

import pytest
import torch

from moe_layer_top_b200 import ops
from tests.operator_helpers import assert_within, product_bound

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
