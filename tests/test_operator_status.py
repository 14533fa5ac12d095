"""The status word of the stand-alone operators that are given none."""

import ctypes
import os

import pytest
import torch

from moe_layer_top_b200 import ops


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ops.library_path()):
        from moe_layer_top_b200 import build
        build.build()
    return ops.lib()


def test_refusals(L):
    assert L.moe_operator_status(0, None, None) == ops.MOE_ERR_INVALID
    assert L.moe_operator_status_word(None) == ops.MOE_ERR_INVALID
    assert b"operator_status" in L.moe_last_error_string()


def _word():
    w = ctypes.c_void_p()
    assert ops.lib().moe_operator_status_word(ctypes.byref(w)) == ops.MOE_OK
    return w


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_read_and_cleared(L):
    assert ops.operator_status() == ops.MOE_STATUS_OK
    waited = torch.zeros((1,), dtype=torch.int64, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.moe_selftest_wait_timeout(1000, _word(), waited.data_ptr(), stream) == ops.MOE_OK
    code = ops.MOE_STATUS_WAIT_TIMEOUT | 0x7F
    assert ops.operator_status(clear=False) == code and ops.operator_status("cuda:0") == code
    assert ops.operator_status() == ops.MOE_STATUS_OK


@pytest.mark.gpu
def test_a_product_leaves_the_word_as_it_is(L):
    """The word keeps the first failure: later calls neither clear nor overwrite it, and their results are right."""
    x, w = torch.randn((40, 256), device="cuda").bfloat16(), torch.randn((1, 64, 256), device="cuda").bfloat16()
    want = ops.grouped_matmul(x, w, None)
    assert ops.operator_status() == ops.MOE_STATUS_OK
    waited = torch.zeros((1,), dtype=torch.int64, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.moe_selftest_wait_timeout(1000, _word(), waited.data_ptr(), stream) == ops.MOE_OK
    assert torch.equal(ops.grouped_matmul(x, w, None), want)
    assert ops.operator_status() == ops.MOE_STATUS_WAIT_TIMEOUT | 0x7F


_FIRST_CALL = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
from moe_layer_top_b200 import ops
x, w = torch.ones((40, 256), device="cuda").bfloat16(), torch.ones((1, 64, 256), device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = ops.grouped_matmul(x, w, None)
g.replay()
torch.cuda.synchronize()
assert (y == 256).all() and ops.operator_status() == 0
print("FIRST-CALL-OK")
"""


@pytest.mark.gpu
def test_the_first_call_of_a_process_may_be_a_captured_one():
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", _FIRST_CALL, root], capture_output=True, text=True, timeout=240)
    assert res.returncode == 0 and "FIRST-CALL-OK" in res.stdout, res.stderr[-2000:]
