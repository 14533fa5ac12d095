"""The stand-alone operators refuse bad arguments on the host, before anything touches a device (no
GPU needed)."""

import ctypes
import os

import pytest
import torch

from moe_layer_top_b200 import ops

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ops.library_path()):
        from moe_layer_top_b200 import build
        build.build()
    return ops.lib()


def _fake(v=1 << 20):
    return ctypes.c_void_p(v)


G = _fake()
ODD = _fake((1 << 20) + 8)       # 8-byte aligned only
BYTE = _fake((1 << 20) + 2)


def _norm(L, x=G, ldx=256, res=G, ldr=256, ro=G, ldo=256, w=G, eps=1e-6, T=4, H=256, y=G, ldy=256, c=None, s=None,
          r=None):
    return L.moe_rms_norm(x, ldx, res, ldr, ro, ldo, w, eps, T, H, y, ldy, c, s, r, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=12), dict(H=-8), dict(H=16392, ldx=16392, ldr=16392, ldo=16392, ldy=16392),
    dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(x=None), dict(x=ODD), dict(w=None), dict(w=ODD),
    dict(ldx=248), dict(ldx=260), dict(ldr=0), dict(ldo=255), dict(ldy=128), dict(ldx=1 << 40),
    dict(res=None), dict(ro=None), dict(res=ODD), dict(ro=ODD), dict(y=ODD), dict(res=None, ro=None, y=None),
    dict(c=G), dict(s=G), dict(c=ODD, s=G), dict(c=G, s=BYTE), dict(r=BYTE),
    dict(c=G, s=G, H=264, ldx=264, ldr=264, ldo=264, ldy=264),
])
def test_rms_norm(L, kw):
    assert _norm(L, **kw) == ops.MOE_ERR_INVALID
    assert b"rms_norm" in L.moe_last_error_string()


def _norm_backward(L, dy=G, lddy=256, s=G, lds=256, w=G, r=G, dr=None, lddr=0, T=4, H=256, dx=G, lddx=256, dw=G,
                   ws=G, n=1 << 30):
    return L.moe_rms_norm_backward(dy, lddy, s, lds, w, r, dr, lddr, T, H, dx, lddx, dw, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=12), dict(H=16400), dict(dy=None), dict(dy=ODD), dict(s=None), dict(lds=8), dict(lddy=260),
    dict(w=None), dict(r=None), dict(r=BYTE), dict(dr=G, lddr=0), dict(dr=ODD, lddr=256), dict(dx=None),
    dict(lddx=248), dict(dw=None), dict(dw=BYTE), dict(ws=None), dict(ws=ODD),
])
def test_rms_norm_backward(L, kw):
    assert _norm_backward(L, **kw) == ops.MOE_ERR_INVALID


def test_rms_norm_backward_workspace(L):
    assert L.moe_rms_norm_backward_workspace_size(3, 4096) == 3 * 4096 * 4
    assert L.moe_rms_norm_backward_workspace_size(0, 256) == 0
    assert L.moe_rms_norm_backward_workspace_size(1 << 20, 256) == L.moe_rms_norm_backward_workspace_size(1 << 19, 256)
    assert L.moe_rms_norm_backward_workspace_size(4, 100) == 0
    need = L.moe_rms_norm_backward_workspace_size(4, 256)
    assert _norm_backward(L, n=need - 1) == ops.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=24), dict(cols=(1 << 20) + 16),
                                dict(x=None), dict(x=ODD), dict(ldx=128), dict(ldx=260), dict(c=None), dict(c=ODD),
                                dict(s=None), dict(s=BYTE)])
def test_row_format(L, kw):
    a = dict(x=G, ldx=256, rows=4, cols=256, c=G, s=G)
    a.update(kw)
    assert L.moe_quantize_rows_fp8(a["x"], a["ldx"], a["rows"], a["cols"], a["c"], a["s"], None) == ops.MOE_ERR_INVALID
    assert L.moe_dequantize_rows_fp8(a["c"], a["s"], a["rows"], a["cols"], a["x"], a["ldx"],
                                     None) == ops.MOE_ERR_INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(G=0), -1), (dict(G=1025), -1), (dict(N=0), -1), (dict(N=12), -1), (dict(K=0), -1),
    (dict(K=20), -1), (dict(off=None), -1), (dict(off=BYTE), -1), (dict(a=None), -1), (dict(a=ODD), -1),
    (dict(lda=8), -1), (dict(lda=260), -1), (dict(b=None), -1), (dict(b=ODD), -1), (dict(out=None), -1),
    (dict(out=ODD), -1), (dict(ldo=8), -1), (dict(ldo=258), -1), (dict(dtype=1), -2), (dict(dtype=7), -2),
    (dict(M=2 ** 31 - 1, N=1 << 20, lda=1 << 20, ldb=1 << 20, ldo=1 << 20), -1),
])
def test_grouped_products(L, kw, code):
    a = dict(a=G, lda=256, b=G, ldb=256, off=G, M=10, G=4, N=256, K=256, out=G, ldo=256, dtype=0)
    a.update(kw)
    sizes = (a["M"], a["G"], a["N"], a["K"])
    tail = (a["out"], a["ldo"], a["dtype"], None, None)
    assert L.moe_grouped_matmul(a["a"], a["lda"], a["b"], a["off"], *sizes, *tail) == code
    assert b"grouped_matmul" in L.moe_last_error_string()
    assert L.moe_grouped_matmul_dx(a["a"], a["lda"], a["b"], a["off"], *sizes, *tail) == code
    if "ldo" in kw:
        return
    assert L.moe_grouped_matmul_dw(a["a"], a["lda"], a["b"], a["ldb"], a["off"], *sizes, a["out"], a["dtype"], 0, None,
                                   None) == code


@pytest.mark.parametrize("kw", [dict(M=2 ** 30 + 1, N=8, K=8), dict(M=2 ** 31 - 1, N=8, K=8), dict(M=8, N=2 ** 30 + 8, K=8),
                                dict(M=8, N=8, K=2 ** 31 - 8), dict(M=8, N=8, K=8, status=BYTE)])
def test_products_whose_positions_leave_32_bits(L, kw):
    a = {"status": None, **kw}
    ld, sizes = 2 ** 31, (a["M"], 1, a["N"], a["K"])
    tail = (G, ld, 0, a["status"], None)
    assert L.moe_grouped_matmul(G, ld, G, G, *sizes, *tail) == ops.MOE_ERR_INVALID
    assert L.moe_grouped_matmul_dx(G, ld, G, G, *sizes, *tail) == ops.MOE_ERR_INVALID
    assert L.moe_grouped_matmul_dw(G, ld, G, ld, G, *sizes, G, 0, 0, a["status"], None) == ops.MOE_ERR_INVALID
    k = max(a["K"] // 16 * 16, 16)
    assert L.moe_matmul_fp8(G, G, G, G, a["M"], a["N"], k, *tail) == ops.MOE_ERR_INVALID


def test_backward_workspace_of_the_most_rows(L):
    most = L.moe_rms_norm_backward_workspace_size(1 << 24, 8)
    assert L.moe_rms_norm_backward_workspace_size(2 ** 31 - 1, 8) == most > 0


def test_accumulated_gradient_needs_fp32(L):
    args = (G, 256, G, 256, G, 10, 4, 256, 256, G)
    assert L.moe_grouped_matmul_dw(*args, ops.DTYPE_BF16, 1, None, None) == ops.MOE_ERR_UNSUPPORTED
    assert L.moe_grouped_matmul_dw(*args, ops.DTYPE_FP32, 2, None, None) == ops.MOE_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(K=24), dict(K=8), dict(xs=None), dict(xs=BYTE), dict(ws=None), dict(x=ODD),
                                dict(w=None), dict(y=ODD), dict(ldy=128), dict(N=4), dict(M=-1)])
def test_fp8_products(L, kw):
    a = dict(x=G, xs=G, w=G, ws=G, M=10, N=256, K=256, y=G, ldy=256)
    a.update(kw)
    head = (a["x"], a["xs"], a["w"], a["ws"])
    assert L.moe_matmul_fp8(*head, a["M"], a["N"], a["K"], a["y"], a["ldy"], 0, None, None) == ops.MOE_ERR_INVALID
    assert L.moe_grouped_matmul_fp8(*head, G, a["M"], 3, a["N"], a["K"], a["y"], a["ldy"], 0, None,
                                    None) == ops.MOE_ERR_INVALID


def test_no_rows_is_a_no_op(L):
    assert _norm(L, T=0, x=None, y=None, res=None, ro=None, w=None) == ops.MOE_OK
    assert L.moe_quantize_rows_fp8(None, 256, 0, 256, None, None, None) == ops.MOE_OK
    assert L.moe_grouped_matmul(None, 256, None, G, 0, 4, 256, 256, None, 256, 0, None, None) == ops.MOE_OK


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: ops.rms_norm(_cpu(4, 64), _cpu(64)),
    lambda: ops.rms_norm(_cpu(64), _cpu(64)),
    lambda: ops.rms_norm_backward(_cpu(4, 64), _cpu(4, 64), _cpu(64), _cpu(4, dtype=torch.float32)),
    lambda: ops.quantize_rows_fp8(_cpu(4, 64, dtype=torch.float16)),
    lambda: ops.dequantize_rows_fp8(_cpu(4, 64), _cpu(1, 4, dtype=torch.float32)),
    lambda: ops.matmul_fp8(_cpu(4, 64), _cpu(1, 4), _cpu(8, 64), _cpu(1, 1)),
    lambda: ops.grouped_matmul(_cpu(4, 64), _cpu(2, 8, 64), None),
    lambda: ops.grouped_matmul(_cpu(4, 64), _cpu(8, 64), None),
    lambda: ops.grouped_matmul_dx(_cpu(4, 8), _cpu(2, 8, 64), None),
    lambda: ops.grouped_matmul_dw(_cpu(4, 8), _cpu(4, 64), None),
    lambda: ops.rms_norm("x", _cpu(64)),
    lambda: ops.rms_norm(_cpu(4, 64), _cpu(64), stream=0),
    lambda: ops.quantize_rows_fp8(_cpu(4, 64), 7),
])
def test_python_refuses_other_tensors(call):
    with pytest.raises(ValueError):
        call()
