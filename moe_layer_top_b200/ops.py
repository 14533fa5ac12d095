"""ctypes binding of ``libmoe_b200.so`` (argument marshalling only).

Every function here forwards torch tensors' device pointers and sizes to the C
ABI declared in ``include/moe_b200.h``; all computation happens in the CUDA
kernels.  The library is loaded on first use; if it is missing or cannot be
loaded the call raises ``RuntimeError`` -- there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_b200.so")
_lib = None
_lock = threading.Lock()

MOE_OK = 0
MOE_ERR_INVALID = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4

MOE_STATUS_OK = 0
MOE_STATUS_BAD_EXPERT_ID = 1
MOE_STATUS_WAIT_TIMEOUT = 0x100

DTYPE_BF16 = 0
DTYPE_FP8_E4M3 = 1
DTYPE_MXFP8_E4M3 = 2
DTYPE_FP32 = 3

MODE_AUTO = 0
MODE_NORMAL = 1
MODE_SWAP_AB = 2

STAGE_ROUTE, STAGE_ALIGN, STAGE_GATHER, STAGE_GEMM1, STAGE_GEMM2, STAGE_COMBINE = range(6)
NUM_STAGES = 6
STAGE_NAMES = ("route", "align", "gather", "gemm1", "gemm2", "combine")

EXPORTED = (
    "moe_last_error_string", "moe_route", "moe_align_capacity", "moe_align_workspace_size", "moe_align",
    "moe_quantize_weights_fp8", "moe_resolve_problem", "moe_workspace_size", "moe_get_workspace_layout",
    "moe_fused_forward", "moe_forward_stages", "moe_read_status", "moe_version", "moe_align_noalloc",
    "moe_selftest_wait_timeout", "moe_quantize_weights_mxfp8", "moe_combine_allreduce_flag_count",
    "moe_combine_allreduce", "moe_combine_allreduce_emulated", "moe_combine_reduce_scatter_flag_count",
    "moe_combine_reduce_scatter", "moe_combine_reduce_scatter_emulated", "moe_rms_norm",
    "moe_rms_norm_backward_workspace_size", "moe_rms_norm_backward", "moe_quantize_rows_fp8",
    "moe_dequantize_rows_fp8", "moe_grouped_matmul", "moe_grouped_matmul_fp8", "moe_grouped_matmul_dx",
    "moe_grouped_matmul_dw", "moe_matmul_fp8", "moe_operator_status", "moe_operator_status_word",
)

MAX_RANKS = 16


class MoeProblem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("H", ctypes.c_int32),
        ("I", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("mode", ctypes.c_int32),
        ("block_m", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("split_k", ctypes.c_int32),
        ("router_weight_on_input", ctypes.c_int32), ("swiglu_limit", ctypes.c_float),
        ("persistent_decode", ctypes.c_int32), ("num_global_experts", ctypes.c_int32),
        ("first_expert", ctypes.c_int32), ("reserved", ctypes.c_int32 * 1),
    ]


class MoeAllreduceRank(ctypes.Structure):
    _fields_ = [("y", ctypes.c_void_p), ("pos_of_flat", ctypes.c_void_p), ("partial", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("flags", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class MoeWorkspaceLayout(ctypes.Structure):
    _fields_ = [
        ("status", ctypes.c_int64), ("topk_ids", ctypes.c_int64), ("topk_weights", ctypes.c_int64),
        ("sorted_token_ids", ctypes.c_int64), ("expert_ids", ctypes.c_int64),
        ("num_tokens_post_padded", ctypes.c_int64), ("expert_counts", ctypes.c_int64),
        ("expert_offsets", ctypes.c_int64), ("align_scratch", ctypes.c_int64), ("pos_of_flat", ctypes.c_int64),
        ("a1", ctypes.c_int64),
        ("a1_scale", ctypes.c_int64), ("a2", ctypes.c_int64), ("a2_scale", ctypes.c_int64), ("y", ctypes.c_int64),
        ("partials", ctypes.c_int64), ("total_bytes", ctypes.c_int64), ("capacity", ctypes.c_int32), ("block_m", ctypes.c_int32),
        ("mode", ctypes.c_int32), ("align_chunks", ctypes.c_int32),
    ]


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded C library (raises if it is not built or cannot be loaded)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built: run `python -m moe_layer_top_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER(MoeProblem)
        sig = {
            "moe_last_error_string": (ctypes.c_char_p, []),
            "moe_version": (i32, []),
            "moe_route": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp]),
            "moe_align_capacity": (i64, [i32, i32, i32, i32]),
            "moe_align_workspace_size": (sz, [i32, i32, i32]),
            "moe_align": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_align_noalloc": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]),
            "moe_quantize_weights_fp8": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, vp]),
            "moe_quantize_weights_mxfp8": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, vp]),
            "moe_resolve_problem": (ctypes.c_int, [P]),
            "moe_workspace_size": (sz, [P]),
            "moe_get_workspace_layout": (ctypes.c_int, [P, ctypes.POINTER(MoeWorkspaceLayout)]),
            "moe_fused_forward": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_forward_stages": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i32, i32, vp]),
            "moe_read_status": (ctypes.c_int, [P, vp, i32, ctypes.POINTER(i32), vp]),
            "moe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, vp, vp, vp]),
            "moe_combine_allreduce_flag_count": (i32, [i32, i32]),
            "moe_combine_allreduce": (ctypes.c_int, [i32, i32, i32, i32, i32, ctypes.POINTER(MoeAllreduceRank),
                                                     ctypes.c_uint32, ctypes.c_uint32, vp]),
            "moe_combine_allreduce_emulated": (ctypes.c_int, [i32, i32, i32, i32, ctypes.POINTER(MoeAllreduceRank),
                                                              ctypes.c_uint32, ctypes.c_uint32, vp]),
            "moe_combine_reduce_scatter_flag_count": (i32, [i32, i32]),
            "moe_combine_reduce_scatter": (ctypes.c_int, [i32, i32, i32, i32, i32,
                                                          ctypes.POINTER(MoeAllreduceRank), ctypes.c_uint32,
                                                          ctypes.c_uint32, vp]),
            "moe_combine_reduce_scatter_emulated": (ctypes.c_int, [i32, i32, i32, i32,
                                                                   ctypes.POINTER(MoeAllreduceRank),
                                                                   ctypes.c_uint32, ctypes.c_uint32, vp]),
            "moe_rms_norm": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, ctypes.c_float, i32, i32, vp, i64, vp, vp,
                                            vp, vp]),
            "moe_rms_norm_backward_workspace_size": (sz, [i32, i32]),
            "moe_rms_norm_backward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, i64, i32, i32, vp, i64, vp, vp,
                                                     sz, vp]),
            "moe_quantize_rows_fp8": (ctypes.c_int, [vp, i64, i64, i32, vp, vp, vp]),
            "moe_dequantize_rows_fp8": (ctypes.c_int, [vp, vp, i64, i32, vp, i64, vp]),
            "moe_grouped_matmul": (ctypes.c_int, [vp, i64, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp]),
            "moe_grouped_matmul_fp8": (ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp]),
            "moe_grouped_matmul_dx": (ctypes.c_int, [vp, i64, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp]),
            "moe_grouped_matmul_dw": (ctypes.c_int, [vp, i64, vp, i64, vp, i32, i32, i32, i32, vp, i32, i32, vp,
                                                     vp]),
            "moe_matmul_fp8": (ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, vp, i64, i32, vp, vp]),
            "moe_operator_status": (ctypes.c_int, [i32, ctypes.POINTER(i32), vp]),
            "moe_operator_status_word": (ctypes.c_int, [ctypes.POINTER(vp)]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moe error {code}: {msg}")
        self.code = code


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, lib().moe_last_error_string().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def problem(T, E, topk, H, I, fp8=False, mode=MODE_AUTO, block_m=0, renormalize=True, split_k=True,
            mx=False, router_weight_on_input=False, swiglu_limit=0.0, persistent_decode=False,
            num_global_experts=0, first_expert=0) -> MoeProblem:
    """A moe_problem; ``fp8`` selects E4M3 weights with 128x128 fp32 block scales, ``mx`` MXFP8
    (E4M3 with per-32 E8M0 scales); ``router_weight_on_input`` (top-1 only) scales x by the router
    weight before GEMM1; ``swiglu_limit`` > 0 clamps gate and up before the activation.
    Expert parallelism: ``E`` experts held here, global experts ``[first_expert, first_expert + E)``
    of ``num_global_experts`` that the router scores (0 = ``E``)."""
    p = MoeProblem()
    p.num_global_experts, p.first_expert = int(num_global_experts), int(first_expert)
    p.T, p.E, p.topk, p.H, p.I = int(T), int(E), int(topk), int(H), int(I)
    p.weight_dtype = DTYPE_MXFP8_E4M3 if mx else (DTYPE_FP8_E4M3 if fp8 else DTYPE_BF16)
    p.router_weight_on_input = 1 if router_weight_on_input else 0
    p.swiglu_limit = float(swiglu_limit)
    p.persistent_decode = 1 if persistent_decode else 0
    p.mode, p.block_m, p.renormalize = int(mode), int(block_m), 1 if renormalize else 0
    p.split_k = 0 if split_k else 1
    return p


def resolve_problem(p: MoeProblem) -> MoeProblem:
    q = MoeProblem.from_buffer_copy(p)
    _check(lib().moe_resolve_problem(ctypes.byref(q)))
    return q


def workspace_size(p: MoeProblem) -> int:
    n = lib().moe_workspace_size(ctypes.byref(p))
    if n == 0 and p.T > 0:
        _check(lib().moe_resolve_problem(ctypes.byref(MoeProblem.from_buffer_copy(p))))
    return int(n)


def workspace_layout(p: MoeProblem) -> MoeWorkspaceLayout:
    L = MoeWorkspaceLayout()
    _check(lib().moe_get_workspace_layout(ctypes.byref(p), ctypes.byref(L)))
    return L


def alloc_workspace(p: MoeProblem, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of moe_workspace_size(p) bytes (torch allocations are 256-byte aligned)."""
    return torch.empty(max(workspace_size(p), 256), dtype=torch.uint8, device=device)


def route(logits: torch.Tensor, topk: int, renormalize=True, stream=None):
    T, E = logits.shape
    ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route(_ptr(logits.contiguous()), T, E, topk, 1 if renormalize else 0, _ptr(ids), _ptr(w),
                           _stream(stream)))
    return ids, w


def align_capacity(T, topk, E, block_m) -> int:
    return int(lib().moe_align_capacity(T, topk, E, block_m))


def align(topk_ids: torch.Tensor, E: int, block_m: int, stream=None):
    T, k = topk_ids.shape
    dev = topk_ids.device
    cap = align_capacity(T, k, E, block_m)
    sorted_ids = torch.empty((max(cap, 1),), dtype=torch.int32, device=dev)[:cap]
    expert_ids = torch.empty((max(cap // block_m, 1),), dtype=torch.int32, device=dev)[:cap // block_m]
    ntpp = torch.empty((1,), dtype=torch.int32, device=dev)
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    ws = torch.empty((max(int(lib().moe_align_workspace_size(T, k, E)), 256),), dtype=torch.uint8, device=dev)
    _check(lib().moe_align(_ptr(topk_ids.contiguous()), T, k, E, block_m, _ptr(sorted_ids), _ptr(expert_ids),
                           _ptr(ntpp), _ptr(counts), _ptr(offsets), _ptr(ws), ws.numel(), _stream(stream)))
    return {"sorted_token_ids": sorted_ids, "expert_ids": expert_ids, "num_tokens_post_padded": ntpp,
            "expert_counts": counts, "expert_offsets": offsets, "capacity": cap, "workspace": ws}


def quantize_weights_fp8(w: torch.Tensor, stream=None):
    """bf16 [..., rows, cols] -> (E4M3 codes as uint8 [..., rows, cols], fp32 scales [..., rows/128, cols/128])."""
    w = w.contiguous()
    *lead, rows, cols = w.shape
    batches = 1
    for d in lead:
        batches *= d
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty((*lead, rows // 128, cols // 128), dtype=torch.float32, device=w.device)
    _check(lib().moe_quantize_weights_fp8(_ptr(w), batches, rows, cols, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def quantize_weights_mxfp8(w: torch.Tensor, stream=None):
    """bf16 [..., rows, cols] -> (E4M3 codes uint8 [..., rows, cols], E8M0 scale factors uint8
    [..., rows * cols / 32] in the SF-atom layout of the header)."""
    w = w.contiguous()
    *lead, rows, cols = w.shape
    batches = 1
    for d in lead:
        batches *= d
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    sf = torch.empty((*lead, rows * cols // 32), dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize_weights_mxfp8(_ptr(w), batches, rows, cols, _ptr(codes), _ptr(sf), _stream(stream)))
    return codes, sf


def sf_atoms_to_rows(sf_atoms: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Re-index SF atoms of [.., rows, cols] into the natural [.., rows, cols/32] order (for tests and tools)."""
    lead = sf_atoms.shape[:-1]
    a = sf_atoms.reshape(*lead, rows // 128, cols // 128, 32, 4, 4)      # [rb, kb, n%32, (n%128)/32, k-group]
    a = a.permute(*range(len(lead)), len(lead), len(lead) + 3, len(lead) + 2, len(lead) + 1, len(lead) + 4)
    return a.reshape(*lead, rows, cols // 32)


def _forward_args(p, x, logits, topk_ids, topk_weights, w13, w2, w13_scale, w2_scale, out, ws):
    return (ctypes.byref(p), _ptr(x), _ptr(logits), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(w2),
            _ptr(w13_scale), _ptr(w2_scale), _ptr(out), _ptr(ws), ws.numel())


def fused_forward(p: MoeProblem, x, w13, w2, *, logits=None, topk_ids=None, topk_weights=None, w13_scale=None,
                  w2_scale=None, out=None, ws=None, stream=None):
    """Run the whole layer; returns ``out`` [T, H] bf16 (allocated if not given)."""
    if out is None:
        out = torch.empty((p.T, p.H), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = alloc_workspace(p, x.device)
    _check(lib().moe_fused_forward(*_forward_args(p, x, logits, topk_ids, topk_weights, w13, w2, w13_scale, w2_scale,
                                                  out, ws), _stream(stream)))
    return out


def forward_stages(p: MoeProblem, x, w13, w2, begin: int, end: int, *, logits=None, topk_ids=None,
                   topk_weights=None, w13_scale=None, w2_scale=None, out=None, ws=None, stream=None):
    _check(lib().moe_forward_stages(*_forward_args(p, x, logits, topk_ids, topk_weights, w13, w2, w13_scale,
                                                   w2_scale, out, ws), begin, end, _stream(stream)))
    return out


def read_status(p: MoeProblem, ws, clear=True, stream=None) -> int:
    st = ctypes.c_int32(-1)
    _check(lib().moe_read_status(ctypes.byref(p), _ptr(ws), 1 if clear else 0, ctypes.byref(st), _stream(stream)))
    return int(st.value)


def workspace_views(p: MoeProblem, ws: torch.Tensor) -> dict:
    """Typed views of the intermediates inside a workspace (for tests and tools)."""
    q = resolve_problem(p)
    L = workspace_layout(q)
    nflat = q.T * q.topk
    cap = L.capacity
    mx = q.weight_dtype == DTYPE_MXFP8_E4M3
    fp8 = q.weight_dtype == DTYPE_FP8_E4M3 or mx
    a1_rows = q.T if q.mode == MODE_SWAP_AB else cap

    def view(off, n, dtype, shape):
        if off < 0:
            return None
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype).reshape(shape)

    return {
        "status": view(L.status, 1, torch.int32, (1,)),
        "topk_ids": view(L.topk_ids, nflat, torch.int32, (q.T, q.topk)),
        "topk_weights": view(L.topk_weights, nflat, torch.float32, (q.T, q.topk)),
        "sorted_token_ids": view(L.sorted_token_ids, cap, torch.int32, (cap,)),
        "expert_ids": view(L.expert_ids, cap // q.block_m, torch.int32, (cap // q.block_m,)),
        "num_tokens_post_padded": view(L.num_tokens_post_padded, 1, torch.int32, (1,)),
        "expert_counts": view(L.expert_counts, q.E, torch.int32, (q.E,)),
        "expert_offsets": view(L.expert_offsets, q.E + 1, torch.int32, (q.E + 1,)),
        # GEMM1 token rows: sorted copy [cap, H] for normal tiles, one row per token [T, H] for swap-AB
        "a1": view(L.a1, a1_rows * q.H, torch.uint8 if fp8 else torch.bfloat16, (a1_rows, q.H)),
        "pos_of_flat": view(L.pos_of_flat, nflat, torch.int32, (nflat,)),
        "a1_scale_t": None if mx else view(L.a1_scale, cap * (q.H // 128), torch.float32, (q.H // 128, cap)),
        "a1_sf": view(L.a1_scale, cap * q.H // 32, torch.uint8, (cap * q.H // 32,)) if mx else None,
        "a2": view(L.a2, cap * q.I, torch.uint8 if fp8 else torch.bfloat16, (cap, q.I)),
        "a2_scale_t": None if mx else view(L.a2_scale, cap * (q.I // 128), torch.float32, (q.I // 128, cap)),
        "a2_sf": view(L.a2_scale, cap * q.I // 32, torch.uint8, (cap * q.I // 32,)) if mx else None,
        "y": view(L.y, nflat * q.H, torch.bfloat16, (nflat, q.H)),
        "partials": view(L.partials, (L.total_bytes - L.partials) // 4, torch.float32, (-1,)),
        "layout": L,
        "problem": q,
    }


def selftest_wait_timeout(timeout_us: int, stream=None):
    """Run the bounded-wait self-test; returns (status, waited_ns) after a sync."""
    st = torch.zeros((1,), dtype=torch.int32, device="cuda")
    waited = torch.zeros((1,), dtype=torch.int64, device="cuda")
    _check(lib().moe_selftest_wait_timeout(int(timeout_us), _ptr(st), _ptr(waited), _stream(stream)))
    torch.cuda.synchronize()
    return int(st.item()), int(waited.item())


# ----------------------------------------------------------------------------- fused combine + all-reduce
def combine_allreduce_flag_count(T: int, world: int) -> int:
    """int32 entries of each rank's flags array (zero them once before the first call)."""
    return int(lib().moe_combine_allreduce_flag_count(int(T), int(world)))


def _ranks_array(ranks):
    arr = (MoeAllreduceRank * len(ranks))()
    for i, r in enumerate(ranks):
        for name in ("y", "pos_of_flat", "partial", "out", "flags", "status"):
            v = r.get(name)
            setattr(arr[i], name, None if v is None else (v if isinstance(v, int) else v.data_ptr()))
    return arr


def combine_allreduce(T, topk, H, rank, ranks, epoch, timeout_us=2_000_000, stream=None):
    """This rank's fused combine + all-reduce.  ``ranks``: one dict per rank with ``y``,
    ``pos_of_flat``, ``partial``, ``out``, ``flags``, ``status`` -- tensors, or device addresses
    (ints) of peers' buffers as mapped in this process."""
    arr = _ranks_array(ranks)
    _check(lib().moe_combine_allreduce(int(T), int(topk), int(H), len(ranks), int(rank), arr, int(epoch),
                                       int(timeout_us), _stream(stream)))


def combine_allreduce_emulated(T, topk, H, ranks, epoch, timeout_us=2_000_000, stream=None):
    """Every rank's fused combine + all-reduce in one cooperative launch on this GPU (all buffers local)."""
    arr = _ranks_array(ranks)
    _check(lib().moe_combine_allreduce_emulated(int(T), int(topk), int(H), len(ranks), arr, int(epoch),
                                                int(timeout_us), _stream(stream)))


def combine_reduce_scatter_flag_count(T: int, world: int) -> int:
    """int32 entries of each rank's flags array for the reduce-scatter form (T tokens per rank)."""
    return int(lib().moe_combine_reduce_scatter_flag_count(int(T), int(world)))


def combine_reduce_scatter(T, topk, H, rank, ranks, epoch, timeout_us=2_000_000, stream=None):
    """This rank's fused combine + reduce-scatter (T tokens per rank; partial [world*T, H], out [T, H])."""
    arr = _ranks_array(ranks)
    _check(lib().moe_combine_reduce_scatter(int(T), int(topk), int(H), len(ranks), int(rank), arr, int(epoch),
                                            int(timeout_us), _stream(stream)))


def combine_reduce_scatter_emulated(T, topk, H, ranks, epoch, timeout_us=2_000_000, stream=None):
    """Every rank's fused combine + reduce-scatter in one cooperative launch on this GPU."""
    arr = _ranks_array(ranks)
    _check(lib().moe_combine_reduce_scatter_emulated(int(T), int(topk), int(H), len(ranks), arr, int(epoch),
                                                     int(timeout_us), _stream(stream)))



# ----------------------------------------------------------------------------- stand-alone operators
# Tensors of other types, shapes, devices or layouts than a function documents raise ValueError here; what
# the C ABI checks (sizes, alignment) raises MoeError.  The work runs on `stream`, or on the current stream
# of the tensors' device; outputs and workspaces are allocated for that stream.  A wait inside a product's kernel that
# runs out is recorded in `status` (int32 [1]) or, without it, in the device's word that operator_status() reads.
_OUT_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}


def _refuse(name, t, dtype, shape, device, rows):
    """Raise for a tensor that is not what ``_rows`` or ``_flat`` needs."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: type {t.dtype}, {dtype} is needed")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, needed on the device of the first argument ({device})")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, {tuple(shape)} is needed")
    raise ValueError(f"{name}: " + ("its last dimension must have stride 1" if rows else "must be contiguous"))


def _rows(name, t, dtype, shape, device):
    """(address, elements between rows) of a 2-D tensor of this type, shape and device whose rows are contiguous (a
    single row's stride says nothing)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device):
        _refuse(name, t, dtype, shape, device, True)
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        _refuse(name, t, dtype, shape, device, True)
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _flat(name, t, dtype, shape, device):
    """The address of a contiguous tensor of this type, shape and device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _refuse(name, t, dtype, shape, device, False)
    return t.data_ptr()


def _sizes(name, t, dims=2):
    """The sizes of a call's first argument, a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name}: a {dims}-dimensional tensor is needed")
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, a CUDA tensor is needed")
    return t.shape


def _on(stream, t):
    """The context of a call that was given a stream: what it allocates belongs to that stream, so that neither a
    workspace that it drops nor an output that its caller drops is handed out while the stream still uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        raise ValueError(f"stream: a torch.cuda.Stream is needed, got {type(stream).__name__}")
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream: on {stream.device}, needed on the device of the first argument ({t.device})")
    return torch.cuda.stream(stream)


def _run(fn, device, *args):
    """Call a C entry point on the tensors' device, whichever device is current.  (These calls are as short as
    their kernels: addresses go as plain numbers and the stream is read as one.)"""
    index = device.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _run(fn, device, *args)
    rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        _check(rc)


def _like(x, dtype=None):
    """A new contiguous tensor of x's shape (the cheapest of torch's allocating calls)."""
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _out_dtype(out, out_dtype):
    dtype = out_dtype or (torch.bfloat16 if out is None else getattr(out, "dtype", None))
    if dtype not in _OUT_DTYPES:
        raise ValueError(f"out_dtype: {dtype}, torch.bfloat16 or torch.float32 is needed")
    return dtype


def _out(out, out_dtype, rows, cols, like):
    """The output of a product, new or checked: (tensor, address, elements between rows, type's number)."""
    dtype = _out_dtype(out, out_dtype)
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=like.device)
        return out, out.data_ptr(), cols, _OUT_DTYPES[dtype]
    return out, *_rows("out", out, dtype, (rows, cols), like.device), _OUT_DTYPES[dtype]


def _status(status, dev):
    return None if status is None else _flat("status", status, torch.int32, (1,), dev)


def operator_status(device=None, clear=True, stream=None) -> int:
    """The status of the products that were given no ``status`` on a device (default: the current one) and enqueued on
    ``stream`` (default: its current stream) so far: MOE_STATUS_OK, or the first failure since it was last cleared.
    Waits for the stream."""
    st = ctypes.c_int32(-1)
    with torch.cuda.device(device):
        _check(lib().moe_operator_status(1 if clear else 0, ctypes.byref(st), _stream(stream)))
    return int(st.value)


def _offsets(offsets, G, dev):
    if offsets is None:
        if G != 1:
            raise ValueError(f"offsets: needed for {G} groups")
        return None
    return _flat("offsets", offsets, torch.int32, (G + 1,), dev)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *, residual=None, residual_out=None, y=True,
             fp8=False, rstd=False, stream=None) -> dict:
    """RMS norm of the rows of x [T, H] bf16, after the addition of ``residual`` if given.

    Returns a dict: ``residual`` (bf16(x + residual), written to ``residual_out`` if given, which may be the
    residual itself; None without residual), ``y`` (bf16 [T, H]; True allocates it, a tensor receives it, False
    leaves it out), ``codes`` and ``scales`` (with ``fp8``: the FP8 rows of y, uint8 [T, H] and fp32
    [ceil(H / 128), T]) and ``rstd`` (fp32 [T] if asked for)."""
    if stream is not None:
        with _on(stream, x):
            return rms_norm(x, weight, eps, residual=residual, residual_out=residual_out, y=y, fp8=fp8, rstd=rstd)
    shape = T, H = _sizes("x", x)
    dev, bf16 = x.device, torch.bfloat16
    x_p, x_ld = _rows("x", x, bf16, shape, dev)
    w_p = _flat("weight", weight, bf16, (H,), dev)
    r_p = r_ld = o_p = o_ld = y_p = y_ld = c_p = s_p = rstd_p = codes = scales = None
    if residual is not None:
        r_p, r_ld = _rows("residual", residual, bf16, shape, dev)
        if residual_out is None:
            residual_out = _like(x)
            o_p, o_ld = residual_out.data_ptr(), H
        else:
            o_p, o_ld = _rows("residual_out", residual_out, bf16, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out: given without residual")
    if y is True:
        y = _like(x)
        y_p, y_ld = y.data_ptr(), H
    elif y is False or y is None:
        y = None
    else:
        y_p, y_ld = _rows("y", y, bf16, shape, dev)
    if fp8:
        codes = _like(x, torch.uint8)
        scales = torch.empty((H + 127) // 128, T, dtype=torch.float32, device=dev)
        c_p, s_p = codes.data_ptr(), scales.data_ptr()
    if rstd:
        rstd = x.new_empty(T, dtype=torch.float32)
        rstd_p = rstd.data_ptr()
    _run(lib().moe_rms_norm, dev, x_p, x_ld, r_p, r_ld or 0, o_p, o_ld or 0, w_p, eps, T, H, y_p, y_ld or 0,
         c_p, s_p, rstd_p)
    return {"residual": residual_out, "y": y, "codes": codes, "scales": scales,
            "rstd": rstd if rstd_p is not None else None}


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *, dresidual=None,
                      dx=None, ws=None, stream=None):
    """Backward pass of :func:`rms_norm`: (dx bf16 [T, H], dweight fp32 [H]).

    ``s`` is what was normalised (x, or the ``residual`` that the forward pass returned), ``dresidual`` the
    gradient that reaches it by other ways; ``ws`` a uint8 workspace of
    ``moe_rms_norm_backward_workspace_size`` bytes (allocated if not given)."""
    if stream is not None:
        with _on(stream, dy):
            return rms_norm_backward(dy, s, weight, rstd, dresidual=dresidual, dx=dx, ws=ws)
    shape = T, H = _sizes("dy", dy)
    dev, bf16 = dy.device, torch.bfloat16
    dy_p, dy_ld = _rows("dy", dy, bf16, shape, dev)
    s_p, s_ld = _rows("s", s, bf16, shape, dev)
    w_p = _flat("weight", weight, bf16, (H,), dev)
    rstd_p = _flat("rstd", rstd, torch.float32, (T,), dev)
    r_p, r_ld = (None, 0) if dresidual is None else _rows("dresidual", dresidual, bf16, shape, dev)
    if dx is None:
        dx = _like(dy)
        dx_p, dx_ld = dx.data_ptr(), H
    else:
        dx_p, dx_ld = _rows("dx", dx, bf16, shape, dev)
    dweight = dy.new_empty(H, dtype=torch.float32)
    L = lib()
    if ws is None:
        ws = dy.new_empty(max(L.moe_rms_norm_backward_workspace_size(T, H), 16), dtype=torch.uint8)
    else:
        _flat("ws", ws, torch.uint8, getattr(ws, "shape", None), dev)
    _run(L.moe_rms_norm_backward, dev, dy_p, dy_ld, s_p, s_ld, w_p, rstd_p, r_p, r_ld, T, H, dx_p, dx_ld,
         dweight.data_ptr(), ws.data_ptr(), ws.numel())
    return dx, dweight


def quantize_rows_fp8(x: torch.Tensor, stream=None):
    """bf16 [rows, cols] -> FP8 rows: (E4M3 codes as uint8 [rows, cols], fp32 scales [ceil(cols / 128), rows])."""
    if stream is not None:
        with _on(stream, x):
            return quantize_rows_fp8(x)
    shape = rows, cols = _sizes("x", x)
    dev = x.device
    x_p, x_ld = _rows("x", x, torch.bfloat16, shape, dev)
    codes = _like(x, torch.uint8)
    scales = torch.empty((cols + 127) // 128, rows, dtype=torch.float32, device=dev)
    _run(lib().moe_quantize_rows_fp8, dev, x_p, x_ld, rows, cols, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def dequantize_rows_fp8(codes: torch.Tensor, scales: torch.Tensor, *, out=None, stream=None):
    """FP8 rows -> the bf16 [rows, cols] values that they stand for."""
    if stream is not None:
        with _on(stream, codes):
            return dequantize_rows_fp8(codes, scales, out=out)
    shape = rows, cols = _sizes("codes", codes)
    dev = codes.device
    c_p = _flat("codes", codes, torch.uint8, shape, dev)
    s_p = _flat("scales", scales, torch.float32, ((cols + 127) // 128, rows), dev)
    if out is None:
        out = _like(codes, torch.bfloat16)
        o_p, o_ld = out.data_ptr(), cols
    else:
        o_p, o_ld = _rows("out", out, torch.bfloat16, shape, dev)
    _run(lib().moe_dequantize_rows_fp8, dev, c_p, s_p, rows, cols, o_p, o_ld)
    return out


def matmul_fp8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *, out=None,
               out_dtype=None, status=None, stream=None):
    """y [M, N] = x . w^T of FP8 rows x [M, K] (codes and scales of :func:`quantize_rows_fp8` or
    :func:`rms_norm`) and a weight w [N, K] with one scale per 128 x 128 block; bf16 or fp32."""
    if stream is not None:
        with _on(stream, x):
            return matmul_fp8(x, x_scale, w, w_scale, out=out, out_dtype=out_dtype, status=status)
    M, K = _sizes("x", x)
    N = _sizes("w", w)[0]
    dev, kb = x.device, (K + 127) // 128
    x_p = _flat("x", x, torch.uint8, (M, K), dev)
    xs_p = _flat("x_scale", x_scale, torch.float32, (kb, M), dev)
    w_p = _flat("w", w, torch.uint8, (N, K), dev)
    ws_p = _flat("w_scale", w_scale, torch.float32, ((N + 127) // 128, kb), dev)
    out, o_p, o_ld, dtype = _out(out, out_dtype, M, N, x)
    _run(lib().moe_matmul_fp8, dev, x_p, xs_p, w_p, ws_p, M, N, K, o_p, o_ld, dtype, _status(status, dev))
    return out


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets, *, x_scale=None, w_scale=None, out=None, out_dtype=None,
                   status=None, stream=None):
    """y[r] = x[r] . w[g]^T for the rows offsets[g] <= r < offsets[g + 1] of every group g.

    x [M, K] bf16 and w [G, N, K] bf16; or FP8 rows x with ``x_scale`` [ceil(K / 128), M] and E4M3 weights with
    ``w_scale`` [G, ceil(N / 128), ceil(K / 128)].  ``offsets`` int32 [G + 1] on the device (None: one group of
    all rows).  y [M, N] bf16 or fp32; rows of no group are not written."""
    if stream is not None:
        with _on(stream, x):
            return grouped_matmul(x, w, offsets, x_scale=x_scale, w_scale=w_scale, out=out, out_dtype=out_dtype,
                                  status=status)
    M, K = _sizes("x", x)
    G, N, _ = _sizes("w", w, 3)
    dev = x.device
    if (x_scale is None) != (w_scale is None):
        raise ValueError("x_scale and w_scale: give both (FP8) or neither (bf16)")
    off_p = _offsets(offsets, G, dev)
    if x_scale is None:
        x_p, x_ld = _rows("x", x, torch.bfloat16, (M, K), dev)
        w_p = _flat("w", w, torch.bfloat16, (G, N, K), dev)
        out, o_p, o_ld, dtype = _out(out, out_dtype, M, N, x)
        _run(lib().moe_grouped_matmul, dev, x_p, x_ld, w_p, off_p, M, G, N, K, o_p, o_ld, dtype,
             _status(status, dev))
        return out
    kb = (K + 127) // 128
    x_p = _flat("x", x, torch.uint8, (M, K), dev)
    w_p = _flat("w", w, torch.uint8, (G, N, K), dev)
    xs_p = _flat("x_scale", x_scale, torch.float32, (kb, M), dev)
    ws_p = _flat("w_scale", w_scale, torch.float32, (G, (N + 127) // 128, kb), dev)
    out, o_p, o_ld, dtype = _out(out, out_dtype, M, N, x)
    _run(lib().moe_grouped_matmul_fp8, dev, x_p, xs_p, w_p, ws_p, off_p, M, G, N, K, o_p, o_ld, dtype,
         _status(status, dev))
    return out


def grouped_matmul_dx(dy: torch.Tensor, w: torch.Tensor, offsets, *, out=None, out_dtype=None, status=None,
                      stream=None):
    """Gradient of :func:`grouped_matmul`'s rows: dx[r] = dy[r] . w[g] (dy [M, N], w [G, N, K] bf16 -> [M, K])."""
    if stream is not None:
        with _on(stream, dy):
            return grouped_matmul_dx(dy, w, offsets, out=out, out_dtype=out_dtype, status=status)
    M, N = _sizes("dy", dy)
    G, _, K = _sizes("w", w, 3)
    dev = dy.device
    dy_p, dy_ld = _rows("dy", dy, torch.bfloat16, (M, N), dev)
    w_p = _flat("w", w, torch.bfloat16, (G, N, K), dev)
    off_p = _offsets(offsets, G, dev)
    out, o_p, o_ld, dtype = _out(out, out_dtype, M, K, dy)
    _run(lib().moe_grouped_matmul_dx, dev, dy_p, dy_ld, w_p, off_p, M, G, N, K, o_p, o_ld, dtype,
         _status(status, dev))
    return out


def grouped_matmul_dw(dy: torch.Tensor, x: torch.Tensor, offsets, *, out=None, out_dtype=None, accumulate=False,
                      status=None, stream=None):
    """Gradient of :func:`grouped_matmul`'s weights: dw[g] = sum of dy[r]^T x[r] over the group's rows (dy [M, N],
    x [M, K] bf16 -> [G, N, K] bf16 or fp32; zero for an empty group).  ``accumulate`` adds to an fp32 ``out``."""
    if stream is not None:
        with _on(stream, dy):
            return grouped_matmul_dw(dy, x, offsets, out=out, out_dtype=out_dtype, accumulate=accumulate, status=status)
    M, N = _sizes("dy", dy)
    K = _sizes("x", x)[1]
    dev = dy.device
    dy_p, dy_ld = _rows("dy", dy, torch.bfloat16, (M, N), dev)
    x_p, x_ld = _rows("x", x, torch.bfloat16, (M, K), dev)
    G = 1 if offsets is None else _sizes("offsets", offsets, 1)[0] - 1
    off_p = _offsets(offsets, G, dev)
    if accumulate and out is None:
        raise ValueError("accumulate: needs out")
    dtype = _out_dtype(out, out_dtype)
    if out is None:
        out = torch.empty(G, N, K, dtype=dtype, device=dev)
        o_p = out.data_ptr()
    else:
        o_p = _flat("out", out, dtype, (G, N, K), dev)
    _run(lib().moe_grouped_matmul_dw, dev, dy_p, dy_ld, x_p, x_ld, off_p, M, G, N, K, o_p, _OUT_DTYPES[dtype],
         1 if accumulate else 0, _status(status, dev))
    return out
