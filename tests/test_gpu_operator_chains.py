"""The stand-alone operators together, as a model runs them: in front of and beside the layer, in a training
step of the experts, captured into graphs, on other streams, and past 32-bit offsets."""

import pytest
import torch

from moe_layer_top_b200 import inputs, ops
from tests.operator_helpers import assert_within, offsets_of, product_bound, quantize_weight, row_values, weight_values

pytestmark = pytest.mark.gpu

EPS = 1e-6


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


def _swiglu(h):
    """The layer's activation with its rounding points."""
    gate, up = h.float().chunk(2, -1)
    return (torch.nn.functional.silu(gate).to(torch.bfloat16).float() * up).to(torch.bfloat16)


def _by_expert(ids, E):
    """Assignments sorted by expert: (flat ids in that order, offsets)."""
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    off = torch.zeros((E + 1,), dtype=torch.int32, device=ids.device)
    off[1:] = counts.cumsum(0)
    return order, off


@pytest.mark.parametrize("T", [1, 7, 64, 700])
def test_norm_router_and_experts_are_the_layer(T):
    """Residual addition and norm, router logits, routing, the experts' two FP8 products and the combine, against
    fused_forward on the same normalised rows and weights: the same codes go into the first product, and both
    follow the layer's rounding points, so they differ by fp32 summation orders and the roundings those flip --
    the layer's own tolerance between orientations (2e-2 normwise) covers that with room."""
    E, k, H, I = 8, 2, 512, 256
    cfg = inputs.make_custom_config("chain", E=E, topk=k, H=H, I=I, fp8=True, routing="logits")
    w13, w2 = inputs.make_weights(cfg, 3, device="cuda")
    q13, s13 = ops.quantize_weights_fp8(w13)
    q2, s2 = ops.quantize_weights_fp8(w2)
    router, gain = _randn(1, 1, E, H, std=0.1), (1 + 0.1 * _randn(2, H)).to(torch.bfloat16)
    x, residual = _randn(3, T, H), _randn(4, T, H)

    norm = ops.rms_norm(x, gain, EPS, residual=residual, fp8=True)
    logits = ops.grouped_matmul(norm["y"], router, None, out_dtype=torch.float32)
    ids, weights = ops.route(logits, k)
    order, off = _by_expert(ids, E)
    token = order // k
    h = ops.grouped_matmul(norm["codes"][token], q13, off, x_scale=norm["scales"][:, token].contiguous(), w_scale=s13)
    a, a_scale = ops.quantize_rows_fp8(_swiglu(h))
    y = ops.grouped_matmul(a, q2, off, x_scale=a_scale, w_scale=s2, out_dtype=torch.float32)
    out = torch.zeros((T, H), device="cuda").index_add_(0, token, y * weights.flatten()[order][:, None])

    p = ops.problem(T, E, k, H, I, fp8=True)
    ref = ops.fused_forward(p, norm["y"], q13, q2, logits=logits, w13_scale=s13, w2_scale=s2).float()
    err = (out - ref).norm() / ref.norm()
    assert torch.isfinite(out).all() and err <= 2e-2, f"normwise relative error {err:.3e}"
    ref_logits = norm["y"].double() @ router[0].double().t()
    assert_within(logits, ref_logits, product_bound(ref_logits, norm["y"].double().abs() @ router[0].double().abs().t(),
                                                    H, torch.float32))


def test_training_step_of_the_experts():
    """Norm, grouped product, and their backward passes against automatic differentiation in double."""
    sizes, N, K = [40, 0, 3, 150, 64], 264, 136
    off, M = offsets_of(sizes), 257
    s, gain, w = _randn(11, M, K, std=2.0), (1 + 0.1 * _randn(12, K)).to(torch.bfloat16), _randn(13, 5, N, K, std=0.1)
    c = _randn(14, M, N, std=0.1)
    fwd = ops.rms_norm(s, gain, EPS, rstd=True)
    y = ops.grouped_matmul(fwd["y"], w, off)
    dx_norm = ops.grouped_matmul_dx(c, w, off)
    dw = ops.grouped_matmul_dw(c, fwd["y"], off, out_dtype=torch.float32)
    ds, dgain = ops.rms_norm_backward(dx_norm, s, gain, fwd["rstd"])

    sd, gd, wd = (t.double().requires_grad_() for t in (s, gain, w))
    n = sd * (sd.square().mean(-1, keepdim=True) + EPS).rsqrt() * gd
    g = torch.repeat_interleave(torch.arange(5, device="cuda"), torch.tensor(sizes, device="cuda"))
    yd = torch.einsum("mk,mnk->mn", n, wd[g])
    (yd * c.double()).sum().backward()
    # each quantity passes at most two bf16 roundings (2^-8 each) and sums of independent errors: 2^-7 normwise
    for got, ref in ((y, yd), (ds, sd.grad), (dgain, gd.grad), (dw, wd.grad)):
        assert (got.double() - ref).norm() <= 2.0 ** -7 * ref.norm()


def _everything(t):
    """One pass through every operator; the results in a list."""
    n = ops.rms_norm(t["x"], t["gain"], EPS, residual=t["res"], fp8=True, rstd=True)
    codes, scales = ops.quantize_rows_fp8(n["y"])
    back = ops.dequantize_rows_fp8(n["codes"], n["scales"])
    z = ops.matmul_fp8(codes, scales, t["wq"][0], t["ws"][0])
    y = ops.grouped_matmul(n["y"], t["w"], t["off"])
    y8 = ops.grouped_matmul(codes, t["wq"], t["off"], x_scale=scales, w_scale=t["ws"])
    dx = ops.grouped_matmul_dx(y, t["w"], t["off"])
    dw = ops.grouped_matmul_dw(y, n["y"], t["off"])
    ds, dgain = ops.rms_norm_backward(dx, n["residual"], t["gain"], n["rstd"], dresidual=t["x"])
    return [n["residual"], n["y"], n["codes"], n["scales"], n["rstd"], back, z, y, y8, dx, dw, ds, dgain]


def _tensors(seed, sizes, N, K):
    M, G = sum(sizes), len(sizes)
    t = dict(x=_randn(seed, M, K), res=_randn(seed + 1, M, K), gain=(1 + 0.1 * _randn(5, K)).to(torch.bfloat16),
             w=_randn(seed + 2, G, N, K, std=0.1), off=offsets_of(sizes))
    t["wq"], t["ws"] = quantize_weight(t["w"])
    return t


SETS = [([5, 0, 60, 3], 136, 272), ([700, 0, 300, 33, 513, 1000], 2056, 528), ([2], 256, 4096)]


@pytest.mark.parametrize("sizes,N,K", SETS)
def test_back_to_back_launches_agree_with_separate_ones(sizes, N, K):
    """Kernels start under their predecessors' tails; every one of them waits for what it reads."""
    t = _tensors(21, sizes, N, K)
    torch.cuda.synchronize()
    want = [r.clone() for r in _everything(t)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = _everything(t)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("sizes,N,K", SETS)
def test_captured_and_replayed(sizes, N, K):
    """Two captured graphs of the whole pass, replayed in turn and with new values in the same buffers."""
    t, u = _tensors(31, sizes, N, K), _tensors(41, sizes, N, K)
    want_t, want_u = [r.clone() for r in _everything(t)], [r.clone() for r in _everything(u)]
    graphs = []
    for v in (t, u):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _everything(v)
        graphs.append((g, out))
    for _ in range(2):
        for (g, out), want in zip(graphs, (want_t, want_u)):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    for k in t:
        t[k].copy_(u[k])
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want_u))


def test_two_streams_at_once():
    sets = [_tensors(51, *SETS[1]), _tensors(61, *SETS[1])]
    want = [[r.clone() for r in _everything(t)] for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _everything(sets[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_stream_argument():
    t = _tensors(71, *SETS[0])
    want = ops.grouped_matmul(t["x"], t["w"], t["off"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    ops.grouped_matmul(t["x"], t["w"], t["off"], out=out, stream=s)
    y = torch.empty_like(t["x"])
    ops.rms_norm(t["x"], t["gain"], EPS, y=y, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(y, ops.rms_norm(t["x"], t["gain"], EPS)["y"])


def test_outputs_belong_to_the_stream_argument():
    """Memory that the current stream has freed but has still to write is not handed to a call on another stream."""
    x, dy = _randn(75, 512, 4096), _randn(76, 512, 4096)
    gain = (1 + 0.1 * _randn(77, 4096)).to(torch.bfloat16)
    w = _randn(78, 1, 4096, 4096)
    rstd = ops.rms_norm(x, gain, EPS, rstd=True)["rstd"]
    s = torch.cuda.Stream()
    calls = [lambda **kw: ops.rms_norm_backward(dy, x, gain, rstd, **kw)[0],
             lambda **kw: ops.rms_norm(x, gain, EPS, **kw)["y"],
             lambda **kw: ops.grouped_matmul(x, w, None, **kw)]
    for call in calls:
        want = call()
        late = torch.empty_like(want)
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)  # about 25 ms
        late.fill_(float("nan"))
        del late
        got = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_another_device_than_the_current_one():
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    t = _tensors(81, *SETS[0])
    want = _everything(t)
    with torch.cuda.device(1):
        got = _everything(t)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ----------------------------------------------------------------------------- past 32-bit offsets
def test_rows_past_two_to_the_31():
    T, H = 270_000, 8192     # 2.2e9 elements
    x = _randn(91, 1000, H).repeat(270, 1)
    gain = (1 + 0.1 * _randn(92, H)).to(torch.bfloat16)
    n = ops.rms_norm(x, gain, EPS, fp8=True, rstd=True)
    first = ops.rms_norm(x[:1000].contiguous(), gain, EPS, fp8=True, rstd=True)
    assert torch.equal(n["y"][-1000:], first["y"]) and torch.equal(n["codes"][-1000:], first["codes"])
    assert torch.equal(n["scales"][:, -1000:], first["scales"]) and torch.equal(n["rstd"][-1000:], first["rstd"])
    codes, scales = ops.quantize_rows_fp8(n["y"])
    assert torch.equal(codes[-1000:], first["codes"]) and torch.equal(scales[:, -1000:], first["scales"])
    del n["y"]
    back = ops.dequantize_rows_fp8(codes, scales)
    assert torch.equal(back[-1000:], ops.dequantize_rows_fp8(first["codes"], first["scales"]))
    del codes, back
    dx, _ = ops.rms_norm_backward(x, x, gain, n["rstd"])
    small, _ = ops.rms_norm_backward(x[:1000].contiguous(), x[:1000].contiguous(), gain, first["rstd"])
    assert torch.equal(dx[-1000:], small)


def test_products_past_two_to_the_31():
    M, N, K = 270_000, 8, 8192
    sizes = [M - 300, 0, 300]
    off = offsets_of(sizes)
    x = _randn(93, 1000, K).repeat(270, 1)
    w = _randn(94, 3, N, K, std=0.1)
    y = ops.grouped_matmul(x, w, off)
    ref = x[-300:].double() @ w[2].double().t()
    assert_within(y[-300:], ref, product_bound(ref, x[-300:].double().abs() @ w[2].double().abs().t(), K, y.dtype))
    dx = ops.grouped_matmul_dx(y, w, off)
    ref = y[-300:].double() @ w[2].double()
    assert_within(dx[-300:], ref, product_bound(ref, y[-300:].double().abs() @ w[2].double().abs(), N, y.dtype))
    dw = ops.grouped_matmul_dw(y, x, off, out_dtype=torch.float32)
    a, b = y[-300:].double(), x[-300:].double()
    assert_within(dw[2], a.t() @ b, product_bound(a.t() @ b, a.abs().t() @ b.abs(), 300, torch.float32))
    del dx, x, y
    G, N, K = 530, 2048, 2056   # weights and their gradient: 2.2e9 elements
    w = torch.zeros((G, N, K), dtype=torch.bfloat16, device="cuda")
    w[-1] = _randn(95, N, K, std=0.1)
    off = torch.zeros((G + 1,), dtype=torch.int32, device="cuda")
    off[-1] = 40
    x, dy = _randn(96, 40, K), _randn(97, 40, N)
    ref = x.double() @ w[-1].double().t()
    assert_within(ops.grouped_matmul(x, w, off), ref,
                  product_bound(ref, x.double().abs() @ w[-1].double().abs().t(), K, torch.bfloat16))
    ref = dy.double() @ w[-1].double()
    assert_within(ops.grouped_matmul_dx(dy, w, off), ref,
                  product_bound(ref, dy.double().abs() @ w[-1].double().abs(), N, torch.bfloat16))
    dw = ops.grouped_matmul_dw(dy, x, off, out=w)
    ref = dy.double().t() @ x.double()
    assert_within(dw[-1], ref, product_bound(ref, dy.double().abs().t() @ x.double().abs(), 40, torch.bfloat16))
    assert not dw[:-1].any()


def test_fp8_products_past_two_to_the_31():
    G, N, K = 530, 2048, 2064
    wq = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((G, 16, 17), device="cuda")
    wq[-1], ws[-1] = quantize_weight(_randn(98, N, K, std=0.1))
    off = torch.zeros((G + 1,), dtype=torch.int32, device="cuda")
    off[-1] = 40
    codes, scales = ops.quantize_rows_fp8(_randn(99, 40, K))
    y = ops.grouped_matmul(codes, wq, off, x_scale=scales, w_scale=ws)
    xv, wv = row_values(codes, scales), weight_values(wq[-1], ws[-1])
    ref = xv @ wv.t()
    assert_within(y, ref, product_bound(ref, xv.abs() @ wv.abs().t(), K, torch.bfloat16, fp8=True))
