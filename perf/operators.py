"""Timed and checked cases of the stand-alone operators: the RMS norm (forward with the residual's
addition and an FP8 output, and backward), the FP8 matrix product with block scales, and the
matrix products grouped by expert (forward, and the two products of the backward pass).

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs of one, ``run()`` one pass: with
``own`` false in plain torch operations, with ``own`` true through the package's entry points.
``exact()`` evaluates the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's hidden state between two layers of a decoding model: launch latency
        dict(name="norm fp8 T=1", op="norm", T=1, H=7168, residual=True, fp8=True),
        # the rows of a prefill batch, normalised and quantised for the FP8 products that follow
        dict(name="norm fp8 T=8192", op="norm", T=8192, H=7168, residual=True, fp8=True),
        # a ragged training batch, forward (rstd is kept for the backward pass)
        dict(name="norm bf16 T=1037", op="norm", T=1037, H=4104, residual=False, fp8=False),
        # the same norm's backward pass in a large training batch
        dict(name="norm backward T=16384", op="norm_backward", T=16384, H=4096, dres=True),
        # a dense projection in FP8 for one token: the weights are read once
        dict(name="linear fp8 M=1", op="linear", M=1, N=4096, K=7168),
        # ragged sizes: a partial scale block in K, a partial tile in M and N
        dict(name="linear fp8 M=333", op="linear", M=333, N=2056, K=1616),
        # a prefill batch through the same projection: bound by the tensor cores
        dict(name="linear fp8 M=8192", op="linear", M=8192, N=4096, K=7168),
        # 64 decoding tokens with 8 experts each: the hit experts' weights are read once
        dict(name="grouped bf16 decode", op="grouped", M=512, G=128, N=4096, K=1536, skew=0.0, fp8=False),
        # 512 tokens with 8 experts each, a few experts taking most of the rows
        dict(name="grouped fp8 skewed", op="grouped", M=4096, G=256, N=7168, K=2048, skew=1.2, fp8=True),
        # the experts' down projection of a training batch
        dict(name="grouped bf16 training", op="grouped", M=32768, G=128, N=4096, K=1536, skew=0.3, fp8=False),
        # a toy layer's backward pass: launch latency
        dict(name="grouped backward tiny", op="grouped_backward", M=32, G=8, N=256, K=128, skew=0.0),
        # the gradients of that training batch's rows and weights
        dict(name="grouped backward training", op="grouped_backward", M=32768, G=128, N=4096, K=1536, skew=0.3),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], evenly spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "linear", "grouped", "grouped", "grouped_backward"])
    if op == "norm":
        fp8 = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 256, 7168, 16 if fp8 else 8),
                    residual=rng.random() < 0.5, fp8=fp8)
    if op == "norm_backward":
        return dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 256, 4096, 8), dres=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 128, 4096, 8), K=_log(rng, 128, 7168, 16))
    G = _log(rng, 4, 128)
    N, K = _log(rng, 128, 4096, 8), _log(rng, 128, 1536, 8)
    skew = rng.choice([0.0, 0.3, 0.8, 1.2])
    if op == "grouped":
        fp8 = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, 32768), G=G, N=N, K=(K + 15) // 16 * 16 if fp8 else K, skew=skew, fp8=fp8)
    return dict(op=op, M=_log(rng, 1, 32768), G=G, N=N, K=K, skew=skew)


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        # x (and the residual, read and written), the weight; the output in 16 or 8 bits
        per = 2 + (4 if case["residual"] else 0)
        out = H + 4 * ((H + 127) // 128) if case["fp8"] else 2 * H + 4
        return {"bytes": T * (per * H + out) + 2 * H, "flops": 5 * T * H}
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * (6 + (2 if case["dres"] else 0)) + 4 * T + 6 * H, "flops": 9 * T * H}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * math.ceil(N / 128) * math.ceil(K / 128) + 2 * M * N,
                "flops": 2 * M * N * K}
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    hit = sum(1 for c in _counts(M, G, case["skew"]) if c)
    if op == "grouped":
        e = 1 if case["fp8"] else 2
        scales = 4 * math.ceil(K / 128) * (M + hit * math.ceil(N / 128)) if case["fp8"] else 0
        return {"bytes": e * (M * K + hit * N * K) + scales + 2 * M * N + 4 * (G + 1), "flops": 2 * M * N * K}
    # dy and x once, the hit experts' weights, dx, and every expert's weight gradient
    return {"bytes": 2 * (M * (N + 2 * K) + hit * N * K + G * N * K) + 4 * (G + 1), "flops": 4 * M * N * K}


# ----------------------------------------------------------------------------- inputs
def _counts(M, G, skew):
    """Rows of each group: experts by a power law of exponent ``skew`` (0: even), drawn from a
    fixed stream of the sizes, so that the work of a case does not depend on the seed."""
    r = np.random.RandomState((M * 1000003 + G * 1009 + int(skew * 100)) % (1 << 32))
    p = 1.0 / np.arange(1, G + 1) ** skew
    return r.permutation(r.multinomial(M, p / p.sum())).tolist()


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)


def _quantize_weight(w):
    """bf16 [N, K] -> E4M3 codes (uint8) and one fp32 scale for each 128 x 128 block."""
    N, K = w.shape
    nb, kb = math.ceil(N / 128), math.ceil(K / 128)
    f = torch.zeros((nb * 128, kb * 128), device=w.device)
    f[:N, :K] = w
    f = f.view(nb, 128, kb, 128)
    s = f.abs().amax((1, 3)).clamp(min=1e-10) / 448
    q = (f / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(nb * 128, kb * 128)[:N, :K].contiguous().view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _randn(g, T, H)
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
        s["residual"] = _randn(g, T, H, std=3.0) if case["residual"] else None
        return s
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        s["dy"] = _randn(g, T, H, std=0.01)
        s["x"] = _randn(g, T, H, std=2.0)
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
        s["dres"] = _randn(g, T, H, std=0.01) if case["dres"] else None
        return s
    if op == "linear":
        s["x"] = _randn(g, case["M"], case["K"], std=0.5)
        s["w"], s["w_scale"] = _quantize_weight(_randn(g, case["N"], case["K"], std=0.02))
        return s
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    s["sizes"] = _counts(M, G, case["skew"])
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(s["sizes"])]).astype(np.int32)).cuda()
    x = _randn(g, M, K, std=0.5)
    if op == "grouped" and case["fp8"]:
        s["x"], s["x_scale"] = _quantize_rows(x)
        s["w"] = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
        s["w_scale"] = torch.empty((G, math.ceil(N / 128), math.ceil(K / 128)), device="cuda")
        for e in range(G):
            s["w"][e], s["w_scale"][e] = _quantize_weight(_randn(g, N, K, std=0.02))
        return s
    s["x"], s["w"] = x, _randn(g, G, N, K, std=0.02)
    if op == "grouped_backward":
        s["dy"] = _randn(g, M, N, std=0.01)
    return s


# ----------------------------------------------------------------------------- plain forms
def _row_groups(v):
    """[T, H] -> [T, ceil(H / 128), 128], zero-padded."""
    T, H = v.shape
    n = math.ceil(H / 128)
    if n * 128 != H:
        v = torch.cat([v, v.new_zeros((T, n * 128 - H))], 1)
    return v.view(T, n, 128)


def _row_scales(amax):
    """The smallest power of two that is at least max(amax, 1e-10) / 448."""
    m, e = torch.frexp(amax.clamp(min=1e-10) * (1.0 / 448))
    return torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))


def _quantize_rows(x):
    """bf16 [T, H] -> E4M3 codes (uint8) [T, H] and fp32 scales [ceil(H / 128), T]."""
    v = _row_groups(x.float())
    s = _row_scales(v.abs().amax(-1))
    q = (v / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(x.shape[0], -1)[:, :x.shape[1]].contiguous().view(torch.uint8), s.t().contiguous()


def _row_values(codes, scales):
    """The numbers that quantised rows stand for, in 32 bits."""
    v = _row_groups(codes.view(torch.float8_e4m3fn).float()) * scales.t()[..., None]
    return v.view(codes.shape[0], -1)[:, :codes.shape[1]]


def _weight_values(codes, scales):
    """The numbers that an 8-bit weight stands for, in 32 bits."""
    N, K = codes.shape
    s = scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).float() * s


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"]
        if s["residual"] is not None:
            x = (x.float() + s["residual"].float()).to(torch.bfloat16)
        v = x.float()
        rstd = torch.rsqrt(v.square().mean(-1) + EPS)
        y = (v * rstd[:, None] * s["weight"].float()).to(torch.bfloat16)
        out = {"residual": x if s["residual"] is not None else None, "rstd": rstd}
        if case["fp8"]:
            return {**out, "values": _row_values(*_quantize_rows(y)).to(torch.bfloat16)}
        return {**out, "y": y}
    if op == "norm_backward":
        xhat = s["x"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        a = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (a - xhat * (a * xhat).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xhat).sum(0)}
    if op == "linear":
        x = _row_values(*_quantize_rows(s["x"]))
        return {"y": (x @ _weight_values(s["w"], s["w_scale"]).t()).to(torch.bfloat16)}
    # one product for each group that has rows
    hit = [e for e, n in enumerate(s["sizes"]) if n]
    if op == "grouped":
        if case["fp8"]:
            x = _row_values(s["x"], s["x_scale"]).split(s["sizes"])
            y = [x[e] @ _weight_values(s["w"][e], s["w_scale"][e]).t() for e in hit]
        else:
            x = s["x"].float().split(s["sizes"])
            y = [x[e] @ s["w"][e].float().t() for e in hit]
        return {"y": torch.cat(y).to(torch.bfloat16)}
    x, dy = s["x"].float().split(s["sizes"]), s["dy"].float().split(s["sizes"])
    return {"dx": torch.cat([dy[e] @ s["w"][e].float() for e in hit]).to(torch.bfloat16),
            "dw": torch.stack([(b.t() @ a).to(torch.bfloat16) for a, b in zip(x, dy)])}


# ----------------------------------------------------------------------------- the package's operators
def _own(s):
    from moe_layer_top_b200 import ops

    case = s["case"]
    op = case["op"]
    if op == "norm":
        r = ops.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], y=not case["fp8"], fp8=case["fp8"],
                         rstd=True)
        out = {"residual": r["residual"], "rstd": r["rstd"]}
        if case["fp8"]:
            return {**out, "values": ops.dequantize_rows_fp8(r["codes"], r["scales"])}
        return {**out, "y": r["y"]}
    if op == "norm_backward":
        dx, dweight = ops.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dresidual=s["dres"])
        return {"dx": dx, "dweight": dweight}
    if op == "linear":
        codes, scales = ops.quantize_rows_fp8(s["x"])
        return {"y": ops.matmul_fp8(codes, scales, s["w"], s["w_scale"])}
    if op == "grouped":
        if case["fp8"]:
            return {"y": ops.grouped_matmul(s["x"], s["w"], s["offsets"], x_scale=s["x_scale"], w_scale=s["w_scale"])}
        return {"y": ops.grouped_matmul(s["x"], s["w"], s["offsets"])}
    return {"dx": ops.grouped_matmul_dx(s["dy"], s["w"], s["offsets"]),
            "dw": ops.grouped_matmul_dw(s["dy"], s["x"], s["offsets"])}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- 64 bits
def _pow2(e):
    """2^e in double, exactly (a power function need not be), for integers e within the normal range."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decode(codes):
    """E4M3 codes (uint8) -> doubles, from the format's definition."""
    c = torch.arange(256, device=codes.device)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _pow2(e - 7))
    table = torch.where(c >= 128, -mag, mag)
    return table[codes.long()]


def _exact_rows(codes, scales):
    k = torch.arange(codes.shape[1], device=codes.device) // 128
    return _decode(codes) * scales.double()[k].t()


def _exact_weight(codes, scales):
    n = torch.arange(codes.shape[0], device=codes.device) // 128
    k = torch.arange(codes.shape[1], device=codes.device) // 128
    return _decode(codes) * scales.double()[n[:, None], k[None, :]]


def _exact_quantized(x):
    """The row quantisation by its definition: the grid of the values is searched, none is cast."""
    T, H = x.shape
    out = torch.empty((T, H), dtype=torch.float64, device=x.device)
    grid = _decode(torch.arange(127, dtype=torch.uint8, device=x.device))  # the non-negative values, ascending
    for c in range(0, H, 128):
        v = x[:, c:c + 128].double()
        amax = v.abs().amax(1, keepdim=True).clamp(min=1e-10)
        scale = _pow2(torch.ceil(torch.log2(amax / 448)))
        u = (v.abs() / scale).clamp(max=448.0)
        hi = torch.searchsorted(grid, u.contiguous()).clamp(1, 126)
        lo = hi - 1
        mid = (grid[lo] + grid[hi]) / 2
        up = (u > mid) | ((u == mid) & (hi % 2 == 0))
        out[:, c:c + 128] = torch.sign(v) * torch.where(up, grid[hi], grid[lo]) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        if case["residual"]:
            # the sum is stored in bf16 and the norm is taken of what is stored (the sum of two bf16
            # numbers is exact in 64 bits; 32 bits in between could round twice)
            x = (x + s["residual"].double()).to(torch.bfloat16).double()
        rstd = 1 / torch.sqrt((x * x).sum(1) / x.shape[1] + EPS)
        out = {"residual": x if case["residual"] else None, "rstd": rstd}
        # the quantised values step at rounding borders: no 64-bit number stands beside them
        return {**out, "values": None} if case["fp8"] else {**out, "y": x * rstd[:, None] * s["weight"].double()}
    if op == "norm_backward":
        x, dy, w, r = s["x"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        n = x * r[:, None]
        proj = torch.einsum("th,h,th->t", dy, w, n) / x.shape[1]
        dx = (dy * w - n * proj[:, None]) * r[:, None]
        return {"dx": dx + s["dres"].double() if case["dres"] else dx, "dweight": torch.einsum("th,th->h", dy, n)}
    if op == "linear":
        return {"y": _exact_quantized(s["x"]) @ _exact_weight(s["w"], s["w_scale"]).t()}
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    off = s["offsets"].tolist()
    if op == "grouped":
        y = torch.empty((M, N), dtype=torch.float64, device="cuda")
        for e in range(G):
            a, b = off[e], off[e + 1]
            if b > a:
                if case["fp8"]:
                    y[a:b] = _exact_rows(s["x"][a:b], s["x_scale"][:, a:b]) @ _exact_weight(s["w"][e], s["w_scale"][e]).t()
                else:
                    y[a:b] = s["x"][a:b].double() @ s["w"][e].double().t()
        return {"y": y}
    dx = torch.empty((M, K), dtype=torch.float64, device="cuda")
    dw = torch.zeros((G, N, K), dtype=torch.float64, device="cuda")
    for e in range(G):
        a, b = off[e], off[e + 1]
        if b > a:
            dy = s["dy"][a:b].double()
            dx[a:b] = dy @ s["w"][e].double()
            dw[e] = dy.t() @ s["x"][a:b].double()
    return {"dx": dx, "dw": dw}
