"""64-bit references and error bounds shared by the tests of the stand-alone operators.

A product's bound per element: every term is exact in fp32 (bf16 x bf16; E4M3 x E4M3), the terms
are added in fp32 in an order and rounding mode of the hardware's choice, so the sum is off by at
most one fp32 step (2^-23) of the running magnitude per addition, n 2^-23 sum|a b| in all; then one
rounding of the result, half a step of its type.  E4M3 tensor-core sums may keep as few as 14 bits
of the largest term inside a 128-deep block (published for the previous generation), 2^-13 of the
block's magnitude."""

from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FP8_SUM = 2.0 ** -13


def pow2(e):
    """2^e in double, exactly (a power function need not be), for integers e within the normal range."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def decode_e4m3(codes):
    """E4M3 codes (uint8) -> doubles."""
    c = torch.arange(256, device=codes.device)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * pow2(e - 7))
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)[codes.long()]


def row_values(codes, scales):
    k = torch.arange(codes.shape[1], device=codes.device) // 128
    return decode_e4m3(codes) * scales.double()[k].t()


def weight_values(codes, scales):
    """[.., N, K] codes with [.., ceil(N / 128), ceil(K / 128)] scales."""
    n = torch.arange(codes.shape[-2], device=codes.device) // 128
    k = torch.arange(codes.shape[-1], device=codes.device) // 128
    return decode_e4m3(codes) * scales.double()[..., n[:, None], k[None, :]]


def quantize_rows(x):
    """The row format's rule in plain torch: (codes uint8, scales [ceil(cols / 128), rows])."""
    rows, cols = x.shape
    g = math.ceil(cols / 128)
    v = torch.zeros((rows, g * 128), device=x.device)
    v[:, :cols] = x.float()
    v = v.view(rows, g, 128)
    finite = torch.isfinite(v)
    amax = torch.where(finite, v.abs(), torch.zeros_like(v)).amax(-1).clamp(min=1e-10)
    m, e = torch.frexp(amax * (torch.ones_like(amax) / 448))
    s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    q = (v / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.where(finite, q, torch.full_like(q, 0x7F))
    return q.view(rows, -1)[:, :cols].contiguous(), s.t().contiguous()


def quantize_weight(w):
    """[.., N, K] -> E4M3 codes and one fp32 scale per 128 x 128 block, padded with zeros where a block is cut."""
    lead, (N, K) = w.shape[:-2], w.shape[-2:]
    nb, kb = math.ceil(N / 128), math.ceil(K / 128)
    f = torch.zeros((*lead, nb * 128, kb * 128), device=w.device)
    f[..., :N, :K] = w
    f = f.view(*lead, nb, 128, kb, 128)
    amax = f.abs().amax((-3, -1)).clamp(min=1e-10)
    s = amax / torch.full_like(amax, 448.0)   # a division by a number may be a product with its reciprocal
    q = (f / s[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(*lead, nb * 128, kb * 128)[..., :N, :K].contiguous(), s.contiguous()


def offsets_of(sizes, start=0):
    o = [start]
    for n in sizes:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def assert_within(got, ref, bound):
    """|got - ref| <= bound element by element; got finite."""
    assert got.shape == ref.shape
    g = got.double()
    assert torch.isfinite(g).all(), "non-finite output"
    over = (g - ref).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    at = int(over.argmax()) if over.numel() else 0
    assert worst <= 0, (f"off by {(g - ref).abs().flatten()[at].item():.3e}, bound "
                        f"{bound.flatten()[at].item():.3e}, at {at} of {tuple(got.shape)}")


def product_bound(ref, mag, terms, out_dtype, fp8=False):
    return HALF_STEP[out_dtype] * ref.abs() * (1 + 2.0 ** -7) + (terms * 2.0 ** -23 + (FP8_SUM if fp8 else 0)) * mag
