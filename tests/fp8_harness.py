"""The 8-bit operators from their definitions in 64 bits (torch, CPU or GPU)."""
from __future__ import annotations

import math

import torch

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the smallest step


def pad(x, rows, cols):
    out = x.new_zeros(rows, cols)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def up(n, m):
    return -(-n // m) * m


def blocks_of(x, kind):
    """x as [row blocks, rows of a block, column blocks, 128], padded with zeros."""
    high = BLOCK if kind == "tile" else 1
    r, c = up(x.shape[0], high), up(x.shape[1], BLOCK)
    return pad(x, r, c).view(r // high, high, c // BLOCK, BLOCK)


def encode(x, kind):
    """(codes as e4m3 values in float64, scale exponents), [rows, cols] and [row blocks, column blocks]."""
    b = blocks_of(x.double(), kind)
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), 0.0).amax((1, 3))
    f, p = torch.frexp(top / 448.0)
    e = torch.where(f == 0.5, p - 1, p)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    z = torch.where(finite, b, 0.0) / torch.exp2(e.double())[:, None, :, None]
    step = torch.exp2((torch.frexp(z)[1] - 1).clamp(min=-6).double() - 3)
    z = torch.round(z / step) * step
    z = torch.where(finite, z, math.nan)
    rows = b.shape[0] * b.shape[1]
    return z.reshape(rows, -1)[:x.shape[0], :x.shape[1]], e


def exponents(m):
    """The scale exponents of an Fp8Matrix, [row blocks, column blocks]."""
    s = m.scales.view(torch.uint8).long() - 127
    n = m.rows if m.kind == "row" else -(-m.rows // BLOCK)
    return s[:, :n].t()


def codes(m):
    return m.codes.view(torch.float8_e4m3fn)[:, :m.cols].double()


def values(m):
    """The float64 matrix that an Fp8Matrix stands for."""
    e = exponents(m)
    if m.kind == "tile":
        e = e.repeat_interleave(BLOCK, 0)[:m.rows]
    return codes(m) * torch.exp2(e.double()).repeat_interleave(BLOCK, 1)[:, :m.cols]


def padding_is_zero(m):
    pad_codes = m.codes.view(torch.uint8)[:, m.cols:up(m.cols, BLOCK)]
    return bool((pad_codes & 0x7f == 0).all())


def rms_norm(x, residual, weight, eps, dtype):
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(dtype).double()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * weight.double()


def rms_norm_grad(dy, h, dh, weight, rstd):
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    g = dy * w
    mean = (g * h).mean(1, keepdim=True)
    dx = r * (g - h * r * r * mean)
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * h * r).sum(0)


def tokens(gen, rows, cols, sigma, device):
    n = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    return n(rows, cols) * sigma * torch.exp(0.7 * n(rows, 1)) * torch.exp(0.7 * n(1, cols))
