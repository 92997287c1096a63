"""Rotary positions in 64 bits, with the bounds that the kernels' arithmetic obeys.

u = 2^-24 is fp32's half step, h the half step of the output's type.  An angle is kept in turns:
position * (freq / 2 pi) in 64 bits, off by 3 of 2^-53 of itself; its fraction, at most 1/2, is rounded
to fp32 (u / 2), sine and cosine are within 4 u of 1 of what they should be, and their product with
factor is rounded (u |factor|).  So with e = 2 pi (3 * 2^-53 |turns| + u / 2) + 5 u a component
a cos - b sin is off by factor (|a| + |b|) (e + 2 u) before it is rounded (h of itself)."""
import math

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def turned(x, positions, freqs, begin, interleaved, factor, sign=1):
    """(y, tolerance before rounding) in 64 bits for x [rows, heads, D] (64 bits)."""
    n = freqs.shape[0]
    turns = positions.double()[:, None] * (freqs / (2 * math.pi))
    angle = sign * 2 * math.pi * (turns - turns.round())
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    i = torch.arange(n, device=x.device)
    first, second = (begin + 2 * i, begin + 2 * i + 1) if interleaved else (begin + i, begin + n + i)
    a, b = x[..., first], x[..., second]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = factor * (a * c - b * s), factor * (a * s + b * c)
    e = 2 * math.pi * (3 * 2.0 ** -53 * turns.abs() + U / 2)[:, None] + 7 * U
    tol[..., first] = tol[..., second] = abs(factor) * (a.abs() + b.abs()) * e
    return y, tol


def check(x, y, positions, freqs, begin, interleaved, factor, sign=1):
    x64, y64 = (t.double().unflatten(1, (1, -1)) if t.dim() == 2 else t.double() for t in (x, y))
    ref, tol = turned(x64, positions, freqs, begin, interleaved, factor, sign)
    # 2^-126: below it, the smallest normal number, products may give 0
    tol = HALF[x.dtype] * (ref.abs() + tol) * (tol > 0) + tol + 2.0 ** -126 * (tol > 0)
    err = (y64 - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


def make(rows, heads, D, dtype, seed, pad=0, far=1000, dims=3):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(rows, heads * D + pad, generator=g).to(dtype).cuda()
    x = wide[:, :heads * D]
    pos = torch.randint(0, far, (rows,), generator=g, dtype=torch.int32).cuda()
    return (x.unflatten(1, (heads, D)) if dims == 3 else x), pos
