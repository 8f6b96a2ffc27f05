"""Plain 64-bit (or, where results are exact, 32-bit) references of the matrix
operators, in numpy and torch on the CPU; written from the definitions."""

import math

import numpy as np
import torch

DEFAULT = (3.4445, -4.7750, 2.0315)
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def newton_schulz(g, steps=5, coeffs=None, scale=1.0):
    """float64 tensor [rows, cols] -> float64."""
    n = torch.linalg.vector_norm(g)
    x = g / n if float(n) != 0.0 else g
    for k in range(steps):
        a, b, c = coeffs[k] if coeffs is not None else DEFAULT
        gram = x @ x.t()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return scale * x


def rel(got, want):
    want = want.double()
    return float((got.double().cpu() - want).norm() / want.norm())


def gradient(rows, cols, seed, batch=1, low_rank=True):
    g = torch.Generator().manual_seed(seed)
    x = 0.3 * torch.randn((batch, rows, cols), generator=g)
    if low_rank:
        r = max(1, min(rows, cols) // 8)
        u, v = torch.randn((batch, rows, r), generator=g), torch.randn((batch, r, cols), generator=g)
        x = x + u @ v / math.sqrt(r)
    return 1e-3 * x


def mx4_encode(x):
    """float64 array [rows, cols] -> (codes [rows, padded cols] as whole numbers 0..15, scale bytes [rows, blocks])."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    codes = np.zeros((rows, blocks * 32), np.uint8)
    scales = np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            v = x[r, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            top = np.max(np.abs(v))
            e = max(-127, math.frexp(top)[1] - 3) if top > 0 else -127
            scales[r, b] = e + 127
            for i, y in enumerate(v):
                a = abs(float(y)) * 2.0 ** -e
                d = np.abs(GRID - min(a, 6.0))
                best = np.flatnonzero(d == d.min())
                code = next((k for k in best if k % 2 == 0), best[0])
                codes[r, 32 * b + i] = code | (8 if math.copysign(1.0, y) < 0 else 0)
    return codes, scales


def mx4_decode(codes, scales, cols):
    v = GRID[codes & 7] * np.where(codes > 7, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(scales.shape + (32,)) * s[..., None]).reshape(codes.shape)[:, :cols]


def mx4_pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def mx4_tile(scales):
    """Scale bytes [rows, blocks] in the library's tiles, as one flat array."""
    rows, blocks = scales.shape
    rt, kt = (rows + 127) // 128, (blocks + 3) // 4
    out = np.zeros(rt * kt * 512, np.uint8)
    for r in range(rows):
        for b in range(blocks):
            out[(r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = scales[r, b]
    return out
