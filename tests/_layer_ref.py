"""Plain references of the residual stream's operators and of microscaled 8-bit
floats, in numpy and torch on the CPU; written from the definitions."""

import math

import numpy as np
import torch

from _matrix_ref import mx4_decode, mx4_encode

#: Every magnitude of e4m3 by its code 0..126 (127 stands for NaN).
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])
MASK = 0xFFFFFFFF


def philox(seed, stream, group):
    """The 4 words of Philox4x32-10 for one counter, in Python's whole numbers."""
    c = [group & MASK, group >> 32 & MASK, stream & MASK, stream >> 32 & MASK]
    k = [seed & MASK, seed >> 32 & MASK]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & MASK, (p >> 32) ^ c[3] ^ k[1], p & MASK]
        k = [k[0] + 0x9E3779B9 & MASK, k[1] + 0xBB67AE85 & MASK]
    return c


def kept(rows, cols, p, seed, stream, first_row=0):
    """(which elements stay, the factor as fp32 holds it)."""
    k = min(65535, int(math.floor(p * 65536 + 0.5)))
    groups = (cols + 7) // 8
    keep = np.zeros((rows, groups * 8), bool)
    for r in range(rows):
        for g in range(groups):
            w = philox(seed, stream, (first_row + r) * groups + g)
            for e in range(8):
                keep[r, 8 * g + e] = (w[e // 2] >> 16 * (e % 2) & 0xFFFF) >= k
    return torch.from_numpy(keep[:, :cols].copy()), float(np.float32(65536 / (65536 - k)))


def dropped(x, mask):
    """x (any type) in fp32: one rounded product for what is kept, 0 for the rest."""
    keep, factor = mask
    return torch.where(keep, x.float() * factor, torch.zeros(()))


def norm64(h, weight, eps):
    """(y, 1 / rms) in float64."""
    h, weight = h.double(), weight.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * r * weight, r


def norm_grad64(dy, h, weight, eps, dh_in=None):
    """(dh, dw), and what bounds the rounding of either: the sums of magnitudes."""
    dy, h, weight = dy.double(), h.double(), weight.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    g = dy * weight
    k = r * r * (g * h).mean(1, keepdim=True)
    dh = r * (g - h * k)
    size = r * (g.abs() + h.abs() * r * r * (g * h).abs().mean(1, keepdim=True))
    if dh_in is not None:
        dh, size = dh + dh_in.double(), size + dh_in.double().abs()
    t = dy * h * r
    return dh, t.sum(0), size, t.abs().sum(0)


def mx8_scale_byte(top):
    return 255 if not math.isfinite(top) else max(-127, math.frexp(top)[1] - 9) + 127 if top > 0 else 0


def e4m3_code(a):
    """The code of magnitude a (float): nearest, ties to the even code, saturating."""
    i = int(np.searchsorted(E4M3, a))
    if i >= len(E4M3):
        return len(E4M3) - 1
    if i == 0 or E4M3[i] == a:
        return i
    up, down = E4M3[i] - a, a - E4M3[i - 1]
    return i if up < down or (up == down and i % 2 == 0) else i - 1


def mx8_encode(x):
    """float64 array [rows, cols] -> (codes [rows, padded cols], scale bytes [rows, blocks])."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    codes, scales = np.zeros((rows, blocks * 32), np.uint8), np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            v = x[r, 32 * b:32 * b + 32]
            scales[r, b] = mx8_scale_byte(float(np.max(np.abs(v))))
            if scales[r, b] == 255:
                continue
            for i, y in enumerate(v):
                codes[r, 32 * b + i] = e4m3_code(abs(float(y)) * 2.0 ** (127 - int(scales[r, b]))) | (128 if math.copysign(1.0, y) < 0 else 0)
    return codes, scales


def mx8_decode(codes, scales, cols):
    v = E4M3[np.minimum(codes & 127, 126)] * np.where(codes > 127, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(scales.shape + (32,)) * s[..., None]).reshape(codes.shape)[:, :cols]


ENCODE = {4: mx4_encode, 8: mx8_encode}
DECODE = {4: mx4_decode, 8: mx8_decode}


def within(got, want, bound):
    """Whether every element of got is as near to want as its bound says."""
    d = (got.double().cpu() - want).abs()
    worst = (d - bound).max() if d.numel() else torch.tensor(-1.0)
    return float(worst) <= 0


def half_step(want, dtype):
    """How far one rounding to dtype may take a value: half a step, or half the smallest subnormal number."""
    f = torch.finfo(dtype)
    return (want.abs() * (f.eps / 2)).clamp(min=f.tiny * f.eps / 2)
