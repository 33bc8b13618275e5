"""Reference of the quantised K^F/V^F rows (include/hs.h, hs_kv_quant) for the
tests: numpy in float64, no code shared with the library.

Scales and zeros are bf16, so for bf16 rows every division below is far from a
rounding border of the codes unless it lies on one exactly, and float64 and
fp32 agree on every code: (n + 1/2) scale has at most 13 significant bits, x
has 8, so x / scale differs from a midpoint by 0 or by more than 2^-16 of
itself, and both formats divide to within 2^-24.  (In 4 bits x - zero is exact
in fp32 while the row spans fewer than 2^15 of its smallest steps, which the
tests' rows do.)
"""
import numpy as np
import torch


def bf16(x):
    """float64 array rounded to bf16 (through fp32: for the quotients used here
    the two roundings equal one), as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().bfloat16().double().numpy()


def e4m3(y):
    """float64 array rounded to e4m3 (ties to even, saturating), as float64."""
    a = np.minimum(np.abs(y), 1e30)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(y) * np.minimum(np.round(a / step) * step, 448.0)


def encode(x, fmt):
    """(code values, scale, zero), float64, of rows x [..., d]."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if fmt == "int4":
            lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
            s, z = bf16((hi - lo) / 15), bf16(lo)
            c = np.clip(np.round((x - z) / np.where(s > 0, s, 1.0)), 0, 15)
        else:
            s = bf16(np.abs(x).max(-1, keepdims=True) / 448)
            z = np.zeros_like(s)
            c = e4m3(x / np.where(s > 0, s, 1.0))
    c = np.where(s > 0, c, 0.0)
    bad = ~np.isfinite(x).all(-1, keepdims=True) | ~np.isfinite(s) | ~np.isfinite(z)
    return np.where(bad, 0.0, c), np.where(bad, np.nan, s)[..., 0], np.where(bad, np.nan, z)[..., 0]


def codes_of(codes, fmt):
    """Code values, float64, of stored uint8 codes (a tensor)."""
    b = codes.cpu().numpy()
    if fmt == "int4":
        return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1).astype(np.float64)
    bits = np.arange(256)
    e, m = (bits >> 3) & 15, bits & 7
    mag = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    mag = np.where(bits % 128 == 127, np.nan, mag)
    return np.where(bits > 127, -mag, mag)[b]


def values(codes, entry, fmt):
    """What stored rows stand for, float64."""
    s = entry.double().cpu().numpy()
    return codes_of(codes, fmt) * s[..., :1] + s[..., 1:]
