"""Rows of an 8-bit cache from their definition (float64, no code shared with the
package): E4M3 values from their bits, a row's exponent, the nearest code."""
from __future__ import annotations

import numpy as np
import torch

LIMITS = {torch.bfloat16: (-80, 80), torch.float16: (-15, 7)}


def _values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10.0))
    v = np.where(b & 128, -v, v)
    v[(b & 127) == 127] = np.nan
    return v


VALUES = _values()
POSITIVE = VALUES[:127]  # codes 0 .. 126, increasing


def decode(codes, scale):
    """uint8 codes [..., D] and scale bytes [...] as float64."""
    return torch.from_numpy(VALUES)[codes.long()] * torch.exp2(scale.double() - 127)[..., None]


def exponent(top, dtype):
    """The least e with top <= 448 2^e, within the type's limits (numpy float64; 0 takes the least)."""
    lo, hi = LIMITS[dtype]
    m, x = np.frexp(np.where(np.isfinite(top) & (top > 0), top, 1.0))  # top = m 2^x, m in [0.5, 1)
    e = x - 9 + (m > 0.875)
    return np.where(top == 0, lo, np.where(np.isinf(top), hi, np.clip(e, lo, hi))).astype(np.int64)


def quantise(x, dtype):
    """(codes, scale bytes) of rows x [..., D], a tensor of any type."""
    v = x.double().numpy()
    top = np.nanmax(np.abs(v), axis=-1, initial=0.0) if v.size else np.zeros(v.shape[:-1])
    e = exponent(np.nan_to_num(top, nan=0.0, posinf=np.inf), dtype)
    y = np.abs(v) * np.exp2(-e.astype(np.float64))[..., None]
    y = np.minimum(y, 448.0)  # NaN stays
    hi = np.clip(np.searchsorted(POSITIVE, np.nan_to_num(y)), 1, 126)  # POSITIVE[hi - 1] < y <= POSITIVE[hi], or y = 0
    below, above = np.nan_to_num(y) - POSITIVE[hi - 1], POSITIVE[hi] - np.nan_to_num(y)
    code = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)  # ties to the even code
    code = np.where(np.isnan(v), 127, code) | np.where(np.signbit(v) & ~np.isnan(v), 128, 0)
    return torch.from_numpy(code.astype(np.uint8)), torch.from_numpy((e + 127).astype(np.uint8))
