"""Plain 64-bit definitions of the 8-bit pool's operators and the rotary tables,
for the tests.

Everything is numpy float64 or Python integers; nothing here uses the library
or its kernels.
"""
from __future__ import annotations

import math

import numpy as np

from tests.fp4_ref import E4M3, nearest_even

LOW, HIGH = -120, 119


# --------------------------------------------------------------------------- #
# elements and scales
# --------------------------------------------------------------------------- #
def element(x: np.ndarray) -> np.ndarray:
    """e4m3 bytes of x: nearest, ties to even, saturating at 448; NaN and infinities are NaN."""
    bad = ~np.isfinite(x)
    code = nearest_even(np.where(bad, 0.0, np.abs(x)), E4M3)
    return np.where(bad, 0x7F, code + 128 * np.signbit(x)).astype(np.uint8)


def value(code: np.ndarray) -> np.ndarray:
    return np.append(E4M3, np.nan)[code & 127] * np.where(code & 128, -1.0, 1.0)


def needed(top: np.ndarray) -> np.ndarray:
    """The smallest e in range with top <= 448 * 2^e."""
    m, x = np.frexp(top)  # top = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = np.where(m <= 0.875, x - 9, x - 8)
    return np.clip(np.where(top == 0, LOW, e), LOW, HIGH)


def runs(rows, block):
    """(first token, first row, tokens) of each run of consecutive rows in one block."""
    out, i = [], 0
    while i < len(rows):
        n = 1
        while i + n < len(rows) and rows[i + n] == rows[i] + n and rows[i + n] % block:
            n += 1
        out.append((i, int(rows[i]), n))
        i += n
    return out


def store(codes, exps, rows, x, block):
    """Rows x [N, H, d] (float64) into codes [R, H, d] and exps [ceil(R / block), H], in place."""
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    for i, row, n in runs(rows, block):
        b, off = row // block, row % block
        e = needed(fin[i:i + n].max((0, 2)))
        if off:
            before = exps[b].astype(int)
            e = np.maximum(e, before)
            old = slice(row - off, row)
            grown = e > before
            codes[old][:, grown] = element(value(codes[old]) * 2.0 ** (before - e)[:, None])[:, grown]
        codes[row:row + n] = element(x[i:i + n] * 2.0 ** -e[:, None])
        exps[b] = e
    return codes, exps


def values(codes, exps, block):
    """float64 [R, H, d] that codes [R, H, d] and exps [ceil(R / block), H] stand for."""
    e = np.repeat(np.asarray(exps, dtype=np.float64), block, 0)[:len(codes)]
    return value(codes) * 2.0 ** e[..., None]


# --------------------------------------------------------------------------- #
# rotary positions
# --------------------------------------------------------------------------- #
def frequencies(rotary, base, kind="plain", factor=1.0, origin=0, slow=1.0, fast=None, attention=None):
    """theta_j of each pair and the factor of cos and sin."""
    fast = fast if fast is not None else 32.0 if kind == "yarn" else 4.0
    if kind == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    out = []
    for j in range(rotary // 2):
        theta = base ** (-2 * j / rotary)
        if kind == "linear":
            theta /= factor
        elif kind == "bands":
            turns = origin * theta / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            theta = (1 - keep) * theta / factor + keep * theta
        elif kind == "yarn":
            at = [rotary * math.log(origin / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (fast, slow)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary - 1)
            if hi <= lo:
                hi = lo + 0.001
            s = min(1.0, max(0.0, (j - lo) / (hi - lo)))
            theta = s * theta / factor + (1 - s) * theta
        out.append(theta)
    if attention is None:
        attention = 0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0
    return out, attention


def table(turns, attention, positions):
    """cos and sin rows from fixed-point turns, the angle reduced in whole numbers."""
    rows = []
    for p in positions:
        angle = [((int(p) * t) % (1 << 64)) / float(1 << 64) * 2 * math.pi for t in turns]
        rows.append([attention * math.cos(a) for a in angle] + [attention * math.sin(a) for a in angle])
    return np.array(rows).reshape(len(rows), 2 * len(turns))


def rotate(x, cos_sin, interleaved):
    """x [N, H, d] (float64) turned by cos_sin [N, rotary], and how far fp32
    arithmetic may be off: one rounding of a product and one of the sum, at most
    2^-23 of the terms' magnitudes together."""
    h = cos_sin.shape[1] // 2
    c, s = cos_sin[:, None, :h], cos_sin[:, None, h:]
    y, off = x.copy(), np.zeros(x.shape)
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    off[..., a] = 2.0 ** -23 * (np.abs(x[..., a] * c) + np.abs(x[..., b] * s))
    off[..., b] = 2.0 ** -23 * (np.abs(x[..., b] * c) + np.abs(x[..., a] * s))
    return y, off
