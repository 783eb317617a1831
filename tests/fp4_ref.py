"""Plain 64-bit definitions of the 4-bit pool's operators, for the tests.

Everything is numpy float64 or Python integers; nothing here uses the library
or its kernels.
"""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 16
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# the 127 finite non-negative e4m3 values by bit pattern
E4M3 = np.array([(f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
                 for e in range(16) for f in range(8)][:127])


def bf16_to_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest to x >= 0; a tie goes to the even index
    (the index is the format's bit pattern, so that is ties to even)."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where(a < b, lo, np.where(b < a, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(x: np.ndarray, exp: int):
    """(codes [..., D] 0..15, scale bytes [..., D/16]) of float64 x (from bf16)."""
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK)) * 2.0 ** -exp
    amax = np.abs(b).max(-1)  # NaN if the block has one
    nan = np.isnan(amax)
    sb = np.where(nan, 0x7F, nearest_even(np.where(nan, 0.0, amax) / 6, E4M3))
    s = E4M3[np.where(nan, 0, sb)][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        m = np.where(s > 0, np.abs(b) / s, 0.0)
    m = np.where(np.isnan(m), 0.0, m)
    codes = nearest_even(m, E2M1) + 8 * np.signbit(b)
    return codes.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(data: np.ndarray, scales: np.ndarray, exp: int) -> np.ndarray:
    """float64 [..., D] that packed data [..., D/2] and scale bytes [..., D/16] stand for."""
    codes = np.stack([data & 15, data >> 4], -1).reshape(data.shape[:-1] + (2 * data.shape[-1],))
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.append(E4M3, np.nan)[scales & 127] * np.where(scales & 128, -1.0, 1.0)
    return v * np.repeat(s, BLOCK, -1) * 2.0 ** exp


def decode(q, k, v, page_table, lens, sm_scale):
    """Attention of q [B, Hq, D] over k, v [R, Hkv, D] (float64), and per output
    the sum of weights times |v| (what a relative error of the weights scales
    with) and the largest |q||k| sum of a score."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, mag, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq))
    for r in range(B):
        n = int(lens[r])
        if n == 0:
            continue
        rows = np.asarray(page_table[r, :n])
        for g in range(Hkv):
            kk, vv = k[rows, g], v[rows, g]
            qq = q[r, g * G:(g + 1) * G]
            s = sm_scale * qq @ kk.T
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[r, g * G:(g + 1) * G] = w @ vv
            mag[r, g * G:(g + 1) * G] = w @ np.abs(vv)
            top[r, g * G:(g + 1) * G] = (np.abs(sm_scale) * np.abs(qq) @ np.abs(kk).T).max(1)
    return out, mag, top


def decode_bound(out, mag, top, vmax, n_max, weight_step=2.0 ** -11):
    """How far bf16 output may be from `out`: half a bf16 step of the result;
    the weights' rounding to fp16 (2^-11, or weight_step); each score's error d, from at most
    2^8 fp32 roundings (2^-24 each) of terms that sum to `top`, of the score
    itself and of its base-2 exponent, which moves a weight and the sum by
    e^d - 1 < 2d each; 2^-20 for the exponential, the sums and the merge; and
    weights below 2^-32 of the largest, which are lost."""
    d = (2.0 ** -16 + 2.0 ** -21) * (top + 1.0)
    weight = weight_step + 2.0 ** -20 + 4 * d
    return 2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * weight[..., None] * mag + n_max * 2.0 ** -32 * vmax + 1e-30


def build_slots(cached, extend, table, free, page, dummy, total):
    """The slots of one step: (table, out_loc, positions, q_offsets, seq_lens, pages)."""
    table = np.array(table)
    B, W = table.shape
    loc, pos = [dummy] * total, [0] * total
    off, ends, used = [0], [], 0
    for r in range(B):
        c, e = int(cached[r]), max(int(extend[r]), 0)
        start = max(c, 0)
        end = min(start + e, W)
        first = used
        owned = -(-start // page)
        if c >= 0:
            used += max(0, -(-end // page) - owned)
        for t in range(min(e, max(0, total - off[-1]))):
            p, row = start + t, dummy
            if p < W and c >= 0:
                if p < owned * page:
                    row = int(table[r, c - 1]) + p - (c - 1)
                elif first + p // page - owned < len(free):
                    row = int(free[first + p // page - owned]) * page + p % page
            if p < W:
                table[r, p] = row
            loc[off[-1] + t], pos[off[-1] + t] = row, p
        off.append(off[-1] + e)
        ends.append(end)
    return table, np.array(loc), np.array(pos), np.array(off), np.array(ends), used
