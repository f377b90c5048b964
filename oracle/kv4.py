"""The 4-bit cache's number format and attention with modified scores (fp64).  Test infrastructure only.

A row of 128 values is four groups of 32.  A group of values x holds
    z = min x                               (bf16, exact for bf16 inputs)
    s = (max x - min x) / 15 rounded to bf16 (nearest, ties to even), 0 below 2^-100
    n = (x - z) / s rounded to nearest, ties to even, within 0..15 (0 if s is 0)
and stands for s * n + z.  A group with a NaN, an infinity or a magnitude
above 2^126 stands for NaN.  All roundings here are made on exact rational
numbers where fp64 could be on the wrong side of a border.

Attention over such values: scores t_j = scale * q . k_j, capped by
softcap * tanh(t_j / softcap), less slope * |pos_q - pos_j|, over the keys that
the query sees; rows that see nothing give 0.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

GROUP = 32


def _bf16_bits_of_fraction(v: Fraction) -> int:
    """bf16 bits (sign 0) of a non-negative rational, rounded to nearest even."""
    if v == 0:
        return 0
    e = v.numerator.bit_length() - v.denominator.bit_length()   # v in (2^(e-1), 2^(e+1))
    if v < Fraction(2) ** e:
        e -= 1
    e = max(e, -126)
    unit = Fraction(2) ** (e - 7)
    n = round(v / unit)                                         # Python rounds halves to even
    if n == 256:
        n, e = 128, e + 1
    if e + 127 > 254:
        return 0x7F80
    return n if n < 128 else ((e + 127) << 7) | (n - 128)


def quantise_group(x: np.ndarray):
    """One group of 32 fp64 values (each a bf16 number) -> (codes [32], s, z) with s, z fp64."""
    if not np.all(np.isfinite(x)) or np.max(np.abs(x)) > 2.0 ** 126:
        return np.zeros(GROUP, dtype=np.uint8), np.nan, np.nan
    lo, hi = Fraction(float(x.min())), Fraction(float(x.max()))
    bits = _bf16_bits_of_fraction((hi - lo) / 15)
    s = float(np.array([bits << 16], dtype=np.uint32).view(np.float32)[0])
    if s < 2.0 ** -100:
        return np.zeros(GROUP, dtype=np.uint8), 0.0, float(lo)
    fs = Fraction(s)
    n = [min(15, max(0, round((Fraction(float(v)) - lo) / fs))) for v in x]
    return np.array(n, dtype=np.uint8), s, float(lo)


def quantise_rows(x: np.ndarray):
    """x [rows][128] fp64 -> codes uint8 [rows][128], s [rows][4], z [rows][4] (fp64)."""
    R, d = x.shape
    codes = np.zeros((R, d), dtype=np.uint8)
    s, z = np.zeros((R, d // GROUP)), np.zeros((R, d // GROUP))
    for r in range(R):
        for g in range(d // GROUP):
            codes[r, g * GROUP:(g + 1) * GROUP], s[r, g], z[r, g] = quantise_group(x[r, g * GROUP:(g + 1) * GROUP])
    return codes, s, z


def values(codes: np.ndarray, s: np.ndarray, z: np.ndarray) -> np.ndarray:
    """s * n + z, fp64, codes [..., 128], s and z [..., 4]."""
    return codes.astype(np.float64) * np.repeat(s, GROUP, -1) + np.repeat(z, GROUP, -1)


def unpack(codes_bytes: np.ndarray) -> np.ndarray:
    """[..., 64] bytes -> [..., 128] codes: value 2i in the low half of byte i."""
    out = np.empty(codes_bytes.shape[:-1] + (codes_bytes.shape[-1] * 2,), dtype=np.uint8)
    out[..., 0::2] = codes_bytes & 15
    out[..., 1::2] = codes_bytes >> 4
    return out


def modified_scores(t: np.ndarray, distance: np.ndarray, softcap: float, slope: float) -> np.ndarray:
    if softcap > 0:
        t = softcap * np.tanh(t / softcap)
    return t - slope * np.abs(distance)


def masked_softmax(t: np.ndarray, seen: np.ndarray):
    """(p, log-sum-exp) of a 1-d score row over the seen keys; zeros and -inf if there are none."""
    p = np.zeros(t.shape)
    if not seen.any():
        return p, -np.inf
    m = t[seen].max()
    e = np.exp(t[seen] - m)
    p[seen] = e / e.sum()
    return p, m + np.log(e.sum())


def decode(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, pos: np.ndarray, pos_q: int, softcap=0.0,
           slopes=None, window=0, n_sink=0):
    """q [G][d], k and v [S][d], pos [S] -> out [G][d], p [G][S].  Keys that are not seen may hold anything."""
    G, S = q.shape[0], k.shape[0]
    seen = np.ones(S, dtype=bool)
    if window > 0:
        seen = (pos_q - pos < window) | (pos < n_sink)
    out, p = np.zeros((G, v.shape[1])), np.zeros((G, S))
    for h in range(G):
        t = np.zeros(S)
        t[seen] = modified_scores(k[seen] @ q[h] * scale, pos_q - pos[seen], softcap, 0.0 if slopes is None else slopes[h])
        p[h], _ = masked_softmax(t, seen)
        out[h] = p[h][seen] @ v[seen]
    return out, p


def prefill(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, softcap=0.0, slope=0.0, window=0, prefix=0,
            doc_start=None):
    """One q head of one sequence: q [n][d] are its last n tokens, k and v [S][d].  -> out [n][d], lse [n]."""
    n, S = q.shape[0], k.shape[0]
    j = np.arange(S)
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    for i in range(n):
        pos = S - n + i
        seen = j <= pos
        if window > 0:
            seen &= pos - j < window
        seen |= j < prefix
        if doc_start is not None:
            seen &= j >= doc_start[i]
        t = np.zeros(S)
        t[seen] = modified_scores(k[seen] @ q[i] * scale, pos - j[seen], softcap, slope)
        p, lse[i] = masked_softmax(t, seen)
        out[i] = p[seen] @ v[seen]
    return out, lse
