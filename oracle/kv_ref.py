"""fp64 definitions of the paged key/value cache, its E4M3 form, and attention over keys of another length.

numpy only, written from the formulas and row by row: a cache is [num_pages, Hkv, page, D], position p of sequence b
is row p % page of page table[b][p // page]; an E4M3 row holds code * 2^e with e the least integer >= -120 such that
its largest magnitude is at most 448 * 2^e.
"""
from __future__ import annotations

import math

import numpy as np

E8_NAN = 255


def round_e4m3(x: float) -> float:
    """The E4M3 number nearest to x, |x| <= 448 (ties to even): 3 mantissa bits, least normal 2^-6."""
    if x == 0.0:
        return 0.0
    e = max(math.frexp(abs(x))[1] - 1, -6)
    step = math.ldexp(1.0, e - 3)
    return round(x / step) * step   # Python rounds halves to even


def quantise_row(row):
    """(codes as fp64 values, E8M0 byte) of one row."""
    row = np.asarray(row, dtype=np.float64)
    if not np.all(np.isfinite(row)):
        return np.zeros_like(row), E8_NAN
    amax = float(np.abs(row).max())
    e = -120
    while amax > 448.0 * 2.0 ** e:
        e += 1
    codes = np.array([round_e4m3(float(x) * 2.0 ** -e) for x in row])
    if e >= 120:
        codes = np.clip(codes, -240.0, 240.0)
    return codes, e + 127


def e8_value(byte: int) -> float:
    return math.nan if byte == E8_NAN else 2.0 ** (int(byte) - 127)


def page_row(table_row, page: int, num_pages: int, pos: int):
    """(page, row) of a position, or None where the table has no page for it."""
    if pos < 0 or pos // page >= len(table_row):
        return None
    i = int(table_row[pos // page])
    return (i, pos % page) if 0 <= i < num_pages else None


def gather(cache, scale, table_row, n: int):
    """Positions [0, n) behind one table row: fp64 [Hkv, n, D]; rows without a page are zero.  cache holds fp64
    values (of the codes, where scale, a byte array, is given)."""
    num_pages, hkv, page, d = cache.shape
    out = np.zeros((hkv, n, d))
    for p in range(n):
        at = page_row(table_row, page, num_pages, p)
        if at is None:
            continue
        for h in range(hkv):
            s = 1.0 if scale is None else e8_value(scale[at[0], h, at[1]])
            out[h, p] = cache[at[0], h, at[1]] * s
    return out


def attend(q, k, v, lims, scale: float):
    """q [Hq, T, D], k, v [Hkv, n, D]; query t sees keys j < lims[t].  Returns o, lse and, for tolerances,
    a = sum_j p_j |v_j| and the largest sum_d |q_d k_jd| of each row."""
    Hq, T, D = q.shape
    group = Hq // k.shape[0]
    o, a = np.zeros((Hq, T, D)), np.zeros((Hq, T, D))
    lse, top = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for h in range(Hq):
        for t in range(T):
            n = max(0, min(int(lims[t]), k.shape[1]))
            if n == 0:
                continue
            kk, vv = k[h // group, :n], v[h // group, :n]
            s = scale * (kk @ q[h, t])
            m = s.max()
            w = np.exp(s - m)
            total = w.sum()
            o[h, t], a[h, t] = (w / total) @ vv, (w / total) @ np.abs(vv)
            lse[h, t] = m + math.log(total)
            top[h, t] = (np.abs(kk) @ np.abs(q[h, t])).max()
    return o, lse, a, top


def cross_backward(q, k, v, do, n: int, scale: float):
    """Gradients of one batch row of cross attention over its first n keys: dq [Hq, Nq, D], dk, dv [Hkv, Nk, D]."""
    Hq, group = q.shape[0], q.shape[0] // k.shape[0]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(Hq) if n > 0 else ():
        g = h // group
        s = scale * (q[h] @ k[g, :n].T)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        dp = do[h] @ v[g, :n].T
        ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
        dq[h] = scale * ds @ k[g, :n]
        dk[g, :n] += scale * ds.T @ q[h]
        dv[g, :n] += p.T @ do[h]
    return dq, dk, dv
