"""Plain 64-bit forms of the key/value cache calls, on the CPU, and how far a call may be from them.

Written from the definitions in include/pivot.h with loops over rows and blocks; no code of the library.

Tolerances (each rounding is off by at most half a step relative to the value: bf16 2^-8, fp32 2^-24, e4m3 2^-4):
  scores   z = scale q.k, d products summed in fp32: |dz| <= (d + 8) 2^-24 scale sum|q_i k_i|; a bf16 query may
           enter in two e4m3 parts, exact but for what lies below 2^-18 of the row's largest |q|.
  weights  p is off by dz relative, and by its own rounding: 8 bits at least for bf16 (2^-8, and 2^-18 of the
           largest term), 21 for fp32 (2^-21).
  output   sum p v / sum p: those, and n additions in fp32 (2^-24 each), all relative to A = sum p|v| / sum p;
           and the output type's own rounding.
  lse      dz and n additions, and 2^-21 of its own size (the exponentials and the logarithm are fp32).
"""
import math

import numpy as np
import torch

BLOCK, E_MIN, E_MAX = 16, -60, 60


def e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def round_e4m3(x):
    """Nearest e4m3 value, ties to even, saturating; NaN stays (numpy float64 in and out)."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    with np.errstate(all="ignore"):
        e = np.maximum(np.floor(np.log2(np.where((a > 0) & np.isfinite(a), a, 1.0))), -6)
    e = np.where(2.0 ** e > np.maximum(a, 2.0 ** -6), e - 1, e)
    e = np.where(2.0 ** (e + 1) <= a, e + 1, e)
    ulp = 2.0 ** (e - 3)
    with np.errstate(all="ignore"):
        y = np.minimum(np.round(a / ulp) * ulp, 448.0)
    y = np.where(np.isinf(x), 448.0, y)
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def rows_of(off, lens, rows):
    """[(row, sequence, position)] of the rows that belong to a sequence."""
    out = []
    for b in range(len(lens)):
        for r in range(off[b], off[b + 1]):
            out.append((r, b, lens[b] - off[b + 1] + r))
    return [t for t in out if t[0] < rows]


def page_of(table, b, s, page, pages):
    i = s // page
    if i >= table.shape[1]:
        return -1
    p = int(table[b, i])
    return p if 0 <= p < pages else -1


def rotate(x, cos, sin, interleaved):
    """x [heads, d] float64; one position's cos, sin [rot/2]."""
    h = cos.shape[0]
    y = x.copy()
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y[:, a], y[:, b] = x[:, a] * cos - x[:, b] * sin, x[:, b] * cos + x[:, a] * sin
    return y


def exponent(y):
    """The least e with |y| <= 448 * 2^e for the finite values."""
    y = np.abs(y[np.isfinite(y)])
    top = y.max() if y.size else 0.0
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(pay, exps, table, off, lens, x, cos, sin, interleaved):
    """pay [pages, heads, page, d] float64 payload values, exps int: both changed in place.  Also returns
    {(page, head, slot): (exact value, its uncertainty in fp32)} of the new tokens."""
    pages, heads, page, d = pay.shape
    rows = [t for t in rows_of(off, lens, x.shape[0]) if 0 <= t[2]]
    blocks = {}
    for r, b, p in rows:
        pg = page_of(table, b, p, page, pages)
        if pg >= 0:
            blocks.setdefault((b, p // BLOCK, pg), []).append((r, p))
    exact = {}
    for (b, blk, pg), toks in blocks.items():
        first = toks[0][1]
        in_page = blk * BLOCK % page
        ys, mags = [], []
        for r, p in toks:
            y, mag = x[r].copy(), np.zeros_like(x[r])
            if cos is not None:
                with np.errstate(all="ignore"):
                    y = rotate(x[r], cos[p], sin[p], interleaved)
                    mag = rotate(np.abs(x[r]), np.abs(cos[p]), -np.abs(sin[p]), interleaved)
                    mag = np.maximum(mag, rotate(np.abs(x[r]), np.abs(cos[p]), np.abs(sin[p]), interleaved))
            ys.append(y), mags.append(np.abs(mag) * 3 * 2.0 ** -24)
        for h in range(heads):
            e = exponent(np.concatenate([y[h] for y in ys]))
            if first % BLOCK:
                was = int(exps[pg, h, in_page // BLOCK])
                if e > was:
                    old = pay[pg, h, in_page:in_page + first % BLOCK]
                    old[:] = round_e4m3(old * 2.0 ** (was - e))
                e = max(e, was)
            exps[pg, h, in_page // BLOCK] = e
            for (r, p), y, mag in zip(toks, ys, mags):
                pay[pg, h, p % page] = round_e4m3(y[h] * 2.0 ** -e)
                exact[pg, h, p % page] = (y[h] * 2.0 ** -e, mag[h] * 2.0 ** -e)
    return exact


def attention(q, pay_k, pay_v, k_exp, v_exp, table, off, lens, scale, dtype, window=0, sinks=0, indices=None):
    """out, lse, and how far a call's may be from them; rows of no sequence are NaN."""
    rows, hq, d = q.shape
    pages, hk, page, _ = pay_k.shape
    group = hq // hk
    out = np.full((rows, hq, d), np.nan)
    lse = np.full((rows, hq), np.nan)
    out_tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    bf16 = dtype == torch.bfloat16
    for r, b, p in rows_of(off, lens, rows):
        if indices is None:
            s = np.arange(0, min(p, table.shape[1] * page - 1) + 1)
            if window:
                s = s[(s > p - window) | (s < sinks)]
        else:
            s = indices[r].astype(np.int64)
            s = s[(s >= 0) & (s <= p)]
        pg = np.array([page_of(table, b, int(t), page, pages) for t in s], np.int64)
        s, pg = s[pg >= 0], pg[pg >= 0]
        if s.size == 0:
            out[r], lse[r] = 0.0, -np.inf
            continue
        for j in range(hq):
            h = j // group
            k = pay_k[pg, h, s % page] * 2.0 ** k_exp[pg, h, s % page // BLOCK].astype(float)[:, None]
            v = pay_v[pg, h, s % page] * 2.0 ** v_exp[pg, h, s % page // BLOCK].astype(float)[:, None]
            with np.errstate(all="ignore"):
                z = k @ q[r, j] * scale
                m = z.max()
                w = np.exp(z - m)
                total = w.sum()
                out[r, j] = w @ v / total
                lse[r, j] = m + math.log(total) if total > 0 else np.nan
                dz = (np.abs(k) @ np.abs(q[r, j]) * (d + 8) * 2.0 ** -24 * abs(scale)).max()
                if bf16:
                    dz += np.abs(q[r, j]).max() * np.abs(k).sum(1).max() * 2.0 ** -18 * abs(scale)
                A = w @ np.abs(v) / total
                part = 2.0 ** -8 if bf16 else 2.0 ** -21
                far = 2.0 ** -18 * s.size * (w[:, None] * np.abs(v)).max() / total if bf16 else 0.0
                out_tol[r, j] = (2 * dz + part + (s.size + 16) * 2.0 ** -24) * A + far + \
                    (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(out[r, j]) * 1.01 + 1e-30
                lse_tol[r, j] = dz + (s.size + 16) * 2.0 ** -24 + 2.0 ** -21 * (abs(lse[r, j]) + abs(m) + 1)
    return out, lse, out_tol, lse_tol
