"""Float64 definitions of the operators around the 8-bit paged cache (norm_rope, append, read, attend).
All four are the library's own, without a counterpart in the pages."""
from __future__ import annotations

import numpy as np

BLOCK = 16
EXP_LOW, EXP_HIGH = -120, 121


def norm_rope(x, weight, eps, positions, inv_freq, axis, paired):
    """x [n,H,D], positions [n,axes].  Returns (out, size): |y_a| + |y_b| of the pair of each output, or |y|."""
    x = np.asarray(x, dtype=np.float64)
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    freq = np.asarray(inv_freq, dtype=np.float64)
    t = np.asarray(positions, dtype=np.float64)[:, np.asarray(axis)] * freq
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    p = freq.size
    a, b = (np.arange(0, 2 * p, 2), np.arange(1, 2 * p, 2)) if paired else (np.arange(p), np.arange(p, 2 * p))
    out, size = y.copy(), np.abs(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


def exponent(most):
    """The least e in range with every |x| <= most below 2^(e + 7)."""
    return int(np.clip(np.frexp(most)[1] - 7, EXP_LOW, EXP_HIGH)) if most > 0 else EXP_LOW


def codes_of(x, e):
    """floor(x 2^-e) + 128 of finite values; an infinity the code at its end, NaN code 0."""
    with np.errstate(invalid="ignore"):
        y = np.floor(np.ldexp(np.asarray(x, dtype=np.float64), -e))
    return np.clip(np.nan_to_num(y, nan=-128.0, posinf=127.0, neginf=-128.0), -128, 127).astype(np.int64) + 128


def append(k_codes, v_codes, exponents, K, V, starts, lengths, page_table):
    """Writes to the arrays given (numpy, changed in place)."""
    page, N = k_codes.shape[2], k_codes.shape[0]
    for b in range(len(lengths)):
        count, n = int(starts[b + 1] - starts[b]), int(lengths[b])
        for lo in range(n // BLOCK * BLOCK, n + count, BLOCK):
            if count == 0 or lo // page >= page_table.shape[1] or not 0 <= page_table[b, lo // page] < N:
                continue
            pg, r = page_table[b, lo // page], lo % page
            first, stop = max(lo, n), min(lo + BLOCK, n + count)
            rows = slice(starts[b] + first - n, starts[b] + stop - n)
            for of, (codes, x) in enumerate(((k_codes, K), (v_codes, V))):
                for h in range(codes.shape[1]):
                    new = np.asarray(x[rows, h], dtype=np.float64)
                    e = exponent(np.abs(new[np.isfinite(new)]).max(initial=0.0))
                    if first > lo:
                        was = int(exponents[pg, h, r // BLOCK, of])
                        e = max(e, was)
                        old = codes[pg, h, r:r + first - lo].astype(np.int64) - 128
                        codes[pg, h, r:r + first - lo] = (old >> min(e - was, 40)) + 128
                    codes[pg, h, r + first - lo:r + stop - lo] = codes_of(new, e)
                    exponents[pg, h, r // BLOCK, of] = e


def values(codes, exponents, of, pages, rows):
    """Values of the rows [len(rows), H, D]."""
    e = exponents[pages, :, rows // BLOCK, of].astype(np.float64)
    return (codes[pages, :, rows].astype(np.float64) - 127.5) * np.exp2(e)[..., None]


def attend(Q, k_codes, v_codes, exponents, starts, lengths, page_table, scale, window=0, sinks=0, logit_eps=0.0, value_eps=0.0, least=0.0):
    """Returns (out [n,Hq,D], bound).  Rows of no sequence are NaN in both.

    bound: how far out may be off where a logit is off by t <= logit_eps |scale| sum_d |q_d k_d|, a product
    p_i v_i by value_eps of it and by `least` of the largest p_j 2^e_j (times the code): a factor within
    exp(+-2 max t) on every weight, |out error| <= sum_i p_i |v_i| (exp(2 max t) - 1 + value_eps) +
    least * slots * 128 * max_j p_j 2^e_j."""
    n, Hq, D = Q.shape
    H, page, N = k_codes.shape[1], k_codes.shape[2], k_codes.shape[0]
    G = Hq // H
    out, bound = np.full((n, Hq, D), np.nan), np.full((n, Hq, D), np.nan)
    for b in range(len(lengths)):
        for i in range(starts[b], starts[b + 1]):
            at = int(lengths[b]) + i - int(starts[b])
            s = np.arange(at + 1)
            if window:
                s = s[(s > at - window) | (s < sinks)]
            s = s[s // page < page_table.shape[1]]
            pg = page_table[b, s // page]
            s, pg = s[(pg >= 0) & (pg < N)], pg[(pg >= 0) & (pg < N)]
            out[i], bound[i] = 0.0, 0.0
            if s.size == 0:
                continue
            k, v = values(k_codes, exponents, 0, pg, s % page), values(v_codes, exponents, 1, pg, s % page)
            step = np.exp2(exponents[pg, :, s % page // BLOCK, 1].astype(np.float64))
            for h in range(H):
                q = np.asarray(Q[i, h * G:(h + 1) * G], dtype=np.float64)
                z = scale * (q @ k[:, h].T)
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                t = logit_eps * abs(scale) * (np.abs(q) @ np.abs(k[:, h]).T).max(1, keepdims=True)
                out[i, h * G:(h + 1) * G] = p @ v[:, h]
                bound[i, h * G:(h + 1) * G] = ((np.expm1(2 * t) + value_eps) * (p @ np.abs(v[:, h]))
                                               + least * s.size * 128 * (p * step[:, h]).max(1, keepdims=True))
    return out, bound
