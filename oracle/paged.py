"""Float64 definitions of the paged-cache operators (append, decode, evict), over the row
format of :func:`oracle.compress_mse`.  Paging, ragged lengths and eviction are the
library's own; the quantizer and the rotated-domain decode are the pages'."""
from __future__ import annotations

import numpy as np

from .tq_oracle import compress_mse, pack_indices, unpack_indices


def slot_rows(page_table: np.ndarray, b: int, n: int, page: int):
    """Pages and rows of slots 0 .. n-1 of sequence b."""
    s = np.arange(n)
    return page_table[b, s // page], s % page


def append_rows(x: np.ndarray, Pi: np.ndarray, codebook: np.ndarray, bits: int):
    """Packed codes [n,H,D*bits/8] and fp16 lengths [n,H] of rows x [n,H,D]; KV head h is
    rotated by Pi[h % len(Pi)].  A zero row takes the cells of 0."""
    n, H, D = x.shape
    planes = np.empty((n, H, D * bits // 8), np.uint8)
    norms = np.empty((n, H), np.float16)
    for h in range(H):
        v = np.asarray(x[:, h], dtype=np.float64)
        zero = ~v.any(axis=1)
        v = np.where(zero[:, None], 1.0, v)
        idx, norm = compress_mse(v, Pi[h % len(Pi)], codebook)
        c = np.asarray(codebook, dtype=np.float64)
        idx[zero] = int((0.5 * (c[1:] + c[:-1]) < 0).sum())
        planes[:, h], norms[:, h] = pack_indices(idx, bits), np.where(zero, 0.0, norm)
    return planes, norms


def border_gap(x: np.ndarray, Pi: np.ndarray, codebook: np.ndarray) -> np.ndarray:
    """Distance of each rotated unit coordinate from the nearest midpoint, [n,H,D]."""
    c = np.asarray(codebook, dtype=np.float64)
    mid = 0.5 * (c[1:] + c[:-1])
    gaps = np.empty(x.shape)
    for h in range(x.shape[1]):
        v = np.asarray(x[:, h], dtype=np.float64)
        n = np.sqrt((v * v).sum(1, keepdims=True))
        y = (v / np.where(n > 0, n, 1.0)) @ np.asarray(Pi[h % len(Pi)], dtype=np.float64).T
        gaps[:, h] = np.abs(y[..., None] - mid).min(-1)
    return gaps


def decode_paged(Q, k_plane, k_norm, v_plane, v_norm, page_table, lengths, Pi_k, k_codebook, Pi_v, v_codebook,
                 scale, operand_eps=0.0, value_eps=0.0):
    """Returns (out [B,Hq,D], weights [B,H,G,S] (0 behind a length), bound [B,Hq,D], wrel
    [B,H,G]: the relative bound of the weights).  A page number outside [0, N) makes its slots
    absent.

    bound: how far out may be off where every operand of the key products carries a relative
    error of `operand_eps` and every operand of the value products one of `value_eps`.  With
    e = operand_eps, |logit error| <= t_i = scale nk_i (2e + e^2) sum_d |a_d c_d|, so a weight
    changes by a factor within exp(+-2 max t), and
    |out error| <= sum_j |Pi_v[j,:]| sum_i p_i nv_i |c_ij| (exp(2 max t) - 1 + 2 value_eps + value_eps^2)."""
    N, H, page, _ = k_plane.shape
    D = Q.shape[-1]
    kb, vb = k_plane.shape[-1] * 8 // D, v_plane.shape[-1] * 8 // D
    B, Hq = Q.shape[:2]
    G, S = Hq // H, page_table.shape[1] * page
    Pi_k, Pi_v = (np.asarray(P, dtype=np.float64) for P in (Pi_k, Pi_v))
    kc, vc = (np.asarray(c, dtype=np.float64) for c in (k_codebook, v_codebook))
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    weights, wrel = np.zeros((B, H, G, S)), np.zeros((B, H, G))
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        pg, r = slot_rows(page_table, b, n, page)
        there = np.flatnonzero((pg >= 0) & (pg < N))
        if there.size == 0:
            continue
        pg, r = pg[there], r[there]
        for h in range(H):
            ck = kc[unpack_indices(k_plane[pg, h, r], kb, D)]
            cv = vc[unpack_indices(v_plane[pg, h, r], vb, D)]
            nk, nv = k_norm[pg, h, r].astype(np.float64), v_norm[pg, h, r].astype(np.float64)
            q = np.asarray(Q[b, h * G:(h + 1) * G], dtype=np.float64)
            a = q @ Pi_k[h % len(Pi_k)].T
            s = scale * (a @ ck.T) * nk
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            weights[b, h][:, there] = p
            P = Pi_v[h % len(Pi_v)]
            out[b, h * G:(h + 1) * G] = ((p * nv) @ cv) @ P
            t = (abs(scale) * nk * (np.abs(a) @ np.abs(ck).T)).max(axis=1, keepdims=True)
            grow = np.expm1(2 * t * (2 * operand_eps + operand_eps ** 2))
            wrel[b, h] = grow[:, 0]
            f = grow + 2 * value_eps + value_eps ** 2
            bound[b, h * G:(h + 1) * G] = f * (((p * nv) @ np.abs(cv)) @ np.abs(P))
    return out, weights, bound, wrel


def evict_paged(mass, positions, lengths, seen, budget, recent):
    """For each (sequence, head): (kept slots ascending, slots filled, slots they are filled
    from).  Preference: positions >= seen - recent before the others, among either
    mass (NaN as -inf), then the lower slot."""
    B, H, S = mass.shape
    got = {}
    for b in range(B):
        n = int(lengths[b])
        keep = min(n, budget)
        for h in range(H):
            m = mass[b, h, :n].astype(np.float64)
            m = np.where(np.isnan(m), -np.inf, m)
            safe = positions[b, h, :n].astype(np.int64) >= int(seen[b]) - recent
            order = sorted(range(n), key=lambda s: (not safe[s], -m[s], s))
            kept = np.array(sorted(order[:keep]), dtype=np.int64)
            got[b, h] = (kept, np.setdiff1d(np.arange(keep), kept), kept[kept >= keep])
    return got
