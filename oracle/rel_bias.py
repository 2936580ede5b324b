"""Plain float64 definition of attention with a learned relative position bias (CPU, NumPy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The score of query position i and key
position j is q.k * scale + table[bucket(j - i), h]; everything else is the attention of
``mha_ref`` and the chain rule of ``backward``.

The bucket of a distance d = j - i, in whole numbers: with ``per`` buckets of a side, e = per // 2
and n = |d|, a distance n >= e is in bucket e + t or a later one when
(n / e)^(per - e) >= (max_distance / e)^t, i.e. n^(per - e) >= e^(per - e - t) max_distance^t.
"""
from __future__ import annotations

import numpy as np

from .mha_ref import allowed_keys


def bucket_ref(d: int, num_buckets: int, max_distance: int, bidirectional: bool) -> int:
    per = num_buckets // 2 if bidirectional else num_buckets
    first = per if bidirectional and d > 0 else 0
    n = abs(d) if bidirectional else max(-d, 0)
    e = per // 2
    if n < e:
        return first + n
    t = 0
    while t + 1 < per - e and n ** (per - e) >= e ** (per - e - t - 1) * max_distance ** (t + 1):
        t += 1
    return first + e + t


def bucket_table(lo: int, hi: int, num_buckets, max_distance, bidirectional) -> np.ndarray:
    """bucket_ref of lo .. hi, far distances by their own last bucket."""
    return np.array([bucket_ref(max(min(d, 2 * max_distance), -2 * max_distance), num_buckets,
                                max_distance, bidirectional) for d in range(lo, hi + 1)])


def _scores(q, k, table, h, scale, first, how):
    """[Nq, Nk] scores of one head; query r is at position first + r."""
    Nq, Nk = q.shape[0], k.shape[0]
    scale = 1.0 / np.sqrt(q.shape[1]) if scale is None else scale
    lo = -(first + Nq - 1)
    u = bucket_table(lo, Nk - 1 - first, *how)
    d = np.arange(Nk)[None, :] - (first + np.arange(Nq))[:, None]
    return q @ k.T * scale + table[:, h][u[d - lo]], u[d - lo]


def _softmax(x, ok):
    x = np.where(ok, x, -np.inf)
    top = x.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(x - top)
    tot = e.sum(1, keepdims=True)
    p = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    with np.errstate(divide="ignore"):
        lse = np.where(tot > 0, top + np.log(tot), np.inf)
    return p, lse[:, 0]


def _cases(Q, K, mask, key_len):
    for b in range(Q.shape[0]):
        L = None if key_len is None else int(key_len[b])
        yield b, allowed_keys(mask, Q.shape[2], K.shape[2], L)


def _f64(*a):
    return [np.asarray(x, np.float64) for x in a]


def sdpa_rel_ref(Q, K, V, table, mask="none", key_len=None, scale=None, max_distance=128,
                 bidirectional=True):
    """(O [B,H,Nq,d_v], lse [B,H,Nq])."""
    Q, K, V, table = _f64(Q, K, V, table)
    how = (table.shape[0], max_distance, bidirectional)
    O = np.zeros(Q.shape[:3] + (V.shape[3],))
    lse = np.zeros(Q.shape[:3])
    for b, ok in _cases(Q, K, mask, key_len):
        for h in range(Q.shape[1]):
            x, _ = _scores(Q[b, h], K[b, h], table, h, scale, 0, how)
            p, lse[b, h] = _softmax(x, ok)
            O[b, h] = p @ np.where(ok.any(0)[:, None], V[b, h], 0.0)
    return O, lse


def sdpa_rel_bwd_ref(Q, K, V, table, dO, mask="none", key_len=None, scale=None, max_distance=128,
                     bidirectional=True, given=None):
    """(dQ, dK, dV, dtable) of sum(O * dO).  given = (O, lse): the softmax weights are exp(x - lse)
    and the row term is rowsum(dO * O), as in a backward that starts from a stored forward."""
    Q, K, V, table, dO = _f64(Q, K, V, table, dO)
    how = (table.shape[0], max_distance, bidirectional)
    dQ, dK, dV, dT = (np.zeros_like(a) for a in (Q, K, V, table))
    s = 1.0 / np.sqrt(Q.shape[3]) if scale is None else scale
    for b, ok in _cases(Q, K, mask, key_len):
        seen = ok.any(0)[:, None]
        for h in range(Q.shape[1]):
            k, v = np.where(seen, K[b, h], 0.0), np.where(seen, V[b, h], 0.0)
            x, u = _scores(Q[b, h], k, table, h, scale, 0, how)
            dP = dO[b, h] @ v.T
            if given is None:
                p, _ = _softmax(x, ok)
                D = (p * dP).sum(1, keepdims=True)
            else:
                p = np.where(ok, np.exp(x - np.asarray(given[1][b, h], np.float64)[:, None]), 0.0)
                D = (dO[b, h] * np.asarray(given[0][b, h], np.float64)).sum(1, keepdims=True)
            dS = p * (dP - D)
            dV[b, h] = p.T @ dO[b, h]
            dQ[b, h] = s * dS @ k
            dK[b, h] = s * dS.T @ Q[b, h]
            np.add.at(dT[:, h], u[ok], dS[ok])
    return dQ, dK, dV, dT


def table_grad_bound(Q, K, V, table, dO, O, lse, mask="none", key_len=None, scale=None,
                     max_distance=128, bidirectional=True):
    """[num_buckets, H] how far fp32 arithmetic may take dtable from sdpa_rel_bwd_ref(given=(O, lse)).

    A term is p (dP - D), p = exp(x - lse).  A sum of 64 fp32 products is off by at most 70 roundings
    of 2^-24 times the sum of their sizes, 70 * 2^-24 = 4.2e-6 (with factors of two tf32 terms 2^-21
    more).  For x that is 70 * 2^-24 * (sum |q k| scale, about 5 for normal q and k with scale
    1/sqrt(d), up to 7 over many pairs) < 3e-5 = 2^-15 of p with lse's own rounding; for dP and D it
    is 2^-17 of sum |dO V| and sum |dO O|; adding the terms up, at most 2^-24 times the number of
    additions in a row (under 2^8) of their sizes, 2^-16, is left to the first two."""
    Q, K, V, table, dO, O = _f64(Q, K, V, table, dO, O)
    how = (table.shape[0], max_distance, bidirectional)
    out = np.zeros_like(table)
    for b, ok in _cases(Q, K, mask, key_len):
        seen = ok.any(0)[:, None]
        for h in range(Q.shape[1]):
            k, v = np.where(seen, K[b, h], 0.0), np.where(seen, V[b, h], 0.0)
            x, u = _scores(Q[b, h], k, table, h, scale, 0, how)
            p = np.where(ok, np.exp(x - np.asarray(lse[b, h], np.float64)[:, None]), 0.0)
            D = (dO[b, h] * O[b, h]).sum(1, keepdims=True)
            size = np.abs(dO[b, h]) @ np.abs(v).T + (np.abs(dO[b, h] * O[b, h])).sum(1)[:, None]
            e = p * (2.0 ** -15 * (np.abs(dO[b, h] @ v.T) + np.abs(D)) + 2.0 ** -17 * size)
            np.add.at(out[:, h], u[ok], e[ok])
    return out


def element_bounds(Q, K, V, table, dO, half_step, arith, mask="none", key_len=None, scale=None,
                   max_distance=128, bidirectional=True):
    """(O, dQ, dK, dV): how far each element may be off, whatever the sizes.

    half_step: the type's rounding (bf16 2^-8, fp32 2^-24) of O, of P and dS as operands, and of each
    gradient as it is stored.  O = P V: half_step sum p |V| and half_step |O|.  D = rowsum(dO O) from
    the stored O: off by the sum of |dO| times O's bound.  dS = p (dP - D): half_step |dS| + p times
    D's.  dQ and dK sum those against |K| and |Q|, dV sums half_step p against |dO|.
    arith: what fp32 arithmetic adds to a weight or a product, relative to the sums of sizes: 2^-15
    (see table_grad_bound) and, in the backward, the stored log-sum-exp's rounding, 2^-24 of it."""
    Q, K, V, table, dO = _f64(Q, K, V, table, dO)
    how = (table.shape[0], max_distance, bidirectional)
    s = 1.0 / np.sqrt(Q.shape[3]) if scale is None else scale
    h8, small = half_step, arith
    bO, bQ, bK, bV = np.zeros(dO.shape), *(np.zeros_like(a) for a in (Q, K, V))
    for b, ok in _cases(Q, K, mask, key_len):
        seen = ok.any(0)[:, None]
        for h in range(Q.shape[1]):
            q, g = Q[b, h], dO[b, h]
            k, v = np.where(seen, K[b, h], 0.0), np.where(seen, V[b, h], 0.0)
            x, _ = _scores(q, k, table, h, scale, 0, how)
            p, _ = _softmax(x, ok)
            O, dP = p @ v, g @ v.T
            bO[b, h] = (h8 + small) * (p @ np.abs(v)) + h8 * np.abs(O)
            D = (p * dP).sum(1, keepdims=True)
            dS = p * (dP - D)
            size = np.abs(g) @ np.abs(v).T + np.abs(D)
            off = h8 * np.abs(dS) + p * (np.abs(g) * bO[b, h]).sum(1, keepdims=True) \
                + small * p * size
            bQ[b, h] = s * off @ np.abs(k) + h8 * np.abs(s * dS @ k)
            bK[b, h] = s * off.T @ np.abs(q) + h8 * np.abs(s * dS.T @ q)
            bV[b, h] = (h8 + small) * (p.T @ np.abs(g)) + h8 * np.abs(p.T @ g)
    return bO, bQ, bK, bV


def sdpa_rel_decode_ref(Q, K, V, table, cache_len, causal=True, scale=None, max_distance=128,
                        bidirectional=False):
    """O of one generation step: query r of sequence b is at position cache_len[b] - Nq + r."""
    Q, K, V, table = _f64(Q, K, V, table)
    how = (table.shape[0], max_distance, bidirectional)
    O = np.zeros(Q.shape[:3] + (V.shape[3],))
    Nq = Q.shape[2]
    for b in range(Q.shape[0]):
        L = min(max(int(cache_len[b]), 0), K.shape[2])
        if L == 0:
            continue
        pos = L - Nq + np.arange(Nq)
        ok = np.arange(L)[None, :] <= (pos[:, None] if causal else L)
        for h in range(Q.shape[1]):
            x, _ = _scores(Q[b, h], K[b, h, :L], table, h, scale, L - Nq, how)
            p, _ = _softmax(x, ok)
            O[b, h] = p @ V[b, h, :L]
    return O
