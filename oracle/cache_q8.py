"""The 8-bit key/value cache in float64 NumPy, one token, block and head at a time.

A cache is a dict of k, v (uint8 bytes [B, H, Lmax, 64]), k_scale, v_scale (float64
[B, H, blocks]) and weights ([B, H, Lmax]).  ``code`` is "e4m3" or "int8".
"""
from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_value(byte: int) -> float:
    """1 sign bit, 4 exponent bits (bias 7), 3 mantissa bits; S.1111.111 is NaN, no infinity."""
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return float("nan")
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if s else v


TABLE = {"e4m3": np.array([e4m3_value(b) for b in range(256)]),
         "int8": np.array([b - 256.0 if b > 127 else float(b) for b in range(256)])}


def values_ref(codes, code: str) -> np.ndarray:
    """The numbers that the bytes stand for, without their scale."""
    return TABLE[code][np.asarray(codes, np.uint8)]


def encode_ref(x, code: str) -> np.ndarray:
    """Bytes of the nearest codes to x (ties to the even mantissa or integer), saturating; NaN
    stays NaN in e4m3 and becomes 0 in int8."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    y = np.clip(np.where(nan, 0.0, x), -QMAX[code], QMAX[code])
    if code == "int8":
        return np.rint(y).astype(np.int64).astype(np.uint8)  # rint: ties to even
    mags = TABLE["e4m3"][:127]                    # 0 .. 448, ascending, index = byte
    a = np.abs(y)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)  # mags[hi - 1] <= a <= mags[hi]
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a           # exact: neighbours share an exponent
    byte = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    byte = byte | np.where(np.signbit(y), 128, 0)
    return np.where(nan, 127, byte).astype(np.uint8)


def scale_ref(x, code: str) -> float:
    """The least power of two s with |x| <= QMAX s over the finite x, exponent in [-40, 40]."""
    x = np.abs(np.asarray(x, np.float64))
    amax = float(x[np.isfinite(x)].max(initial=0.0))
    e = -40
    while e < 40 and amax > QMAX[code] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def times_ref(x, factor) -> np.ndarray:
    """x * factor, exact for powers of two, else as the header says: factor and product in fp32."""
    x, factor = np.broadcast_arrays(np.asarray(x, np.float64), np.asarray(factor, np.float64))
    rounded = x.astype(np.float32) * factor.astype(np.float32)
    return np.where(np.frexp(factor)[0] == 0.5, x * factor, rounded)


def append_ref(cache: dict, k, v, cache_len, new_len, block: int, code: str) -> dict:
    """The cache after token i < new_len[b] of k, v went to position cache_len[b] + i."""
    out = {n: np.array(a) for n, a in cache.items()}
    B, H, Lmax, _ = cache["k"].shape
    for b in range(B):
        L = int(np.clip(cache_len[b], 0, Lmax))
        n = k.shape[2] if new_len is None else int(np.clip(new_len[b], 0, k.shape[2]))
        end = min(L + n, Lmax)
        for blk in range(-(-Lmax // block)):
            lo, hi = max(L, blk * block), min(end, (blk + 1) * block)
            if lo >= hi:
                continue
            for h in range(H):
                for name, x in (("k", k), ("v", v)):
                    new = np.asarray(x[b, h, lo - L:hi - L], np.float64)
                    s = scale_ref(new, code)
                    if lo > blk * block:
                        was = float(out[name + "_scale"][b, h, blk])
                        s = max(s, was)
                        if s > was:
                            rows = slice(blk * block, lo)
                            old = times_ref(values_ref(out[name][b, h, rows], code), was / s)
                            out[name][b, h, rows] = encode_ref(old, code)
                    out[name + "_scale"][b, h, blk] = s
                    out[name][b, h, lo:hi] = encode_ref(times_ref(new, 1 / s), code)
                out["weights"][b, h, lo:hi] = 0.0
    return out


def dequantised_ref(cache: dict, name: str, b: int, h: int, L: int, block: int, code: str):
    s = cache[name + "_scale"][b, h, np.arange(L) // block].astype(np.float64)
    return values_ref(cache[name][b, h, :L], code) * s[:, None]


def decode_ref(Q, cache: dict, cache_len, block: int, code: str, causal: bool, scale=None):
    """(O, added weights, sum_j p |v|, max_j(p s) sum_j |code| with s the value's scale, largest
    sum |q||k| scale of a row): the attention of Q [B, Hq, Nq, 64] over the cache, and the three
    sizes its rounding errors go by."""
    B, Hq, Nq, D = Q.shape
    H, Lmax = cache["k"].shape[1:3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    O = np.zeros((B, Hq, Nq, D))
    W = np.zeros((B, H, Lmax))
    pv, low, qk = np.zeros_like(O), np.zeros_like(O), 0.0
    for b in range(B):
        L = int(np.clip(cache_len[b], 0, Lmax))
        for h in range(H):
            k = dequantised_ref(cache, "k", b, h, L, block, code)
            v = dequantised_ref(cache, "v", b, h, L, block, code)
            for g in range(G):
                for i in range(Nq):
                    n = max(L - Nq + 1 + i, 0) if causal else L
                    if n == 0:
                        continue
                    q = np.asarray(Q[b, h * G + g, i], np.float64)
                    s = k[:n] @ q * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    O[b, h * G + g, i] = p @ v[:n]
                    pv[b, h * G + g, i] = p @ np.abs(v[:n])
                    W[b, h, :n] += p
                    s = cache["v_scale"][b, h, np.arange(n) // block]
                    low[b, h * G + g, i] = (p * s).max() * np.abs(v[:n] / s[:, None]).sum(0)
                    qk = max(qk, float((np.abs(k[:n]) @ np.abs(q)).max() * scale))
    return O, W, pv, low, qk


def key_weights_ref(Q, K, lse, mask: str, key_len=None, query_len=None, scale=None):
    """Column sums [B, H, Nk] of exp(q k scale - lse) over the allowed pairs."""
    B, Hq, Nq, D = Q.shape
    H, Nk = K.shape[1:3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    W = np.zeros((B, H, Nk))
    for b in range(B):
        nk = Nk if mask != "key_padding" else int(np.clip(key_len[b], 0, Nk))
        nq = Nq if query_len is None else int(np.clip(query_len[b], 0, Nq))
        for h in range(Hq):
            s = np.asarray(Q[b, h, :nq], np.float64) @ np.asarray(K[b, h // G, :nk], np.float64).T
            p = np.exp(s * scale - np.asarray(lse[b, h, :nq], np.float64)[:, None])
            if mask == "causal":
                p = np.where(np.arange(nk) <= np.arange(nq)[:, None], p, 0.0)
            W[b, h // G, :nk] += p.sum(0)
    return W


def kept_ref(weights, L: int, keep: int, recent: int) -> list[int]:
    """The positions of one head that stay, ascending."""
    if L <= keep:
        return list(range(L))
    recent = min(recent, keep)
    w = [(-np.inf if np.isnan(x) else float(x)) for x in weights[:L - recent]]
    best = sorted(range(len(w)), key=lambda j: (-w[j], j))[:keep - recent]
    return sorted(best) + list(range(L - recent, L))


def evict_ref(cache: dict, out: dict, cache_len, keep: int, recent: int, block: int, code: str):
    """(the new cache, its lengths, the kept positions)."""
    out = {n: np.array(a) for n, a in out.items()}
    B, H, Lmax, _ = cache["k"].shape
    kept = np.full((B, H, keep), -1, np.int32)
    length = np.zeros(B, np.int32)
    for b in range(B):
        L = int(np.clip(cache_len[b], 0, Lmax))
        length[b] = min(L, keep)
        for h in range(H):
            at = kept_ref(cache["weights"][b, h], L, keep, recent)
            kept[b, h, :len(at)] = at
            for lo in range(0, len(at), block):
                src = np.array(at[lo:lo + block])
                for name in ("k", "v"):
                    was = cache[name + "_scale"][b, h, src // block]
                    s = was.max()
                    vals = times_ref(values_ref(cache[name][b, h, src], code), (was / s)[:, None])
                    out[name][b, h, lo:lo + len(src)] = np.where(
                        (was == s)[:, None], cache[name][b, h, src], encode_ref(vals, code))
                    out[name + "_scale"][b, h, lo // block] = s
                out["weights"][b, h, lo:lo + len(src)] = cache["weights"][b, h, src]
    return out, length, kept
