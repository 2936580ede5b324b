"""The 8-bit key/value cache on the GPU against its float64 oracle.

Bounds, from the arithmetic.  Codes, scales, lengths and positions are equal.  A score is a sum
of 64 products, each sum rounded once to fp32 (at most half a step, 2^-24 of the running size),
so it is off by at most 64 * 2^-24 * S = 2^-18 S with S = scale * sum |q||k|; a softmax weight
(a ratio of two exponentials) by twice that relatively, plus 2^-19 for the exponentials and the
division.  With n keys added in fp32 the sums are off by n * 2^-24.  The weights
p_j s_j that meet the value codes are fp16, scaled so that the row's largest is 2^13: below 2^-14
an fp16 (of the fp32 path, the second of its two terms) is off by up to half its least step, 2^-25
or 2^-38 of that largest, whatever its own size.  The bf16 path rounds those weights once (2^-11)
and the output to bf16 (2^-8).  Hence
    |O - ref| <= r * sum_j p_j |v_j| + 2^-38 max_j(p_j s_j) sum_j |code_j| (+ 2^-8 |ref|),
    r = 2^-17 S + n 2^-24 + 2^-19 (+ 2^-11)
    |W - ref| <= r * ref  without the bf16 terms (weights are fp32 on both paths).
"""
import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from oracle import cache_q8 as oq

pytestmark = pytest.mark.gpu

mha = pytest.importorskip("transformer_head_scaled_04_gb300")
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_head_scaled_04_gb300 import build

    build.build()
    mha.load_library()
    torch.cuda.set_device(0)
    mha.device_status()
    yield
    assert mha.device_status() == 0, "a kernel recorded a device-side error"


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def fin(a, dtype):
    return si.round_bf16(a) if dtype == "bf16" else np.asarray(a, np.float32)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def strange(g, B, H, Lmax, block, code):
    """A cache dict of arbitrary bytes (NaN codes among them), power-of-two scales and weights."""
    nb = -(-Lmax // block)
    c = {n: g.integers(0, 256, (B, H, Lmax, 64)).astype(np.uint8) for n in "kv"}
    for n in "kv":
        if code == "int8":
            c[n][c[n] == 128] = 127
        c[n + "_scale"] = 2.0 ** g.integers(-9, 3, (B, H, nb))
    c["weights"] = g.random((B, H, Lmax)).astype(np.float32).astype(np.float64)
    return c


def finite(c, code):
    for n in "kv":
        if code == "e4m3":
            c[n][(c[n] & 127) == 127] = 0
    return c


def to_gpu(c, block, code, token_major=False):
    def put(x):
        t = dev(x)
        if token_major:  # [B, Lmax, H, 64] in memory
            t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        return t.view(CODE[code])

    return mha.KvCacheQ8(put(c["k"]), put(c["v"]), dev(c["k_scale"], torch.float32),
                         dev(c["v_scale"], torch.float32), dev(c["weights"], torch.float32), block)


def from_gpu(cache):
    return {"k": cache.k.view(torch.uint8).cpu().numpy(),
            "v": cache.v.view(torch.uint8).cpu().numpy(),
            "k_scale": cache.k_scale.double().cpu().numpy(),
            "v_scale": cache.v_scale.double().cpu().numpy(),
            "weights": cache.weights.double().cpu().numpy()}


def assert_same(got, want, code, what):
    for n in want:
        a, b = np.asarray(got[n]), np.asarray(want[n])
        if n in "kv" and code == "e4m3":  # a NaN may carry either sign
            a = np.where((a & 127) == 127, 127, a)
            b = np.where((b & 127) == 127, 127, b)
        bad = np.argwhere(a != b)
        assert bad.size == 0, f"{what}: {n} differs at {bad[:4].tolist()} of {len(bad)}"


def draw_new(g, B, H, N, dtype):
    x = g.standard_normal((2, B, H, N, 64)) * np.exp2(g.integers(-6, 6, (2, B, H, N, 1)))
    return fin(x[0], dtype), fin(x[1], dtype)


APPEND = [  # B, H, N, Lmax, block, dtype, code, cache_len, new_len
    (3, 2, 1, 100, 16, "bf16", "e4m3", [0, 15, 99], None),
    (3, 2, 1, 100, 64, "f32", "int8", [16, 64, 100], None),        # the last cache is full
    (2, 3, 77, 200, 32, "bf16", "int8", [5, 150], None),           # the second runs past Lmax
    (4, 1, 50, 90, 128, "bf16", "e4m3", [0, 3, 40, 90], [50, 0, 1, 9]),
    (2, 2, 130, 131, 64, "f32", "e4m3", [0, 1], [130, 999]),       # new_len clamps to N
    (2, 1, 33, 40, 16, "f32", "int8", [-3, 1000], None),           # cache_len clamps
    (1, 1, 1, 1, 16, "bf16", "e4m3", [0], None),
]


@pytest.mark.parametrize("B,H,N,Lmax,block,dtype,code,cl,nl", APPEND)
@pytest.mark.parametrize("token_major", [False, True])
def test_append(B, H, N, Lmax, block, dtype, code, cl, nl, token_major):
    g = rng(500 + N + Lmax)
    c = strange(g, B, H, Lmax, block, code)
    k, v = draw_new(g, B, H, N, dtype)
    cache = to_gpu(c, block, code, token_major)
    tk, tv = dev(k, DT[dtype]), dev(v, DT[dtype])
    if token_major:
        tk, tv = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (tk, tv))
    mha.kv_append_q8(cache, tk, tv, i32(cl), i32(nl))
    # an old block's scale that an append may leave (NaN codes stay NaN under any scale)
    want = oq.append_ref(c, k, v, cl, nl, block, code)
    assert_same(from_gpu(cache), want, code, "append")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_extreme_values(code, dtype):
    x = np.zeros((1, 4, 9, 64))
    x[0, 0, 0, :6] = [np.inf, -np.inf, np.nan, 3.0, -0.0, 1e-30]   # beside finite values
    x[0, 1] = 1e30                                                  # past the largest scale
    x[0, 1, 1] = -1e30
    x[0, 2] = 1e-35                                                 # below the smallest
    x[0, 2, 3, 3] = 1e-12
    x[0, 3, :, 0] = np.inf                                          # no finite value but zeros
    x = fin(x, dtype)
    c = finite(strange(rng(540), 1, 4, 20, 16, code), code)
    cache = to_gpu(c, 16, code)
    mha.kv_append_q8(cache, dev(x, DT[dtype]), dev(-x, DT[dtype]), i32([4]))
    assert_same(from_gpu(cache), oq.append_ref(c, x, -x, [4], None, 16, code), code, "extremes")


def test_append_without_weights_and_token_by_token():
    g = rng(545)
    cache = mha.kv_cache_q8(1, 2, 70, block=32, weights=False)
    want = {"k": np.zeros((1, 2, 70, 64), np.uint8), "v": np.zeros((1, 2, 70, 64), np.uint8),
            "k_scale": np.ones((1, 2, 3)), "v_scale": np.ones((1, 2, 3)),
            "weights": np.zeros((1, 2, 70))}
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(70):
        k, v = draw_new(g, 1, 2, 1, "bf16")
        mha.kv_append_q8(cache, dev(k, torch.bfloat16), dev(v, torch.bfloat16), n)
        n += 1
        want = oq.append_ref(want, k, v, [t], None, 32, "e4m3")
    got = from_gpu(cache._replace(weights=torch.zeros(1, 2, 70, device="cuda")))
    assert_same(got, want, "e4m3", "token by token")


def close_decode(got, ref, pv, low, qk, n, dtype, what):
    r = 2.0 ** -17 * qk + n * 2.0 ** -24 + 2.0 ** -19 + (2.0 ** -11 if dtype == "bf16" else 0)
    bound = r * pv + 2.0 ** -38 * low + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + 1e-30
    assert np.all(np.isfinite(got)), what
    worst = (np.abs(got - ref) / bound).max()
    assert worst <= 1, f"{what}: {worst:.3f} of the bound"


def close_weights(got, before, ref, qk, n, what):
    r = 2.0 ** -17 * qk + n * 2.0 ** -24 + 2.0 ** -19
    bound = r * ref + 2.0 ** -24 * np.abs(before + ref)
    bad = np.abs(got - before - ref) > bound
    assert not bad.any(), f"{what}: {np.argwhere(bad)[:3].tolist()}"


DECODE = [  # B, H, Hkv, Nq, Lmax, block, dtype, code, causal, cache_len
    (1, 1, 1, 1, 1, 16, "bf16", "e4m3", True, [1]),
    (3, 2, 2, 1, 700, 64, "bf16", "int8", True, [700, 300, 129]),
    (3, 4, 2, 4, 700, 16, "bf16", "e4m3", True, [700, 63, 64]),
    (2, 16, 2, 16, 333, 32, "bf16", "e4m3", True, [333, 17]),          # 128 rows to a head
    (2, 3, 1, 16, 130, 128, "f32", "int8", False, [130, 65]),          # 48 rows
    (4, 6, 3, 1, 1000, 128, "f32", "e4m3", False, [1000, 0, 1, 517]),
    (3, 2, 1, 8, 300, 64, "bf16", "e4m3", True, [3, 0, 256]),          # rows without keys
    (2, 2, 2, 2, 513, 64, "f32", "e4m3", True, [2, 999]),              # clamps to Lmax
    (2, 5, 5, 7, 197, 16, "bf16", "int8", False, [-4, 190]),
    (1, 8, 1, 3, 5000, 64, "bf16", "int8", True, [4999]),              # one long head
    (70, 3, 3, 1, 40, 16, "f32", "int8", True, [i % 41 for i in range(70)]),
    (1, 64, 4, 16, 300, 16, "f32", "e4m3", True, [300]),               # 256 rows
    (1, 256, 1, 16, 40, 16, "bf16", "int8", False, [40]),              # 4096 rows, the most
    (8, 40, 40, 1, 4100, 64, "bf16", "e4m3", True, [4100, 0, 4096, 4097, 1, 33, 2048, 777]),
    (2, 320, 80, 1, 2100, 32, "f32", "int8", True, [2100, 1025]),
    (1, 16, 8, 8, 768, 64, "bf16", "e4m3", True, [766]),               # one launch
    (4, 4, 4, 16, 383, 16, "f32", "e4m3", False, [383, 0, 33, 2]),
    (150, 1, 1, 1, 100, 32, "bf16", "int8", True, [i % 103 for i in range(150)]),
    (300, 1, 1, 1, 100, 32, "bf16", "int8", True, [i % 103 for i in range(300)]),
]


@pytest.mark.parametrize("B,H,Hkv,Nq,Lmax,block,dtype,code,causal,cl", DECODE)
@pytest.mark.parametrize("add", [False, True])
def test_decode(B, H, Hkv, Nq, Lmax, block, dtype, code, causal, cl, add):
    g = rng(600 + Nq + Lmax)
    c = strange(g, B, Hkv, Lmax, block, code)   # bytes behind cache_len: anything, NaN codes too
    clean = finite({n: np.array(a) for n, a in c.items()}, code)
    for b in range(B):
        L = int(np.clip(cl[b], 0, Lmax))
        for n in "kv":
            c[n][b, :, :L] = clean[n][b, :, :L]
            nb = -(-L // block)                 # and scales behind it too
            c[n + "_scale"][b, :, nb:] = np.nan
    # scales at which scores stay moderate: e4m3 bytes reach 448, integers 127
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    Q = fin(g.standard_normal((B, H, Nq, 64)), dtype)
    cache = to_gpu(c, block, code)
    before = c["weights"].copy()
    O = mha.sdpa_decode_q8(dev(Q, DT[dtype]), cache, i32(cl), causal=causal, add_weights=add)
    ref, W, pv, low, qk = oq.decode_ref(Q, c, cl, block, code, causal)
    n = int(np.clip(max(cl), 0, Lmax))
    got = O.double().cpu().numpy()
    close_decode(got, ref, pv, low, qk, n, dtype, "decode")
    assert np.all(got[pv == 0] == 0)            # rows without keys (or with values all zero)
    w = cache.weights.double().cpu().numpy()
    if add:
        close_weights(w, before, W, qk, n, "decode weights")
        for b in range(B):                      # behind the last position: as they were
            L = int(np.clip(cl[b], 0, Lmax))
            assert np.array_equal(w[b, :, L:], before[b, :, L:])
    else:
        assert np.array_equal(w, before)
    # the same call again gives the same bits
    O2 = mha.sdpa_decode_q8(dev(Q, DT[dtype]), cache, i32(cl), causal=causal)
    assert torch.equal(O, O2)


def test_decode_token_major_scale_and_workspace():
    B, H, Hkv, Nq, Lmax, block = 2, 4, 2, 2, 600, 64
    g = rng(640)
    c = finite(strange(g, B, Hkv, Lmax, block, "int8"), "int8")
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    Q = fin(g.standard_normal((B, H, Nq, 64)), "bf16")
    cache = to_gpu(c, block, "int8", token_major=True)
    tq = dev(Q, torch.bfloat16).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    out = torch.zeros(B, Nq, H, 64, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    ws = torch.empty(mha.decode_q8_workspace_size(B, H, Hkv, Nq, Lmax, False), dtype=torch.uint8,
                     device="cuda")
    mha.sdpa_decode_q8(tq, cache, i32([600, 333]), scale=0.05, workspace=ws, out=out)
    ref, _, pv, low, qk = oq.decode_ref(Q, c, [600, 333], block, "int8", True, scale=0.05)
    close_decode(out.double().cpu().numpy(), ref, pv, low, qk, 600, "bf16", "token-major")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_scales_far_apart_and_not_powers_of_two(dtype):
    # a block whose values are 2^30 smaller than its neighbour's still counts where it is attended
    g = rng(650)
    c = finite(strange(g, 1, 1, 64, 16, "e4m3"), "e4m3")
    c["k_scale"][0, 0] = [0.011, 0.007, 0.02, 0.013]
    c["v_scale"][0, 0] = [2.0 ** 20, 3e-10, 1.0, 0.3]
    for n in "kv":
        c[n + "_scale"] = c[n + "_scale"].astype(np.float32).astype(np.float64)
    Q = np.zeros((1, 2, 1, 64))
    kk = oq.dequantised_ref(c, "k", 0, 0, 64, 16, "e4m3")
    Q[0, 0, 0] = kk[20] * 40 / (kk[20] @ kk[20]) * 8   # the key at 20, in the small block
    Q[0, 1, 0] = g.standard_normal(64)
    Q = fin(Q, dtype)
    O = mha.sdpa_decode_q8(dev(Q, DT[dtype]), to_gpu(c, 16, "e4m3"), i32([64]))
    ref, _, pv, low, qk = oq.decode_ref(Q, c, [64], 16, "e4m3", True)
    close_decode(O.double().cpu().numpy(), ref, pv, low, qk, 64, dtype, "scales far apart")


def test_decode_large_and_small_queries():
    # rows at the ends of bf16's range beside ordinary ones; zero rows attend evenly
    g = rng(655)
    c = finite(strange(g, 1, 1, 100, 32, "int8"), "int8")
    Q = np.zeros((1, 5, 1, 64))
    Q[0, 0, 0] = g.standard_normal(64) * 1e30
    Q[0, 1, 0] = g.standard_normal(64) * 1e-30
    Q[0, 2, 0] = g.standard_normal(64)
    Q[0, 4, 0, 5] = 1e4
    c["k_scale"][...] = 2.0 ** -10
    Q = fin(Q, "bf16")
    O = mha.sdpa_decode_q8(dev(Q, torch.bfloat16), to_gpu(c, 32, "int8"), i32([100]))
    got = O.double().cpu().numpy()
    for h in (1, 2, 3, 4):
        ref, _, pv, low, qk = oq.decode_ref(Q[:, h:h + 1], c, [100], 32, "int8", True)
        close_decode(got[:, h:h + 1], ref, pv, low, qk, 100, "bf16", f"row {h}")
    # scores of 1e30: one key has all the weight
    kk = oq.dequantised_ref(c, "k", 0, 0, 100, 32, "int8")
    vv = oq.dequantised_ref(c, "v", 0, 0, 100, 32, "int8")
    top = vv[np.argmax(kk @ Q[0, 0, 0].astype(np.float64))]
    assert np.all(np.abs(got[0, 0, 0] - top) <= 2.0 ** -8 * np.abs(top))


def test_decode_nan_reaches_only_the_rows_that_see_it():
    # four new positions; the third one's value row and a query row hold NaN
    g = rng(660)
    B, H, Nq, L = 1, 2, 4, 90
    c = finite(strange(g, B, 1, 100, 16, "e4m3"), "e4m3")
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    c["v"][0, 0, L - 2, 7] = 127
    Q = fin(g.standard_normal((B, H, Nq, 64)), "bf16")
    Q[0, 1, 0] = np.nan
    O = mha.sdpa_decode_q8(dev(Q, torch.bfloat16), to_gpu(c, 16, "e4m3"), i32([L])).float().cpu()
    nan = torch.isnan(O[0])
    want = torch.zeros(H, Nq, 64, dtype=torch.bool)
    want[:, 2:, 7] = True      # queries at and behind the position see its value
    want[1, 0] = True          # the row whose query is NaN
    assert torch.equal(nan, want)
    # a key of NaN: every later query's row, no earlier one
    c["v"][0, 0, L - 2, 7] = 0
    c["k"][0, 0, L - 2, 9] = 255
    Q[0, 1, 0] = 0
    O = mha.sdpa_decode_q8(dev(Q, torch.bfloat16), to_gpu(c, 16, "e4m3"), i32([L])).float().cpu()
    assert torch.isnan(O[0, :, 2:]).all() and not torch.isnan(O[0, :, :2]).any()


KEYW = [  # B, H, Hkv, Nq, Nk, dtype, mask, key_len, query_len
    (1, 1, 1, 1, 1, "bf16", "none", None, None),
    (2, 2, 2, 128, 128, "bf16", "causal", None, None),
    (2, 3, 3, 200, 200, "bf16", "causal", None, [200, 77]),
    (2, 4, 2, 77, 300, "bf16", "key_padding", [300, 13], None),
    (3, 4, 1, 130, 257, "bf16", "key_padding", [0, 257, 128], [130, 5, 0]),
    (1, 8, 2, 513, 640, "bf16", "none", None, [400]),
    (2, 2, 1, 50, 50, "f32", "causal", None, [50, 33]),
    (2, 2, 2, 65, 33, "f32", "key_padding", [33, 31], None),
    (1, 3, 3, 300, 40, "f32", "none", None, None),
    (2, 1, 1, 1, 500, "bf16", "none", None, None),
    (1, 4, 2, 1500, 1500, "bf16", "causal", None, [1400]),             # queries split over CTAs
    (160, 2, 2, 130, 130, "bf16", "causal", None, None),               # not split
    (1, 4, 2, 700, 700, "f32", "causal", None, [650]),
    (2, 4, 1, 300, 500, "f32", "key_padding", [500, 0], [300, 20]),
    (320, 2, 1, 20, 150, "f32", "none", None, None),
]


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,dtype,mask,kl,ql", KEYW)
@pytest.mark.parametrize("spare", [0, 37])
def test_key_weights(B, H, Hkv, Nq, Nk, dtype, mask, kl, ql, spare):
    g = rng(700 + Nq + Nk)
    Q, K = fin(g.standard_normal((B, H, Nq, 64)), dtype), fin(g.standard_normal((B, Hkv, Nk, 64)),
                                                             dtype)
    Kx = np.repeat(K, H // Hkv, 1)
    lse = oracle.sdpa_lse_ref(Q, Kx, mask, None if kl is None else np.array(kl, np.int32))
    lse = lse.astype(np.float32)
    tq, tk = dev(Q, DT[dtype]), dev(K, DT[dtype])
    tl = dev(lse)
    if ql is not None:  # rows behind the last query may hold anything
        for b in range(B):
            tq[b, :, ql[b]:] = float("nan")
            tl[b, :, ql[b]:] = float("nan")
    if kl is not None:
        for b in range(B):
            tk[b, :, kl[b]:] = float("nan")
    before = g.random((B, Hkv, Nk + spare)).astype(np.float32)
    w = dev(before)
    got = mha.sdpa_key_weights(tq, tk, tl, mask, i32(kl), i32(ql), weights=w)
    assert got is w
    ref = np.zeros((B, Hkv, Nk + spare))
    ref[..., :Nk] = oq.key_weights_ref(Q, K, lse, mask, kl, ql)
    S = np.abs(Q).astype(np.float64) @ np.abs(Kx).astype(np.float64).transpose(0, 1, 3, 2) / 8
    big = np.abs(lse[np.isfinite(lse)]).max(initial=0.0)
    # one exponential (not a ratio); lse * log2 e is rounded once: 2^-24 |lse|
    r = 2.0 ** -18 * S.max() + 2.0 ** -23 * big + 2.0 ** -20 + (H // Hkv) * Nq * 2.0 ** -24
    err = np.abs(w.double().cpu().numpy() - before - ref)
    bound = r * ref + 2.0 ** -24 * np.abs(before + ref)
    assert np.all(err <= bound), f"{(err / np.maximum(bound, 1e-30)).max():.3f} of the bound"
    assert np.array_equal(w.cpu().numpy()[ref == 0], before[ref == 0])
    again = mha.sdpa_key_weights(tq, tk, tl, mask, i32(kl), i32(ql), weights=dev(before))
    assert torch.equal(again, w)


def test_key_weights_token_major_and_fresh():
    g = rng(750)
    B, H, N = 2, 4, 150
    Q, K = (fin(g.standard_normal((B, N, H, 64)), "bf16") for _ in range(2))
    tq, tk = (dev(x, torch.bfloat16).permute(0, 2, 1, 3) for x in (Q, K))
    _, lse = mha.sdpa_with_lse(tq, tk, tk, "causal", scale=0.2)
    w = mha.sdpa_key_weights(tq, tk, lse, "causal", scale=0.2)
    ref = oq.key_weights_ref(np.moveaxis(Q, 1, 2), np.moveaxis(K, 1, 2), lse.cpu().numpy(),
                             "causal", scale=0.2)
    assert np.allclose(w.cpu().numpy(), ref, rtol=1e-3)
    assert np.allclose(w.sum(-1).cpu().numpy(), N, rtol=1e-3)  # every row's weights sum to 1


EVICT = [  # B, H, Lmax, Lout, keep, recent, block, code, cache_len
    (2, 2, 100, 64, 50, 7, 16, "e4m3", [100, 60]),
    (3, 1, 300, 200, 129, 0, 64, "int8", [300, 129, 130]),
    (3, 2, 90, 90, 40, 40, 32, "e4m3", [90, 41, 0]),
    (2, 1, 50, 7, 1, 0, 16, "int8", [50, 1]),
    (2, 1, 50, 7, 1, 5, 128, "e4m3", [50, -3]),
    (1, 2, 5000, 1300, 1025, 100, 128, "e4m3", [9999]),
    (1, 1, 2049, 2049, 2048, 1000, 16, "int8", [2049]),
    (1, 2, 9000, 5000, 4999, 64, 64, "e4m3", [9000]),                  # one CTA of 1024 threads,
    (2, 1, 20001, 9000, 9000, 0, 64, "int8", [20001, 16385]),          # two, four and eight,
    (1, 1, 60000, 300, 257, 100, 32, "e4m3", [55555]),
    (1, 1, 131072, 4096, 4096, 7, 128, "int8", [131072]),
    (2, 1, 140000, 600, 600, 11, 64, "e4m3", [140000, 131073]),        # more than they hold
]


@pytest.mark.parametrize("B,H,Lmax,Lout,keep,recent,block,code,cl", EVICT)
@pytest.mark.parametrize("kind", ["random", "ties", "signs"])
@pytest.mark.parametrize("token_major", [False, True])
def test_evict(B, H, Lmax, Lout, keep, recent, block, code, cl, kind, token_major):
    g = rng(800 + Lmax + keep)
    c = finite(strange(g, B, H, Lmax, block, code), code)
    if kind == "ties":          # a handful of different weights, zeros of both signs among them
        c["weights"] = np.array([0.0, -0.0, 1.0, 1.0 + 2.0 ** -23, 2.0 ** -140])[
            g.integers(0, 5, (B, H, Lmax))]
    elif kind == "signs":       # negative ones, infinities and NaN
        w = g.standard_normal((B, H, Lmax)).astype(np.float32).astype(np.float64)
        r = g.random((B, H, Lmax))
        w[r < 0.05], w[(r > 0.05) & (r < 0.3)], w[r > 0.95] = np.inf, -np.inf, np.nan
        c["weights"] = w
    d = strange(g, B, H, Lout, block, code)
    src, out = to_gpu(c, block, code, token_major), to_gpu(d, block, code, token_major)
    n, kept = mha.kv_evict_q8(src, out, i32(cl), keep, recent)
    want, wn, wkept = oq.evict_ref(c, d, cl, keep, recent, block, code)
    assert np.array_equal(n.cpu().numpy(), wn)
    assert np.array_equal(kept.cpu().numpy(), wkept)
    got = from_gpu(out)
    if kind == "signs":         # NaN weights of recent positions move along
        assert np.array_equal(np.isnan(got["weights"]), np.isnan(want["weights"]))
        got["weights"] = np.nan_to_num(got["weights"], nan=7.0)
        want["weights"] = np.nan_to_num(want["weights"], nan=7.0)
    assert_same(got, want, code, "evict")
    clean = from_gpu(src)
    c["weights"], clean["weights"] = (np.nan_to_num(x, nan=7.0) for x in (c["weights"],
                                                                         clean["weights"]))
    assert_same(clean, c, code, "the old cache")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_prompt_then_steps_then_eviction(code):
    """A padded batch of prompts is attended and cached, its weights summed, the caches cut and
    generation goes on from what was kept: every stage against the oracle's."""
    g = rng(900)
    B, Hkv, G, N, Lmax, keep, block = 2, 2, 2, 140, 192, 64, 32
    lens = [140, 90]
    q = fin(g.standard_normal((B, Hkv * G, N, 64)), "bf16")
    k, v = (fin(g.standard_normal((B, Hkv, N, 64)), "bf16") for _ in range(2))
    tq, tk, tv = (dev(x, torch.bfloat16) for x in (q, k, v))
    kx = tk.repeat_interleave(G, 1)
    _, lse = mha.sdpa_with_lse(tq, kx, tv.repeat_interleave(G, 1), "causal")
    cache = mha.kv_cache_q8(B, Hkv, Lmax, block, CODE[code])
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    mha.kv_append_q8(cache, tk, tv, n, i32(lens))
    n += i32(lens)
    mha.sdpa_key_weights(tq, tk, lse, "causal", None, i32(lens), weights=cache.weights)
    c = oq.append_ref({"k": np.zeros((B, Hkv, Lmax, 64), np.uint8),
                       "v": np.zeros((B, Hkv, Lmax, 64), np.uint8),
                       "k_scale": np.ones((B, Hkv, 6)), "v_scale": np.ones((B, Hkv, 6)),
                       "weights": np.zeros((B, Hkv, Lmax))}, k, v, [0, 0], lens, block, code)
    W = oq.key_weights_ref(q, k, lse.cpu().numpy(), "causal", None, lens)
    got = from_gpu(cache)
    assert np.allclose(got["weights"][..., :N], W, rtol=1e-3, atol=1e-6)
    c["weights"] = got["weights"]           # near-equal weights may rank either way: go on from
    assert_same(got, c, code, "prompt")     # the ones that were measured
    small = mha.kv_cache_q8(B, Hkv, keep + 16, block, CODE[code])
    n, kept = mha.kv_evict_q8(cache, small, n, keep, 16)
    blank = from_gpu(mha.kv_cache_q8(B, Hkv, keep + 16, block, CODE[code]))
    c, wn, wkept = oq.evict_ref(c, blank, lens, keep, 16, block, code)
    assert np.array_equal(kept.cpu().numpy(), wkept)
    assert_same(from_gpu(small), c, code, "evicted")
    for step in range(3):
        k, v = (fin(g.standard_normal((B, Hkv, 2, 64)), "bf16") for _ in range(2))
        q = fin(g.standard_normal((B, Hkv * G, 2, 64)), "bf16")
        mha.kv_append_q8(small, dev(k, torch.bfloat16), dev(v, torch.bfloat16), n)
        c = oq.append_ref(c, k, v, n.tolist(), None, block, code)
        n += 2
        O = mha.sdpa_decode_q8(dev(q, torch.bfloat16), small, n, add_weights=True)
        ref, W, pv, low, qk = oq.decode_ref(q, c, n.tolist(), block, code, True)
        close_decode(O.double().cpu().numpy(), ref, pv, low, qk, keep + 8, "bf16", f"step {step}")
        got = from_gpu(small)
        close_weights(got["weights"], c["weights"], W, qk, keep + 8, f"weights {step}")
        c["weights"] = got["weights"]
        assert_same(got, c, code, f"cache {step}")


def test_captured_steps_replay_with_new_lengths():
    """Append, attention with weights and eviction in a CUDA graph on another stream, replayed as
    the cache grows, give what the same calls give outside."""
    g = rng(950)
    B, H, Lmax = 2, 2, 300

    def fresh():
        r = rng(951)
        c = finite(strange(r, B, H, Lmax, 64, "int8"), "int8")
        for n in "kv":
            c[n + "_scale"] *= 2.0 ** -6
        return to_gpu(c, 64, "int8"), mha.kv_cache_q8(B, H, 128, 64, torch.int8)

    steps = [[fin(g.standard_normal((B, H, 1, 64)), "bf16") for _ in range(3)] for _ in range(4)]
    steps = [[dev(x, torch.bfloat16) for x in s] for s in steps]

    def step(cache, small, q, k, v, n, out, n_out, kept, ws):
        mha.kv_append_q8(cache, k, v, n)
        n.add_(1)
        mha.sdpa_decode_q8(q, cache, n, add_weights=True, out=out, workspace=ws)
        mha.kv_evict_q8(cache, small, n, 100, 10, len_out=n_out, kept=kept)

    def buffers():
        return (i32([290, 60]), torch.zeros(B, H, 1, 64, dtype=torch.bfloat16, device="cuda"),
                i32([0, 0]), torch.zeros(B, H, 100, dtype=torch.int32, device="cuda"),
                torch.empty(mha.decode_q8_workspace_size(B, H, H, 1, Lmax, True),
                            dtype=torch.uint8, device="cuda"))

    want = []
    cache, small = fresh()
    buf = buffers()
    for s in steps:
        step(cache, small, *s, *buf)
        want.append((buf[1].clone(), buf[3].clone()))
    final = from_gpu(cache), from_gpu(small)

    cache2, small2 = fresh()
    buf2 = buffers()
    q, k, v = (torch.empty_like(x) for x in steps[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache2, small2, q, k, v, *buf2)
    for s, (o, kept) in zip(steps, want):
        for a, x in zip((q, k, v), s):
            a.copy_(x)
        graph.replay()
        assert torch.equal(buf2[1], o) and torch.equal(buf2[3], kept)
    for a, b in zip(final, (from_gpu(cache2), from_gpu(small2))):
        assert_same(b, a, "int8", "replayed")


def test_two_streams_with_their_own_workspaces():
    g = rng(970)
    c = finite(strange(g, 4, 2, 900, 64, "e4m3"), "e4m3")
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    cache, n = to_gpu(c, 64, "e4m3"), i32([900, 1, 450, 899])
    qs = [dev(fin(g.standard_normal((4, 4, 3, 64)), "bf16"), torch.bfloat16) for _ in range(2)]
    alone = [mha.sdpa_decode_q8(q, cache, n) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(20):
        outs = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                outs.append(mha.sdpa_decode_q8(q, cache, n))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [5, 300])
def test_key_weights_rows_of_infinite_lse(dtype, Nq):
    g = rng(760)
    q, k = fin(g.standard_normal((1, 2, Nq, 64)), dtype), fin(g.standard_normal((1, 2, 70, 64)),
                                                             dtype)
    lse = oracle.sdpa_lse_ref(q, k, "none").astype(np.float32)
    lse[0, :, 1::2] = np.inf
    w = mha.sdpa_key_weights(dev(q, DT[dtype]), dev(k, DT[dtype]), dev(lse))
    keep = np.ascontiguousarray(q[:, :, ::2]), np.ascontiguousarray(lse[:, :, ::2])
    ref = oq.key_weights_ref(keep[0], k, keep[1], "none")
    assert np.allclose(w.cpu().numpy(), ref, rtol=1e-4)


def odd(t):
    """A copy whose first element is 4 bytes off any larger boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.flatten()
    return flat[1:].view(t.shape)


def test_small_alignments_and_odd_sizes_give_the_same_bits():
    # weights, scales, lse and lengths need 4 bytes only
    g = rng(980)
    B, H, Lmax, block = 2, 2, 5001, 16
    c = finite(strange(g, B, H, Lmax, block, "e4m3"), "e4m3")
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    d = strange(g, B, H, 1001, block, "e4m3")
    q, k, v = (dev(fin(g.standard_normal((B, h, 3, 64)), "bf16"), torch.bfloat16)
               for h in (4, 2, 2))
    prompt = [dev(fin(g.standard_normal((B, h, 333, 64)), "bf16"), torch.bfloat16) for h in (4, 2)]
    results = []
    for shift in (lambda t: t, odd):
        cache, out = to_gpu(c, block, "e4m3"), to_gpu(d, block, "e4m3")
        cache, out = (x._replace(k_scale=shift(x.k_scale), v_scale=shift(x.v_scale),
                                 weights=shift(x.weights)) for x in (cache, out))
        n = shift(i32([4998, 77]))
        mha.kv_append_q8(cache, k, v, n, shift(i32([3, 2])))
        n = shift(i32([5001, 79]))
        O = mha.sdpa_decode_q8(q, cache, n, add_weights=True)
        for x in (prompt, [t.float() for t in prompt]):
            lse = shift(torch.full((B, 4, 333), 2.0, device="cuda"))
            mha.sdpa_key_weights(*x, lse, "causal", None, shift(i32([333, 70])),
                                 weights=cache.weights)
        m, kept = mha.kv_evict_q8(cache, out, n, 1000, 17, len_out=shift(i32([0, 0])),
                                  kept=shift(torch.zeros(B, H, 1000, dtype=torch.int32,
                                                         device="cuda")))
        results.append((O, m, kept, from_gpu(cache), from_gpu(out)))
    a, b = results
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    assert_same(a[3], b[3], "e4m3", "cache")
    assert_same(a[4], b[4], "e4m3", "evicted")


def test_offsets_beyond_32_bits():
    """Two heads of 40 million positions: 2.56e9 bytes each in K and in V.  All keys are zero but
    three at the end, which hold all the weight (e^64 over e^0 for every other)."""
    L, dt = 40_000_000, torch.bfloat16
    cache = mha.kv_cache_q8(1, 2, L, 64)
    k = torch.empty(1, 2, 3, 64, dtype=dt, device="cuda")
    k[:, :, 0], k[:, :, 1], k[:, :, 2] = 8, -8, 8
    v = dev(rng(990).integers(-8, 9, (1, 2, 3, 64)).astype(np.float32), dt)
    mha.kv_append_q8(cache, k, v, i32([L - 3]))
    for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        assert torch.equal(codes[:, :, -3:].float() * scale[:, :, -1:, None], x.float())
        assert not codes[:, :, -6:-3].view(torch.uint8).any()
    O = mha.sdpa_decode_q8(torch.ones(1, 4, 1, 64, dtype=dt, device="cuda"), cache, i32([L]),
                           add_weights=True)
    want = ((v[:, :, 0] + v[:, :, 2]).float() / 2).repeat_interleave(2, 1)[:, :, None]
    # the weights are rounded to 2^-11, the output to 2^-8 (values of both signs: of the larger)
    assert torch.all((O.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * 8)
    w = cache.weights
    assert torch.all((w[:, :, [-3, -1]] - 1).abs() < 1e-4)      # a half from each of two queries
    assert w[:, :, :-3].max() < 1e-20 and w[:, :, -2].max() < 1e-20
    w[0, 0, 12_345_678] = w[0, 1, 39_000_001] = 0.25
    out = mha.kv_cache_q8(1, 2, 3, 64)
    n, kept = mha.kv_evict_q8(cache, out, i32([L]), 3, 1)
    assert n.tolist() == [3]
    assert kept.tolist() == [[[12_345_678, L - 3, L - 1], [39_000_001, L - 3, L - 1]]]
    got = out.v.float() * out.v_scale[..., None]
    assert torch.equal(got[:, :, 1:], v[:, :, [0, 2]].float()) and not got[:, :, 0].any()


def test_wrappers_refuse():
    cache, out = mha.kv_cache_q8(1, 2, 64, 16), mha.kv_cache_q8(1, 2, 32, 16)
    n, q = i32([10]), torch.zeros(1, 2, 1, 64, device="cuda")
    for keep, recent in ((0, 0), (33, 0), (-1, 0), (2 ** 32 + 4, 0), (8, -1)):
        with pytest.raises(ValueError):
            mha.kv_evict_q8(cache, out, n, keep, recent)
    mha.kv_evict_q8(cache, out, n, 8, 2 ** 40)          # every kept position a recent one
    for call in (lambda: mha.kv_evict_q8(cache, mha.kv_cache_q8(1, 2, 32, 32), n, 8),
                 lambda: mha.kv_evict_q8(cache._replace(weights=None), out, n, 8),
                 lambda: mha.kv_evict_q8(cache, out, n.long(), 8),
                 lambda: mha.sdpa_decode_q8(q[:, :1].expand(1, 3, 1, 64), cache, n),
                 lambda: mha.sdpa_decode_q8(q, cache._replace(weights=None), n, add_weights=True),
                 lambda: mha.sdpa_decode_q8(q, cache, n, out=q.bfloat16()),
                 lambda: mha.kv_append_q8(cache, q, q[:, :1], n),
                 lambda: mha.kv_append_q8(cache, q, q.cpu(), n),
                 lambda: mha.sdpa_key_weights(q, q, q[..., 0].double())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mha.MhaError):                   # too small a workspace
        mha.sdpa_decode_q8(torch.zeros(1, 2, 1, 64, device="cuda"), mha.kv_cache_q8(1, 2, 4096), n,
                           workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mha.MhaError):                   # a broadcast tensor has strides of 0
        mha.kv_append_q8(cache, q[:, :1].expand(1, 2, 1, 64), q, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_of_one_projection(dtype):
    """q, k and v as views of one [B, N, 3, H, 64] buffer give what copies of them give."""
    g = rng(1000)
    B, N, H = 2, 150, 3
    x = dev(fin(g.standard_normal((B, N, 3, H, 64)), dtype), DT[dtype])
    views = [x[:, :, i].transpose(1, 2) for i in range(3)]
    results = []
    for q, k, v in (views, [t.contiguous() for t in views]):
        cache = mha.kv_cache_q8(B, H, 200, 32)
        n = i32([0, 3])
        mha.kv_append_q8(cache, k, v, n, i32([150, 99]))
        _, lse = mha.sdpa_with_lse(q, k, v, "causal")
        mha.sdpa_key_weights(q, k, lse, "causal", None, i32([150, 99]), weights=cache.weights)
        O = mha.sdpa_decode_q8(q[:, :, 5:9], cache, i32([150, 102]), add_weights=True)
        results.append((O, lse, from_gpu(cache)))
    a, b = results
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert_same(a[2], b[2], "e4m3", "views")


@pytest.mark.parametrize("dtype,N", [("bf16", 130), ("bf16", 700), ("f32", 40), ("f32", 333)])
def test_captured_prompts_replay(dtype, N):
    """A prompt's append, attention weights and eviction in a graph, replayed with new prompts and
    lengths, give what the same calls give outside (queries split over CTAs and not)."""
    g = rng(1010)
    B, H, G = 2, 2, 2
    prompts = [[dev(fin(g.standard_normal((B, h, N, 64)), dtype), DT[dtype])
                for h in (H * G, H, H)] + [i32(n)] for n in ([N, N // 2], [1, N], [0, N - 1])]

    def run(cache, small, q, k, v, lens, lse, zero, n_out, kept):
        cache.weights.zero_()
        mha.kv_append_q8(cache, k, v, zero, lens)
        mha.sdpa_key_weights(q, k, lse, "causal", None, lens, weights=cache.weights)
        mha.kv_evict_q8(cache, small, lens, 30, 3, len_out=n_out, kept=kept)

    def buffers():
        return (mha.kv_cache_q8(B, H, N + 5, 16, weights=True), mha.kv_cache_q8(B, H, 30, 16),
                i32([0, 0]), i32([0, 0]), torch.zeros(B, H, 30, dtype=torch.int32, device="cuda"))

    def lse_of(q, k, v):
        return mha.sdpa_with_lse(q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1),
                                 "causal")[1]

    cache, small, zero, n_out, kept = buffers()
    want = []
    for q, k, v, lens in prompts:
        run(cache, small, q, k, v, lens, lse_of(q, k, v), zero, n_out, kept)
        want.append((n_out.clone(), kept.clone(), from_gpu(cache), from_gpu(small)))
    cache, small, zero, n_out, kept = buffers()
    q, k, v, lens = (t.clone() for t in prompts[0])
    lse = lse_of(q, k, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(cache, small, q, k, v, lens, lse, zero, n_out, kept)
    for p, (wn, wkept, wcache, wsmall) in zip(prompts, want):
        for a, x in zip((q, k, v, lens, lse), p + [lse_of(*p[:3])]):
            a.copy_(x)
        graph.replay()
        assert torch.equal(n_out, wn) and torch.equal(kept, wkept)
        assert_same(from_gpu(cache), wcache, "e4m3", "cache")
        assert_same(from_gpu(small), wsmall, "e4m3", "evicted")
