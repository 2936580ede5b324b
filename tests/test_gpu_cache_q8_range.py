"""The 8-bit cache at the ends of what its entry points take: huge scores, value scales far apart,
rows far below or above 1, scales that are no powers of two, many heads, and the special rows on
every launch path of the generation step.

A generation step has three paths: one launch (up to 768 positions, 152 cache heads, 16 rows to a
head), and two whose second joins a row's pieces, with a block to a row where rows are few and
pieces many, else with a warp to a row.  ``PATHS`` has sizes for each.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import cache_q8 as oq
from test_gpu_cache_q8 import (CODE, DT, assert_same, close_decode, close_weights, dev, fin, finite,
                               from_gpu, i32, rng, strange, to_gpu)

pytestmark = pytest.mark.gpu

mha = pytest.importorskip("transformer_head_scaled_04_gb300")

PATHS = {"one launch": (1, 2, 100), "block join": (1, 1, 5000), "warp join": (40, 4, 790)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_head_scaled_04_gb300 import build

    build.build()
    mha.load_library()
    torch.cuda.set_device(0)
    mha.device_status()
    yield
    assert mha.device_status() == 0, "a kernel recorded a device-side error"


def check_path(path, B, Hkv, rows, Lmax):
    need = mha.decode_q8_workspace_size(B, Hkv * rows, Hkv, 1, Lmax, True)
    assert (need == 0) == (path == "one launch")


def one_key_cache(g, B, H, Lmax, block, code, sign, flip):
    """Key codes that lie along `sign` [64].  With a query sign * a, position j0 of every head has a
    score of 104 * 64 a (flip: -56 * 64 a) and every other one at most 80 (-96) * 64 a."""
    c = finite(strange(g, B, H, Lmax, block, code), code)
    along = np.array([oq.encode_ref(x * sign, code) for x in range(-104, 104, 8)])
    pick = g.integers(0, 2 if flip else 24, (B, H, Lmax))      # -104, -96 or anything to 80
    c["k"] = along[pick]
    j0 = int(g.integers(0, Lmax))
    c["k"][:, :, j0] = oq.encode_ref((-56 if flip else 104) * sign, code)
    c["k_scale"][...] = 2.0 ** -10
    c["weights"][...] = 0
    return c, j0


def rounded_apart(target):
    return 2.0 ** -22 * 1.4427 * target if target * 1.4427 < 4096 else 0.0


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("code,flip", [("e4m3", False), ("int8", True)])
@pytest.mark.parametrize("target", [1e3, 1e5, 3e6, 2.2e7, 1e8, 1e9, 1e30])
def test_decode_weights_of_rows_with_huge_scores(path, dtype, code, flip, target):
    """The best key is 24/104 of the target or more ahead of every other, so it has all the weight
    (e^-173 for any other where the target is 1e3): 1 from each row, up to the rounding of the
    exponential and the division (2^-19).  Up to 4096 in base 2 the score, its maximum and the
    exponent's shift may each be rounded to fp32 apart: 3 * 2^-24 ln 2 of the base-2 score, less
    than 2^-22."""
    B, H, Lmax = PATHS[path]
    check_path(path, B, H, 3, Lmax)
    g = rng(1100 + int(flip))
    sign = g.choice([-1.0, 1.0], 64)
    c, j0 = one_key_cache(g, B, H, Lmax, 32, code, sign, flip)
    Q = np.empty((B, 3 * H, 1, 64))
    Q[...] = sign * target / (104 * 64 / 8 * 2.0 ** -10)
    Q[:, ::3] *= 0.75
    Q = fin(Q, dtype)
    cache = to_gpu(c, 32, code)
    O = mha.sdpa_decode_q8(dev(Q, DT[dtype]), cache, i32([Lmax] * B), add_weights=True)
    w = cache.weights.double().cpu().numpy()
    r = 2.0 ** -19 + rounded_apart(target)
    assert np.abs(w[:, :, j0] - 3).max() <= 3 * r
    w[:, :, j0] = 0
    assert np.abs(w).max() <= 1e-20
    v = oq.values_ref(c["v"][:, :, j0], code) * c["v_scale"][:, :, j0 // 32, None]
    err = np.abs(O.double().cpu().numpy()[:, :, 0] - np.repeat(v, 3, 1))
    bound = (2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else r) * np.abs(v) + 1e-30
    assert np.all(err <= np.repeat(bound, 3, 1))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("target", [1e3, 1e5, 2.2e7, 1e9, 1e30])
@pytest.mark.parametrize("flip", [False, True])
def test_decode_equal_huge_scores_share_the_weight(path, dtype, target, flip):
    """Two equal keys in blocks whose values' scales differ: a half each, whatever the scores."""
    B, H, Lmax = PATHS[path]
    g = rng(1150)
    sign = g.choice([-1.0, 1.0], 64)
    c, j0 = one_key_cache(g, B, H, Lmax, 32, "int8", sign, flip)
    j1 = (j0 + Lmax // 2) % Lmax
    c["k"][:, :, j1] = c["k"][:, :, j0]
    c["v_scale"][:, :, j0 // 32], c["v_scale"][:, :, j1 // 32] = 2.0 ** -6, 2.0 ** 3
    Q = np.empty((B, H, 1, 64))
    Q[...] = sign * target / (104 * 64 / 8 * 2.0 ** -10)
    cache = to_gpu(c, 32, "int8")
    O = mha.sdpa_decode_q8(dev(fin(Q, dtype), DT[dtype]), cache, i32([Lmax] * B), add_weights=True)
    r = 2.0 ** -19 + rounded_apart(target)
    w = cache.weights.double().cpu().numpy()
    assert np.abs(w[:, :, [j0, j1]] - 0.5).max() <= 0.5 * r
    v = [oq.values_ref(c["v"][:, :, j], "int8") * c["v_scale"][:, :, j // 32, None]
         for j in (j0, j1)]
    pv = (np.abs(v[0]) + np.abs(v[1])) / 2
    if dtype == "bf16":
        r += 2.0 ** -11
    want = (v[0] + v[1]) / 2
    bound = r * pv + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    assert np.all(np.abs(O.double().cpu().numpy()[:, :, 0] - want) <= bound + 1e-30)


def weights_of(Q, c, b, h, row, L, block, code, scale=0.125):
    s = oq.dequantised_ref(c, "k", b, h, L, block, code) @ np.asarray(Q[b, row, 0], np.float64)
    p = np.exp(s * scale - (s * scale).max())
    return p / p.sum()


@pytest.mark.parametrize("copies,Lmax", [(1, 96), (1, 768), (240, 790)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("apart", [11, 28, 38, 78])
@pytest.mark.parametrize("order", ["large first", "small first", "mixed"])
def test_decode_values_of_small_scale_beside_large(copies, Lmax, dtype, code, block, apart, order):
    """Columns that only the blocks of small scale have values in are as exact as the others.

    A weight p that meets the codes is fp16 (two terms in the fp32 path) under the largest p s of
    the row so far, 2^13, and off by up to 2^-25 below 2^-14.  Scales less than 2^10 below the
    largest of the tiles so far are summed with them: an error of 2^-38 2^10 max p in p; scales
    further below are summed under their own largest p.  Hence, next to the relative terms,
    2^-28 max p sum_j |v_j| in each column, without any other block's scale."""
    g = rng(1200 + apart)
    c = finite(strange(g, 1, 1, Lmax, block, code), code)
    nb = c["v_scale"].shape[2]
    small = {"large first": np.arange(nb) >= (nb + 1) // 2, "small first": np.arange(nb) < nb // 2,
             "mixed": g.random(nb) < 0.5}[order]
    small[0], small[1] = order == "small first", order != "small first"   # some of either
    c["v_scale"][0, 0] = np.where(small, 2.0 ** -(apart - apart // 2), 2.0 ** (apart // 2))
    large = ~small[np.arange(Lmax) // block]
    c["v"][0, 0, large, :32] = 0
    c["k_scale"][...] = 2.0 ** -9
    Q = np.zeros((1, 3, 1, 64))                  # row 0 attends evenly
    Q[0, 1, 0] = g.standard_normal(64)
    Q[0, 2, 0] = g.standard_normal(64) * 4
    Q = fin(Q, dtype)
    L = Lmax - 3
    # (equal heads, for runs of several tiles to a warp that begin anywhere in a head)
    cache = to_gpu({n: np.repeat(a, copies, 0) for n, a in c.items()}, block, code)
    before = c["weights"].copy()
    O = mha.sdpa_decode_q8(dev(np.repeat(Q, copies, 0), DT[dtype]), cache, i32([L] * copies),
                           add_weights=True)
    got = O.double().cpu().numpy()
    ref, W, pv, _, qk = oq.decode_ref(Q, c, [L], block, code, True)
    close_weights(cache.weights.double().cpu().numpy(), before, W, qk, L, "weights")
    v = np.abs(oq.dequantised_ref(c, "v", 0, 0, L, block, code)).sum(0)
    for row in range(3):
        p = weights_of(Q, c, 0, 0, row, L, block, code)
        close_decode(got[:, row], ref[:, row], pv[:, row], 2.0 ** 10 * p.max() * v, qk, L, dtype,
                     f"row {row}")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,scale", [(1e-30, 1e30), (1e-38, 3e37), (1e30, 1e-31)])
def test_decode_small_and_large_rows_under_a_scale_that_evens_them(path, dtype, size, scale):
    B, H, Lmax = PATHS[path]
    B = min(B, 2) if path != "warp join" else B
    g = rng(1250)
    c = finite(strange(g, B, H, Lmax, 64, "int8"), "int8")
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    c["weights"][...] = 0
    Q = fin(g.standard_normal((B, H, 1, 64)) * size, dtype)
    scale = float(np.float32(scale))
    lens = [Lmax - 5 * (b % 7) for b in range(B)]
    cache = to_gpu(c, 64, "int8")
    O = mha.sdpa_decode_q8(dev(Q, DT[dtype]), cache, i32(lens), scale=scale, add_weights=True)
    ref, W, pv, low, qk = oq.decode_ref(Q, c, lens, 64, "int8", True, scale=scale)
    close_decode(O.double().cpu().numpy(), ref, pv, low, qk, Lmax, dtype, "rows")
    # Weights below 2^-126 come out as 0: fp32 has no normal numbers there and the exponential
    # flushes.  (A value's scale is below 1 here, so the reference m is below the largest score and
    # 2^(x - m) above the weight.)  Scores to both sides of 150 reach e^-300
    w = cache.weights.double().cpu().numpy()
    normal = W >= 2.0 ** -126
    assert np.abs(w[~normal]).max(initial=0.0) <= 2.0 ** -125
    close_weights(w[normal], 0 * W[normal], W[normal], qk, Lmax, "weights")


@pytest.mark.parametrize("dtype,q_size,k_size", [
    ("bf16", 1e30, 1e-30), ("bf16", 1e-30, 1e30), ("f32", 1e30, 1e-30), ("f32", 1e-30, 1e30),
    ("f32", 3e37, 1e-37), ("f32", 1e-37, 1e37), ("f32", 5e37, 1e-42), ("f32", 1.0, 1e-44)])
def test_key_weights_of_rows_far_below_and_above_one(dtype, q_size, k_size):
    """Scores of ordinary size from rows whose values are anything but.  The bound is that of
    test_key_weights."""
    g = rng(1300)
    Q = fin(g.standard_normal((1, 2, 70, 64)) * q_size, dtype)
    K = fin(g.standard_normal((1, 1, 90, 64)) * k_size, dtype)
    lse = oracle.sdpa_lse_ref(Q, np.repeat(K, 2, 1), "none").astype(np.float32)
    w = mha.sdpa_key_weights(dev(Q, DT[dtype]), dev(K, DT[dtype]), dev(lse))
    ref = oq.key_weights_ref(Q, K, lse, "none")
    S = np.abs(Q[0]).astype(np.float64) @ np.abs(K[0, 0]).astype(np.float64).T / 8
    r = 2.0 ** -18 * S.max() + 2.0 ** -23 * np.abs(lse).max() + 2.0 ** -20 + 140 * 2.0 ** -24
    assert np.all(np.abs(w.double().cpu().numpy() - ref) <= r * ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_key_weights_of_more_than_65535_heads(dtype):
    B, H, N = 67, 1000, 3
    g = rng(1350)
    q, k = (dev(fin(g.standard_normal((B, H, N, 64)), dtype), DT[dtype]) for _ in range(2))
    _, lse = mha.sdpa_with_lse(q, k, k, "causal")
    w = mha.sdpa_key_weights(q, k, lse, "causal")
    s = (q.double() @ k.double().transpose(2, 3) / 8).tril()
    p = torch.exp(s - lse.double()[..., None]).tril()
    # sum |q||k| / 8 is below 16: 64 roundings to fp32 are 2^-14 in all; lse is below 16: 2^-20
    assert torch.all((w - p.sum(2)).abs() <= 2.0 ** -11 * p.sum(2))
    assert torch.allclose(w.sum(-1), torch.full((B, H), 3.0, device="cuda"), rtol=2.0 ** -11)


SHARES = r"""
#include "sdpa_key_weights.cu"
// the second launch on its own: shares [split][heads][keys] onto weights [heads][keys]
extern "C" int add_shares(int heads, int keys, int split, float* shares, float* weights) {
  mha::KwParams p = {};
  p.a.Hkv = heads;
  p.a.Nk = keys;
  p.a.ld = keys;
  p.a.weights = weights;
  p.split = split;
  p.part = shares;
  mha::key_weights_add_kernel<<<dim3((keys + 255) / 256, heads), dim3(256)>>>(p);
  return cudaDeviceSynchronize();
}
"""


def test_key_weights_stay_where_a_share_is_missing(tmp_path):
    """A share that a time-out left out is marked, and the keys' running totals stay as they were.
    (The mark is made here: a wait is not made to run out with copies in flight.)"""
    from transformer_head_scaled_04_gb300 import build

    src, lib = tmp_path / "shares.cu", tmp_path / "shares.so"
    src.write_text(SHARES)
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", str(src), "-o",
                    str(lib)], check=True)
    # (lazily: what the file needs of others for the first launch stays unresolved, and uncalled)
    add = ctypes.CDLL(str(lib), mode=os.RTLD_LAZY).add_shares
    g = rng(1380)
    shares = g.random((5, 3, 300)).astype(np.float32)
    shares[2, 1, 250:] = -1
    shares[4, 0, 7] = -1
    before = g.random((3, 300)).astype(np.float32)
    w, s = dev(before), dev(shares)
    assert add(3, 300, 5, ctypes.c_void_p(s.data_ptr()), ctypes.c_void_p(w.data_ptr())) == 0
    missing = (shares < 0).any(0)
    got = w.cpu().numpy()
    assert np.array_equal(got[missing], before[missing])
    want = before + shares.astype(np.float64).sum(0)
    assert np.all(np.abs(got - want)[~missing] <= 5 * 2.0 ** -24 * 6)


APPEND = [  # N, cache_len, scales of the begun blocks
    (3, [20, 33], 0.011), (40, [5, 63], 0.3), (1, [47, 1], 3e-10), (70, [16, 9], 1e4)]


@pytest.mark.parametrize("N,cl,scale", APPEND)
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-3, 30.0])      # the begun block keeps its scale, or not
def test_append_under_scales_that_are_no_powers_of_two(N, cl, scale, code, dtype, size):
    g = rng(1400 + N)
    c = strange(g, 2, 3, 200, 32, code)
    c["k_scale"][...] = np.float32(scale)
    c["v_scale"][...] = np.float32(scale) * g.uniform(0.5, 2, c["v_scale"].shape)
    for n in "kv":
        c[n + "_scale"] = c[n + "_scale"].astype(np.float32).astype(np.float64)
    k, v = (fin(g.standard_normal((2, 3, N, 64)) * size, dtype) for _ in range(2))
    cache = to_gpu(c, 32, code)
    mha.kv_append_q8(cache, dev(k, DT[dtype]), dev(v, DT[dtype]), i32(cl))
    assert_same(from_gpu(cache), oq.append_ref(c, k, v, cl, None, 32, code), code, "append")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 128])
def test_evict_under_scales_that_are_no_powers_of_two(code, block):
    g = rng(1450)
    c, d = strange(g, 2, 2, 900, block, code), strange(g, 2, 2, 400, block, code)
    for n in "kv":
        s = np.exp(g.uniform(-5, 5, c[n + "_scale"].shape))
        c[n + "_scale"] = s.astype(np.float32).astype(np.float64)
    src, out = to_gpu(c, block, code), to_gpu(d, block, code)
    mha.kv_evict_q8(src, out, i32([900, 431]), 333, 20)
    want, _, _ = oq.evict_ref(c, d, [900, 431], 333, 20, block, code)
    assert_same(from_gpu(out), want, code, "evict")


# ---- special rows on every path of the generation step
def plain_cache(g, B, H, Lmax, block, code):
    c = finite(strange(g, B, H, Lmax, block, code), code)
    for n in "kv":
        c[n + "_scale"] *= 2.0 ** -6
    return c


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_token_major_with_a_workspace_on_every_path(path, dtype):
    B, H, Lmax = PATHS[path]
    g = rng(1500)
    c = plain_cache(g, B, H, Lmax, 64, "int8")
    c["weights"][...] = 0
    lens = [Lmax - 7 * (b % 5) for b in range(B)]
    cache = to_gpu(c, 64, "int8", token_major=True)
    Q = fin(g.standard_normal((B, 2 * H, 2, 64)), dtype)
    tq = dev(Q, DT[dtype]).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    out = torch.zeros(B, 2, 2 * H, 64, dtype=DT[dtype], device="cuda").permute(0, 2, 1, 3)
    ws = torch.empty(mha.decode_q8_workspace_size(B, 2 * H, H, 2, Lmax, True), dtype=torch.uint8,
                     device="cuda")
    assert (ws.numel() == 0) == (path == "one launch")
    results = []
    for _ in range(2):                      # the same bits again, the weights' among them
        cache.weights.zero_()
        mha.sdpa_decode_q8(tq, cache, i32(lens), scale=0.05, workspace=ws, out=out,
                           add_weights=True)
        results.append((out.clone(), cache.weights.clone()))
        ws.fill_(255)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    few = min(B, 2)
    ref, W, pv, low, qk = oq.decode_ref(Q[:few], {n: a[:few] for n, a in c.items()}, lens, 64,
                                        "int8", True, scale=0.05)
    close_decode(out[:few].double().cpu().numpy(), ref, pv, low, qk, Lmax, dtype, path)
    close_weights(cache.weights[:few].double().cpu().numpy(), 0 * W, W, qk, Lmax, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_rows_without_keys_on_every_path(path, dtype):
    """Lengths shorter than the number of new queries: the first rows see nothing."""
    B, H, Lmax = PATHS[path]
    g = rng(1520)
    c = plain_cache(g, B, H, Lmax, 32, "e4m3")
    before = c["weights"].copy()
    lens = [b % 4 if b or B > 1 else 3 for b in range(B)]
    Q = fin(g.standard_normal((B, H, 5, 64)), dtype)
    cache = to_gpu(c, 32, "e4m3")
    O = mha.sdpa_decode_q8(dev(Q, DT[dtype]), cache, i32(lens), add_weights=True)
    ref, W, pv, low, qk = oq.decode_ref(Q, c, lens, 32, "e4m3", True)
    got = O.double().cpu().numpy()
    close_decode(got, ref, pv, low, qk, 5, dtype, path)
    assert np.all(got[pv == 0] == 0)
    w = cache.weights.double().cpu().numpy()
    close_weights(w, before, W, qk, 5, path)
    assert np.array_equal(w[W == 0], before[W == 0])


@pytest.mark.parametrize("path", PATHS)
def test_decode_nan_on_every_path(path):
    """NaN in one query row, in a value and in a key, of sequence 0: it reaches the rows that see
    it and nothing else, and the weights of a NaN row's positions only."""
    B, H, Lmax = PATHS[path]
    g = rng(1540)
    Nq, L = 4, Lmax - 3
    for what in ("query", "value", "key"):
        for at in (L - 2, L // 2):
            c = plain_cache(g, B, H, Lmax, 16, "e4m3")
            c["weights"][...] = 0
            Q = fin(g.standard_normal((B, 2 * H, Nq, 64)), "bf16")
            want = torch.zeros(B, 2 * H, Nq, 64, dtype=torch.bool)
            sees = slice(2 if at == L - 2 else 0, Nq)
            if what == "query":
                Q[0, 1, 0] = np.nan
                want[0, 1, 0] = True
            elif what == "value":
                c["v"][0, 0, at, 7] = 127
                want[0, :2, sees, 7] = True
            else:
                c["k"][0, 0, at, 9] = 255
                want[0, :2, sees] = True
            cache = to_gpu(c, 16, "e4m3")
            O = mha.sdpa_decode_q8(dev(Q, torch.bfloat16), cache, i32([L] * B), add_weights=True)
            assert torch.equal(torch.isnan(O).cpu(), want), f"{what} {at}"
            bad = torch.isnan(cache.weights).cpu()
            seen = torch.zeros(B, H, Lmax, dtype=torch.bool)
            if what == "query":
                seen[0, 0, :L - Nq + 1] = True
            elif what == "key":
                seen[0, 0, :L] = True
            assert torch.equal(bad, seen), f"{what} {at}: weights"


@pytest.mark.parametrize("path", PATHS)
def test_captured_steps_on_every_path(path):
    """Append and attention with weights in a graph, replayed while the lengths grow over tile and
    block ends, give what the same calls give outside."""
    B, H, Lmax = PATHS[path]
    g = rng(1560)
    base = plain_cache(g, B, H, Lmax, 64, "int8")
    steps = [[dev(fin(g.standard_normal((B, H, 1, 64)), "bf16"), torch.bfloat16)
              for _ in range(3)] for _ in range(5)]
    ws = torch.empty(mha.decode_q8_workspace_size(B, H, H, 1, Lmax, True), dtype=torch.uint8,
                     device="cuda")

    def step(cache, q, k, v, n, out):
        mha.kv_append_q8(cache, k, v, n)
        n.add_(1)
        mha.sdpa_decode_q8(q, cache, n, add_weights=True, out=out, workspace=ws)

    def begin():
        n = i32([(b * 31) % 60 for b in range(B)])
        n[0] = Lmax - 5
        return to_gpu(base, 64, "int8"), n, torch.zeros_like(steps[0][0])

    cache, n, out = begin()
    want = []
    for s in steps:
        step(cache, *s, n, out)
        want.append(out.clone())
    final = from_gpu(cache)
    cache, n, out = begin()
    q, k, v = (torch.empty_like(x) for x in steps[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, q, k, v, n, out)
    for s, o in zip(steps, want):
        for a, x in zip((q, k, v), s):
            a.copy_(x)
        graph.replay()
        assert torch.equal(out, o)
    assert_same(from_gpu(cache), final, "int8", "replayed")


def test_prompt_eviction_and_steps_in_two_launches():
    """The whole sequence of calls on a cache too long for the one-launch step."""
    g = rng(1580)
    B, H, N, Lmax, keep, block = 2, 1, 1900, 2000, 1200, 64
    lens = [1900, 1300]
    q, k, v = (fin(g.standard_normal((B, H, N, 64)), "bf16") for _ in range(3))
    tq, tk, tv = (dev(x, torch.bfloat16) for x in (q, k, v))
    cache = mha.kv_cache_q8(B, H, Lmax, block)
    n = i32([0, 0])
    mha.kv_append_q8(cache, tk, tv, n, i32(lens))
    _, lse = mha.sdpa_with_lse(tq, tk, tv, "causal")
    mha.sdpa_key_weights(tq, tk, lse, "causal", None, i32(lens), weights=cache.weights)
    c = from_gpu(cache)
    small = mha.kv_cache_q8(B, H, keep + 50, block)
    blank = from_gpu(small)
    n, kept = mha.kv_evict_q8(cache, small, i32(lens), keep, 100)
    c, wn, wkept = oq.evict_ref(c, blank, lens, keep, 100, block, "e4m3")
    assert np.array_equal(kept.cpu().numpy(), wkept) and n.tolist() == wn.tolist()
    assert mha.decode_q8_workspace_size(B, 2 * H, H, 3, keep + 50, True) > 0
    for step in range(2):
        k, v = (fin(g.standard_normal((B, H, 3, 64)), "bf16") for _ in range(2))
        q = fin(g.standard_normal((B, 2 * H, 3, 64)), "bf16")
        mha.kv_append_q8(small, dev(k, torch.bfloat16), dev(v, torch.bfloat16), n)
        c = oq.append_ref(c, k, v, n.tolist(), None, block, "e4m3")
        n = n + 3
        O = mha.sdpa_decode_q8(dev(q, torch.bfloat16), small, n, add_weights=True)
        ref, W, pv, low, qk = oq.decode_ref(q, c, n.tolist(), block, "e4m3", True)
        close_decode(O.double().cpu().numpy(), ref, pv, low, qk, keep + 8, "bf16", f"step {step}")
        got = from_gpu(small)
        close_weights(got["weights"], c["weights"], W, qk, keep + 8, f"weights {step}")
        c["weights"] = got["weights"]
        assert_same(got, c, "e4m3", f"cache {step}")
