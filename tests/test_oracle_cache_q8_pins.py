"""Pins of the 8-bit cache's oracle, independent of its own formulas (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache_q8 as oq


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def empty(B, H, Lmax, block):
    nb = -(-Lmax // block)
    return {"k": np.zeros((B, H, Lmax, 64), np.uint8), "v": np.zeros((B, H, Lmax, 64), np.uint8),
            "k_scale": np.ones((B, H, nb)), "v_scale": np.ones((B, H, nb)),
            "weights": np.zeros((B, H, Lmax))}


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert np.array_equal(oq.TABLE["e4m3"], t.numpy(), equal_nan=True)


def test_e4m3_encoding_is_torchs():
    # torch rounds to nearest even too; every midpoint of neighbours is among the values
    pos = oq.TABLE["e4m3"][:127]
    x = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, rng(1).standard_normal(5000) * 100,
                        rng(2).standard_normal(5000) * 0.01])
    x = np.clip(np.concatenate([x, -x]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oq.encode_ref(x, "e4m3"), want)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_codes_are_the_nearest(code):
    x = rng(3).uniform(-1.2, 1.2, 2000) * oq.QMAX[code]
    got = oq.values_ref(oq.encode_ref(x, code), code)
    table = oq.TABLE[code][np.isfinite(oq.TABLE[code])]
    if code == "int8":
        table = table[table > -128]
    best = np.abs(x[:, None] - table[None]).min(1)
    assert np.array_equal(np.abs(x - got), best)
    assert oq.encode_ref([np.nan], code)[0] == (127 if code == "e4m3" else 0)
    assert oq.values_ref(oq.encode_ref([np.inf, -np.inf], code), code).tolist() == \
        [oq.QMAX[code], -oq.QMAX[code]]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_scale_is_the_least_power_of_two(code):
    for amax in (1e-30, 1e-3, 1.0, 447.9, 448.0, 448.1, 127.0, 127.5, 1e9, 1e30, 0.0):
        s = oq.scale_ref([amax, -amax / 2, np.nan, np.inf], code)
        assert np.log2(s) == round(np.log2(s)) and 2.0 ** -40 <= s <= 2.0 ** 40
        assert s == 2.0 ** 40 or amax <= oq.QMAX[code] * s
        assert s == 2.0 ** -40 or amax > oq.QMAX[code] * s / 2


def test_quantisation_error_is_half_a_step():
    x = rng(4).standard_normal((1, 1, 64, 64))
    for code, rel, step in (("e4m3", 2.0 ** -4, 2.0 ** -10), ("int8", 0.0, 0.5)):
        c = oq.append_ref(empty(1, 1, 64, 64), x, x, [0], None, 64, code)
        back = oq.dequantised_ref(c, "k", 0, 0, 64, 64, code)
        s = c["k_scale"][0, 0, 0]
        assert np.all(np.abs(back - x[0, 0]) <= rel * np.abs(x[0, 0]) + step * s)


def test_append_in_pieces_of_one_scale_equals_append_at_once():
    x = rng(5).standard_normal((1, 2, 40, 64))
    x[:, :, 0, 0] = 7.0  # the largest magnitude comes first: the scale never grows
    at_once = oq.append_ref(empty(1, 2, 50, 64), x, -x, [0], None, 64, "e4m3")
    c = empty(1, 2, 50, 64)
    for lo, hi in ((0, 1), (1, 17), (17, 40)):
        c = oq.append_ref(c, x[:, :, lo:hi], -x[:, :, lo:hi], [lo], None, 64, "e4m3")
    assert all(np.array_equal(c[n], at_once[n]) for n in c)


def test_a_larger_token_rescales_its_block_only():
    x = rng(6).standard_normal((1, 1, 40, 64))
    c = oq.append_ref(empty(1, 1, 64, 16), x, x, [0], None, 16, "int8")
    big = np.full((1, 1, 1, 64), 1000.0)
    d = oq.append_ref(c, big, big, [40], None, 16, "int8")
    assert np.array_equal(c["k"][0, 0, :32], d["k"][0, 0, :32])
    assert d["k_scale"][0, 0, 2] == 8.0 and d["k_scale"][0, 0, 1] == c["k_scale"][0, 0, 1]
    old, new = (oq.dequantised_ref(e, "k", 0, 0, 40, 16, "int8")[32:] for e in (c, d))
    assert np.abs(old - new).max() <= 4.0  # half the new step


@pytest.mark.parametrize("causal", [True, False])
def test_decode_is_the_attention_of_the_dequantised_cache(causal):
    g = rng(7)
    c = oq.append_ref(empty(2, 2, 50, 16), g.standard_normal((2, 2, 45, 64)),
                      g.standard_normal((2, 2, 45, 64)), [0, 0], [45, 20], 16, "e4m3")
    Q = g.standard_normal((2, 4, 3, 64))
    O, W, _, _, _ = oq.decode_ref(Q, c, [45, 20], 16, "e4m3", causal)
    k, v = (np.stack([np.stack([oq.dequantised_ref(c, n, b, h // 2, 50, 16, "e4m3")
                                for h in range(4)]) for b in range(2)]) for n in "kv")
    ref = oracle.sdpa_ref(Q, k, v, "causal_cache" if causal else "key_padding",
                          np.array([45, 20], np.int32))
    assert np.allclose(O, ref, rtol=1e-12, atol=1e-12)
    assert np.allclose(W.sum(-1), 2 * 3)  # two heads of a group, three queries


@pytest.mark.parametrize("mask", ["none", "causal", "key_padding"])
def test_key_weights_are_the_column_sums(mask):
    g = rng(8)
    Q, K = g.standard_normal((2, 4, 30, 64)), g.standard_normal((2, 2, 30, 64))
    kl = np.array([30, 11], np.int32)
    Kx = np.repeat(K, 2, 1)
    lse = oracle.sdpa_lse_ref(Q, Kx, mask, kl)
    W = oq.key_weights_ref(Q, K, lse, mask, kl)
    for b in range(2):
        for h in range(2):
            want = 0.0
            for x in (2 * h, 2 * h + 1):
                allowed = oracle.allowed_keys(mask, 30, 30, int(kl[b]))
                want = want + oracle.attention_weights_ref(Q[b, x], Kx[b, x], allowed).sum(0)
            assert np.allclose(W[b, h], want, rtol=1e-12, atol=1e-14)


def test_padded_query_rows_add_nothing():
    g = rng(9)
    Q, K = g.standard_normal((1, 1, 20, 64)), g.standard_normal((1, 1, 20, 64))
    lse = oracle.sdpa_lse_ref(Q, K, "causal")
    W = oq.key_weights_ref(Q, K, lse, "causal", None, [7])
    W7 = oq.key_weights_ref(Q[:, :, :7], K[:, :, :7], lse[:, :, :7], "causal")
    assert np.array_equal(W[..., :7], W7) and np.all(W[..., 7:] == 0)


def test_kept_positions():
    w = np.array([5.0, 1.0, 5.0, 5.0, 0.0, 9.0, 0.0, 0.0])
    assert oq.kept_ref(w, 8, 4, 1) == [0, 2, 5, 7]      # of three equal weights the lowest two
    assert oq.kept_ref(w, 8, 4, 4) == [4, 5, 6, 7]
    assert oq.kept_ref(w, 8, 4, 9) == [4, 5, 6, 7]
    assert oq.kept_ref(w, 4, 4, 0) == [0, 1, 2, 3]
    assert oq.kept_ref(w, 0, 4, 0) == []
    assert oq.kept_ref(np.array([np.nan, -1.0, -np.inf, np.nan, 2.0]), 5, 2, 0) == [1, 4]


def test_evicting_nothing_copies_and_attention_is_unchanged():
    g = rng(10)
    x = g.standard_normal((1, 1, 33, 64))
    c = oq.append_ref(empty(1, 1, 40, 16), x, x[:, :, ::-1], [0], None, 16, "e4m3")
    c["weights"][...] = g.random((1, 1, 40))
    d, n, kept = oq.evict_ref(c, empty(1, 1, 64, 16), [33], 50, 3, 16, "e4m3")
    assert n[0] == 33 and kept[0, 0, :33].tolist() == list(range(33))
    assert np.array_equal(d["k"][0, 0, :33], c["k"][0, 0, :33])
    assert np.array_equal(d["k_scale"][0, 0, :3], c["k_scale"][0, 0, :3])
