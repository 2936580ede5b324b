"""Pins of the oracle of the learned relative position bias, and the library's buckets against it
(on the host: no GPU)."""
import numpy as np
import pytest

import oracle
from oracle.rel_bias import bucket_ref, sdpa_rel_bwd_ref, sdpa_rel_decode_ref, sdpa_rel_ref


def test_buckets_written_out():
    # 32 buckets, reach 128, both sides: 8 of a side's 16 are single distances, the others double
    # every two: borders 8, 12 (11.3), 16, 23 (22.6), 32, 46 (45.3), 64, 91 (90.5)
    want = list(range(8)) + [8] * 4 + [9] * 4 + [10] * 7 + [11] * 9 + [12] * 14 + [13] * 18 \
        + [14] * 27 + [15] * 100
    assert [bucket_ref(-n, 32, 128, True) for n in range(len(want))] == want
    assert [bucket_ref(n, 32, 128, True) for n in range(1, len(want))] == [16 + u for u in want[1:]]
    # one side: keys after the query share bucket 0; 4 single distances of 8, borders 4 * 8^(t/4)
    want = [0, 1, 2, 3, 4, 4, 4, 5, 5, 5, 5, 5, 6, 6, 6, 6, 6, 6, 6, 6, 7, 7]
    assert [bucket_ref(-n, 8, 32, False) for n in range(len(want))] == want[:7] + want[7:]
    assert {bucket_ref(n, 8, 32, False) for n in range(100)} == {0}
    assert bucket_ref(-32, 8, 32, False) == bucket_ref(-10**6, 8, 32, False) == 7


@pytest.mark.parametrize("num,reach,both", [
    (2, 2, False), (3, 5, False), (4, 9, True), (8, 9, True), (16, 17, False), (32, 128, True),
    (32, 128, False), (64, 500, True), (128, 65, False), (128, 4096, True), (128, 100000, False),
    (10, 6, False), (126, 1000, True)])
def test_library_buckets(num, reach, both):
    import transformer_head_scaled_04_gb300 as mha
    from transformer_head_scaled_04_gb300 import build

    build.build()
    per = num // 2 if both else num
    e = per // 2
    ds = set(range(-200, 201)) | {reach * s + i for s in (1, -1) for i in (-1, 0, 1)}
    for t in range(per - e + 1):  # around every border
        b = round(e * (reach / e) ** (t / (per - e)))
        ds |= {s * (b + i) for s in (1, -1) for i in (-1, 0, 1)}
    for d in sorted(ds):
        assert mha.rel_bucket(d, num, reach, both) == bucket_ref(d, num, reach, both), d
    for d in (2**31 - 1, -2**31):
        far = 4 * reach if d > 0 else -4 * reach
        assert mha.rel_bucket(d, num, reach, both) == bucket_ref(far, num, reach, both)


def draw(seed, B=1, H=2, Nq=5, Nk=7, d=3, num=8):
    g = np.random.Generator(np.random.PCG64(seed))
    n = g.standard_normal
    return n((B, H, Nq, d)), n((B, H, Nk, d)), n((B, H, Nk, d)), n((num, H))


def test_zero_bias_is_plain_attention():
    Q, K, V, T = draw(1)
    O, lse = sdpa_rel_ref(Q, K, V, 0 * T, max_distance=16)
    assert np.allclose(O, oracle.sdpa_ref(Q, K, V), rtol=0, atol=1e-14)
    assert np.allclose(lse, oracle.sdpa_lse_ref(Q, K), rtol=0, atol=1e-14)
    # a bias that all distances share changes nothing but the log-sum-exp
    O1, lse1 = sdpa_rel_ref(Q, K, V, 0 * T + 3.5, max_distance=16)
    assert np.allclose(O1, O, rtol=0, atol=1e-13) and np.allclose(lse1, lse + 3.5, atol=1e-13)


def test_forward_by_hand():
    # one query at position 0, three keys, scores 0: weights go by exp(bias) alone
    Q, K = np.zeros((1, 1, 1, 2)), np.zeros((1, 1, 3, 2))
    V = np.arange(6.0).reshape(1, 1, 3, 2)
    T = np.log(np.array([[1.0], [9.0], [9.0], [2.0]]))  # d = 0: bucket 0; d = 1, 2: bucket 3
    O, lse = sdpa_rel_ref(Q, K, V, T, max_distance=8)
    assert np.allclose(lse, np.log(5.0)) and np.allclose(O[0, 0, 0], (V[0, 0] * [[1], [2], [2]]).sum(0) / 5)


@pytest.mark.parametrize("mask,both", [("none", True), ("causal", False), ("key_padding", True)])
def test_gradients_against_differences(mask, both):
    Q, K, V, T = draw(2, B=2, Nq=6, Nk=6)
    dO = draw(3, B=2, Nq=6, Nk=6)[0]
    kl = [4, 6] if mask == "key_padding" else None
    how = dict(mask=mask, key_len=kl, max_distance=5 if both else 9, bidirectional=both)
    got = sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)
    args = [Q, K, V, T]
    h = 1e-6
    for a, g in zip(args, got):
        want = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + h
            up = (sdpa_rel_ref(*args, **how)[0] * dO).sum()
            a[i] = old - h
            want[i] = (up - (sdpa_rel_ref(*args, **how)[0] * dO).sum()) / (2 * h)
            a[i] = old
        assert np.allclose(g, want, rtol=1e-6, atol=1e-8)
    given = sdpa_rel_bwd_ref(Q, K, V, T, dO, given=sdpa_rel_ref(Q, K, V, T, **how), **how)
    for a, b in zip(got, given):
        assert np.allclose(a, b, rtol=1e-10, atol=1e-12)
    # weights of a row sum to 1 whatever the bias: the table's gradients of a head sum to 0
    assert np.allclose(got[3].sum(0), 0, atol=1e-12)


def test_decode_is_the_last_rows_of_the_causal_forward():
    Q, K, V, T = draw(4, B=2, Nq=9, Nk=9)
    O, _ = sdpa_rel_ref(Q, K, V, T, "causal", max_distance=20, bidirectional=False)
    got = sdpa_rel_decode_ref(Q[:, :, 6:], K, V, T, [9, 9], max_distance=20)
    assert np.allclose(got, O[:, :, 6:], rtol=0, atol=1e-14)
    short = sdpa_rel_decode_ref(Q[:, :, 3:5], K, V, T, [5, 1], max_distance=20)
    assert np.allclose(short[0], O[0, :, 3:5], atol=1e-14)
    # one cached position, two queries: the first has none to see, the second sees that one
    assert np.all(short[1, :, 0] == 0) and np.allclose(short[1, :, 1], V[1, :, 0])


@pytest.mark.parametrize("num,reach,both,n", [
    (7, 8020466, False, 198349), (8, 15688794, False, 352539), (16, 15688794, True, 352539),
    (10, 5497271, False, 340339), (16, 2382133, False, 492869), (31, 10443359, False, 29016),
    (64, 13251718, True, 79977), (64, 1124401, False, 584535), (128, 16723489, True, 11082401),
    # and borders that are whole numbers
    (32, 128, True, 16), (32, 128, True, 64), (8, 32, False, 32), (128, 64 * 2 ** 16, False, 128)])
def test_library_buckets_next_to_a_border(num, reach, both, n):
    # a border lies at n or above it by less than 1e-12 of it (n then belongs to the nearer bucket)
    import transformer_head_scaled_04_gb300 as mha
    from transformer_head_scaled_04_gb300 import build

    build.build()
    for d in (n - 1, n, n + 1):
        for s in (1, -1):
            assert mha.rel_bucket(s * d, num, reach, both) == bucket_ref(s * d, num, reach, both)
