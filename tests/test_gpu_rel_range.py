"""Attention with a learned relative position bias at the ends of what its entry points take, against
the CPU oracle (``oracle.rel_bias``) or the formulas in 64 bits on the GPU."""
import numpy as np
import pytest
import torch

import seeded_inputs as si
from oracle import rel_bias as ref
from parity_util import assert_f32_close
from test_gpu_rel import (BF, F, check_lse, close, det_mode, dev, draw, host, i32,  # noqa: F401
                          near_enough, plain64, within)

pytestmark = pytest.mark.gpu

mha = pytest.importorskip("transformer_head_scaled_04_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_head_scaled_04_gb300 import build

    build.build()
    mha.load_library()
    torch.cuda.set_device(0)
    mha.device_status()
    yield
    assert mha.device_status() == 0, "a kernel recorded a device-side error"


# ------------------------------------------------------------------ fp32: rows of very different sizes
@pytest.mark.parametrize("d", [64, 100])
@pytest.mark.parametrize("size", [1e8, 1e12, 1e30])
@pytest.mark.parametrize("where", ["keys", "queries"])
@pytest.mark.parametrize("hidden", ["causal", "excluded", "faint"])
def test_fp32_rows_that_are_not_seen_may_be_of_any_size(hidden, where, size, d):
    # One huge row that no row of ordinary size sees (or only at a weight of e^-60): the others keep
    # fp32's accuracy.  The last key is seen by the last query alone, whose own row is 0, so that its
    # scores and gradients stay ordinary; the first query sees the first key alone, likewise 0.
    if hidden == "faint" and size > 1e12:
        pytest.skip("at e^-60 it is not faint any more")
    B, H, N = 1, 2, 150
    Q, K, V, dO, T = draw(B, H, N, N, F, 960, dk=d, dv=d)
    if where == "keys":
        V[:, :, -1] *= size
        Q[:, :, -1] = dO[:, :, -1] = 0
        if hidden != "faint":
            K[:, :, -1] *= size
    else:
        dO[:, :, 0] *= size
        K[:, :, 0] = V[:, :, 0] = 0
        if hidden != "faint":
            Q[:, :, 0] *= size
    Q, K, V, dO = (np.asarray(a, np.float32).astype(np.float64) for a in (Q, K, V, dO))
    if hidden != "causal":  # keys after the query
        T[16:] = -np.inf if hidden == "excluded" else -60.0
    how = dict(mask="causal" if hidden == "causal" else "none", max_distance=128)
    q, k, v, g, t = (dev(a, F) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
    with np.errstate(invalid="ignore", over="ignore"):
        rO, rl = ref.sdpa_rel_ref(Q, K, V, T, **how)
        want = (rO,) + ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)[:3]
        bounds = ref.element_bounds(Q, K, V, T, dO, 2.0 ** -24, 2.0 ** -15 + 2.0 ** -24 * 16, **how)
    assert np.abs(rl).max() < 16
    assert np.abs(lse.cpu().numpy() - rl).max() <= 2.0 ** -15 + 2.0 ** -24 * 16
    for a, w, tol, n in zip((O,) + got[:3], want, bounds, ("O", "dQ", "dK", "dV")):
        within(host(a), w, tol, n)
        plain = slice(1, -1)  # the rows of ordinary size, held to the fp32 path's own bounds
        assert_f32_close(host(a)[:, :, plain], w[:, :, plain], f"rel hidden rows {n}")
    given = (host(O), lse.cpu().numpy())
    with np.errstate(invalid="ignore", over="ignore"):
        w = ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, given=given, **how)[3]
        tol = ref.table_grad_bound(Q, K, V, T, dO, *given, **how)
    within(host(got[3]), w, tol + 2.0 ** -24 * np.abs(w), "dtable")


@pytest.mark.parametrize("size", [1e8, 1e30])
@pytest.mark.parametrize("where", ["keys", "queries"])
@pytest.mark.parametrize("hidden", ["causal", "excluded"])
def test_bf16_rows_that_are_not_seen_may_be_of_any_size(hidden, where, size, det_mode):
    # the same inputs in bf16: every element within its own bound
    B, H, N = 1, 2, 150
    Q, K, V, dO, T = draw(B, H, N, N, BF, 961)
    if where == "keys":
        K[:, :, -1] *= size
        V[:, :, -1] *= size
        Q[:, :, -1] = dO[:, :, -1] = 0
    else:
        Q[:, :, 0] *= size
        dO[:, :, 0] *= size
        K[:, :, 0] = V[:, :, 0] = 0
    Q, K, V, dO = (si.round_bf16(a) for a in (Q, K, V, dO))
    if hidden == "excluded":
        T[16:] = -np.inf
    how = dict(mask="causal" if hidden == "causal" else "none", max_distance=128)
    q, k, v, g = (dev(a, BF) for a in (Q, K, V, dO))
    t = dev(T, F)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
    with np.errstate(invalid="ignore", over="ignore"):
        rO, rl = ref.sdpa_rel_ref(Q, K, V, T, **how)
        want = (rO,) + ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)[:3]
        bounds = ref.element_bounds(Q, K, V, T, dO, 2.0 ** -8, 2.0 ** -15 + 2.0 ** -24 * 16, **how)
    check_lse(lse.cpu().numpy(), rl)
    for a, w, tol, n in zip((O,) + got[:3], want, bounds, ("O", "dQ", "dK", "dV")):
        within(host(a), w, tol, n)


# ------------------------------------------------------------------ lengths that the last launch writes
@pytest.mark.parametrize("bias", [False, True])
def test_lengths_from_the_kernel_before(bias):
    # an eviction writes the lengths that the attention right behind it goes by, in one graph: the
    # attention's blocks may start before the eviction is through, but read no length before that
    B, H, L, N = 16, 16, 8192, 300
    cache, small = (mha.kv_cache_q8(B, H, n) for n in (L, N))
    cache.weights.uniform_()
    lens = i32([L if b % 3 else 17 * b for b in range(B)])
    n, kept = torch.zeros_like(lens), torch.empty((B, H, N), dtype=torch.int32, device="cuda")
    torch.manual_seed(2)
    q, k, v = (torch.randn(B, H, N, 64, device="cuda").to(BF) for _ in range(3))
    t = torch.randn(32, H, device="cuda")

    def attend():
        if bias:
            return mha.sdpa_rel_with_lse(q, k, v, t, "key_padding", n)
        return mha.sdpa_with_lse(q, k, v, "key_padding", n)

    def both():
        mha.kv_evict_q8(cache, small, lens, keep=N, len_out=n, kept=kept)
        return attend()

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(20):
        n.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert n.tolist() == [min(x, N) for x in lens.tolist()]
        for a, b in zip(got, attend()):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ NaN and infinities that are seen
@pytest.mark.parametrize("dtype,Nq", [(BF, 1), (BF, 5), (F, 1), (F, 2), (F, 5)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("L", [40, 3000])
def test_step_shows_nan_that_a_query_sees(dtype, Nq, bad, L):
    # a NaN among a query's scores makes its row NaN, not zeros (those say that it sees no key)
    Q, K, V, _, T = draw(3, 2, Nq, L, dtype, 970)
    q, k, v, t = (dev(a, dtype) for a in (Q, K, V, T))
    n = i32([L, L // 2, 0])
    want = mha.sdpa_rel_decode(q, k, v, t, n)
    k[:2, :, 7] = bad
    k[2] = bad
    got = mha.sdpa_rel_decode(q, k, v, t, n)
    assert torch.all(torch.isnan(got[:2])) and torch.all(got[2] == 0)
    k[1] = dev(K, dtype)[1]  # the sequences beside it are as before
    got = mha.sdpa_rel_decode(q, k, v, t, n)
    assert torch.all(torch.isnan(got[0])) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ long sums of the table's gradient
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,H,N", [(65535, 1, 2), (1, 1, 131072)])
def test_table_gradient_over_long_sums(dtype, B, H, N, det_mode):
    # Every pair's dS is the same number: with Q = K = 0, a table of zeros, lse = 0 and O = 0 the weight is
    # 2^0 and dS = dO.V = x.  x has 18 bits, so 64 of them add up exactly; what is left are the roundings
    # of sums over lanes, warps and tiles, fewer than 32 of 2^-24 in a row of additions whose length does
    # not count.  (One running sum of 1024 x is off by 6.6e-6 of it, one of 8192 by 8e-5.)
    if det_mode and dtype is F:
        pytest.skip("the switch works on bf16 alone")
    zero = torch.zeros(B, H, N, 64, dtype=dtype, device="cuda")
    v, do = zero.clone(), zero.clone()
    v[..., 3], v[..., 17], v[..., 40] = 129, 131 / 256, 3 / 1024
    do[..., 3] = do[..., 17] = do[..., 40] = 1
    x = 129 + 131 / 256 + 3 / 1024
    t = torch.zeros(4, H, device="cuda")  # at the query; before it; none; after it
    lse = torch.zeros(B, H, N, device="cuda")
    dq, dk, dv, dt = mha.sdpa_rel_backward(zero, zero, v, t, zero, do, lse, max_distance=2)
    pairs = B * N * (N - 1) / 2
    want = np.array([B * N * x, pairs * x, 0, pairs * x])[:, None].repeat(H, 1)
    within(host(dt), want, 32 * 2.0 ** -24 * want, "dtable")
    assert torch.all(dq == 0) and torch.all(dk == 0)


@pytest.mark.parametrize("dtype,N,causal", [(BF, 4001, False), (BF, 3500, True), (F, 2500, False),
                                            (F, 2100, True)])
def test_table_gradient_of_long_sequences_bucket_by_bucket(dtype, N, causal):
    # every bucket within its own bound (table_grad_bound's, in 64 bits on the GPU), from the stored O and
    # lse; the largest gradients are far above theirs
    torch.manual_seed(N)
    q, k, v, do = (torch.randn(1, 2, N, 64, device="cuda").to(dtype) for _ in range(4))
    t = torch.randn(32, 2, device="cuda") * 1.5
    how = dict(mask="causal" if causal else "none", max_distance=128, bidirectional=not causal)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, do, lse, **how)[3].double()
    want = plain64(q, k, v, t, do, causal, 128, not causal, given=(O, lse))[5]
    q, k, v, do, O = (x.double() for x in (q, k, v, do, O))
    u = torch.tensor(ref.bucket_table(-(N - 1), N - 1, 32, 128, not causal), device="cuda")
    d = torch.arange(N, device="cuda") - torch.arange(N, device="cuda")[:, None]
    x = q @ k.transpose(2, 3) / 8 + t.double()[u[d + N - 1]].permute(2, 0, 1) - lse.double()[..., None]
    if causal:
        x = x.masked_fill(d > 0, -float("inf"))
    dP, D = do @ v.transpose(2, 3), (do * O).sum(-1, keepdim=True)
    size = do.abs() @ v.abs().transpose(2, 3) + (do * O).abs().sum(-1, keepdim=True)
    e = torch.exp(x) * (2.0 ** -15 * (dP.abs() + D.abs()) + 2.0 ** -17 * size)
    tol = torch.zeros_like(want)
    for i in range(2 * N - 1):
        tol[u[i]] += e.diagonal(i - (N - 1), 2, 3).sum((0, 2))
    within(got.cpu().numpy(), want.cpu().numpy(), (tol + 2.0 ** -24 * want.abs()).cpu().numpy(),
           "dtable")
    assert float((want.abs() / tol.clamp(min=1e-30)).max()) > 50  # (a bucket is empty)


# ------------------------------------------------------------------ scales and scores of any size
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("scale", [2.0 ** 64, 2.0 ** -64])
def test_scale_at_its_ends(dtype, scale, det_mode):
    # queries that are that much smaller or larger: ordinary scores
    B, H, N = 1, 2, 200
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 980)
    Q = Q / (8 * scale)
    q, k, v, g, t = (dev(a, dtype) for a in (Q, K, V, dO, T))
    how = dict(scale=scale)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
    rO, rl = ref.sdpa_rel_ref(Q, K, V, T, **how)
    check_lse(lse.cpu().numpy(), rl)
    want = (rO,) + ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)[:3]
    near_enough(dtype, list(zip((O,) + got[:3], want, ("O", "dQ", "dK", "dV"))), rl,
                (Q, K, V, T, dO), how, "rel scale", plain=False)
    n = i32([N])
    close(dtype)(host(mha.sdpa_rel_decode(q[:, :, :3], k, v, t, n, **how)),
                 ref.sdpa_rel_decode_ref(Q[:, :, :3], K, V, T, [N], **how), "rel decode scale")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_large_scores(dtype, mask, det_mode):
    # 2^10 times the scores that the bounds' 2^-15 of a weight goes with: 2^-5, and lse's rounding
    B, H, N, scale = 1, 2, 300, 128.0
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 982)
    q, k, v, g, t = (dev(a, dtype) for a in (Q, K, V, dO, T))
    how = dict(mask=mask, scale=scale)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
    rO, rl = ref.sdpa_rel_ref(Q, K, V, T, **how)
    want = (rO,) + ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)[:3]
    half = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    bounds = ref.element_bounds(Q, K, V, T, dO, half, 2.0 ** -5 + 2.0 ** -24 * np.abs(rl).max(), **how)
    for a, w, tol, n in zip((O,) + got[:3], want, bounds, ("O", "dQ", "dK", "dV")):
        within(host(a), w, tol, n)


@pytest.mark.parametrize("dtype,scale", [(BF, 2.0 ** 18), (F, 2.0 ** 18), (F, 2.0 ** 30), (F, 2.0 ** 64)])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_gradients_of_huge_scores_are_finite(dtype, scale, mask, det_mode):
    # scores of up to 2^24 (fp32: 2^70) and an lse as large, whose difference is mostly rounding
    B, H, N = 1, 2, 300
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 981)
    q, k, v, g, t = (dev(a, dtype) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, mask, scale=scale)
    dq, dk, dv, dt = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, mask, scale=scale)
    for x in (O, lse, dq, dk, dv, dt):
        assert torch.all(torch.isfinite(x))
    if dtype is F:  # weights of at most 1, times factors off by 2^-22, added up
        assert np.all(np.abs(host(dv)) <= np.abs(dO).sum(2, keepdims=True) * (1 + 2.0 ** -15))
