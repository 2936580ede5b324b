"""Attention with a learned relative position bias at the ends of what its entry points take, against
the CPU oracle (``oracle.rel_bias``) or the formulas in 64 bits on the GPU."""
import numpy as np
import pytest
import torch

from oracle import rel_bias as ref
from parity_util import assert_f32_close
from test_gpu_rel import BF, F, dev, draw, host, i32, within

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
    if hidden == "faint" and size > 1e12:
        return  # at e^-60 it is not faint any more
    Q, K, V, dO = (np.asarray(a, np.float32).astype(np.float64) for a in (Q, K, V, dO))
    if hidden != "causal":  # keys after the query
        T[16:] = -np.inf if hidden == "excluded" else -60.0
    how = dict(mask="causal" if hidden == "causal" else "none", max_distance=128)
    q, k, v, g, t = (dev(a, F) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
    with np.errstate(invalid="ignore"):
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
    with np.errstate(invalid="ignore"):
        w = ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, given=given, **how)[3]
        tol = ref.table_grad_bound(Q, K, V, T, dO, *given, **how)
    within(host(got[3]), w, tol + 2.0 ** -24 * np.abs(w), "dtable")


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
