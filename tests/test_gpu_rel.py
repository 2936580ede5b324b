"""Attention with a learned relative position bias: the CUDA path through the C ABI against the CPU
oracle (``oracle.rel_bias``) on the same inputs.

O and the gradients of Q, K and V are held to the bounds of attention without bias (the bias enters
the scores in fp32); the gradient of the bias to a bound on fp32 arithmetic (``table_grad_bound``)
against the formula from the same stored O and lse, and, with the bf16 rounding of O in the row term
counted, against the formula from the inputs alone."""
import numpy as np
import pytest
import torch

import seeded_inputs as si
from oracle import rel_bias as ref
from parity_util import BF16_REL_L2, assert_bf16_close, assert_f32_close, errors

pytestmark = pytest.mark.gpu

mha = pytest.importorskip("transformer_head_scaled_04_gb300")

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_head_scaled_04_gb300 import build

    build.build()
    mha.load_library()
    torch.cuda.set_device(0)
    mha.device_status()
    yield
    assert mha.device_status() == 0, "a kernel recorded a device-side error"


def dev(a, t):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)


def host(t):
    return t.float().cpu().numpy()


def i32(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def draw(B, H, Nq, Nk, dtype, seed, num=32, dk=64, dv=64, size=1.5):
    g = np.random.Generator(np.random.PCG64(seed))
    fin = si.round_bf16 if dtype is BF else (lambda a: np.asarray(a, np.float32).astype(np.float64))
    n = g.standard_normal
    Q, K, V, dO = (fin(n(s)) for s in ((B, H, Nq, dk), (B, H, Nk, dk), (B, H, Nk, dv),
                                       (B, H, Nq, dv)))
    return Q, K, V, dO, si.round_bf16(n((num, H)) * size)  # the table holds in either type


def close(dtype):
    return assert_bf16_close if dtype is BF else assert_f32_close


def within(got, want, tol, what):
    d = np.abs(np.asarray(got, np.float64) - want)
    ok = bool(np.all(d <= tol + 1e-30))  # a NaN fails
    worst = np.unravel_index(int(np.argmax(np.where(d <= tol, 0, d / (tol + 1e-30)))), d.shape)
    assert ok, f"{what}: {d[worst]:.3e} at {worst}, at most {np.broadcast_to(tol, d.shape)[worst]:.3e}"


def near_enough(dtype, pairs, rl, args, how, what, many=True, plain=True):
    """(got, want, name) of O, dQ, dK, dV: each element within its own bound, and where roundings
    average out (many pairs) 5e-3 in norm in bf16 (three of about 1.7e-3 on the way to a gradient);
    fp32 with ordinary log-sum-exps (plain) as attention without bias."""
    lse = np.abs(rl[np.isfinite(rl)]).max(initial=0.0)
    half = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    bounds = ref.element_bounds(*args, half, 2.0 ** -15 + 2.0 ** -24 * lse, **how)
    for (got, want, n), tol in zip(pairs, bounds):
        got = host(got)
        within(got, want, tol, f"{what} {n}")
        if dtype is F and plain:
            assert_f32_close(got, want, f"{what} {n}")
        if dtype is BF and many:
            rel = errors(got, want)[1]
            assert rel <= BF16_REL_L2, f"{what} {n}: relative norm {rel:.3e}"


def check_lse(got, want, atol=1e-4):
    # fp32 sums of 64 products and of the weights, and logarithms, at values up to about 20
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    f = np.isfinite(want)
    assert np.all(got[~f] == np.inf) and np.allclose(got[f], want[f], rtol=1e-6, atol=atol)


def check(B, H, Nq, Nk, mask, kl, dtype, seed, num=32, reach=128, both=True, table=F, dk=64, dv=64,
          scale=None, edit=None, what=None):
    """Forward and backward of one case; edit(Q, K, V, dO, T) changes the inputs first."""
    Q, K, V, dO, T = draw(B, H, Nq, Nk, dtype, seed, num, dk, dv)
    if scale == 1.0:
        Q = Q * (si.round_bf16(np.float64(dk) ** -0.5) if dk != 64 else 0.125)
        Q = si.round_bf16(Q) if dtype is BF else np.asarray(Q, np.float32).astype(np.float64)
    if edit is not None:
        edit(Q, K, V, dO, T)
    what = what or f"rel {B}x{H} {Nq}x{Nk} {mask} {num}/{reach}/{both}"
    how = dict(mask=mask, scale=scale, max_distance=reach, bidirectional=both)
    q, k, v, g = (dev(a, dtype) for a in (Q, K, V, dO))
    t = dev(T, table)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, key_len=i32(kl), **how)
    dq, dk_, dv_, dt = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, key_len=i32(kl), **how)
    assert dt.dtype is table and dt.shape == t.shape
    rO, rl = ref.sdpa_rel_ref(Q, K, V, T, key_len=kl, **how)
    rq, rk, rv, rt = ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, key_len=kl, **how)
    check_lse(lse.cpu().numpy(), rl)
    assert torch.equal(mha.sdpa_rel(q, k, v, t, key_len=i32(kl), **how), O)
    pairs = [(O, rO, "O"), (dq, rq, "dQ"), (dk_, rk, "dK"), (dv_, rv, "dV")]
    near_enough(dtype, pairs, rl, (Q, K, V, T, dO), dict(how, key_len=kl), what,
                min(Nq, Nk) >= 32, edit is None)
    # the table's gradient, from the stored forward
    given = (host(O), lse.cpu().numpy())
    want = ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, key_len=kl, given=given, **how)[3]
    tol = ref.table_grad_bound(Q, K, V, T, dO, *given, key_len=kl, **how)
    got = host(dt).astype(np.float64)
    half = 2.0 ** -8 if table is BF else 2.0 ** -24
    within(got, want, tol + half * np.abs(want), f"{what} dtable")
    # and from the inputs alone: O's own rounding moves a row's term by half a step of |dO| |O|
    eps = 2.0 ** -8 if dtype is BF else 2.0 ** -22
    row = (np.abs(dO) * np.abs(rO)).sum(-1).sum((0, 2))  # [H], every weight at most 1
    within(got, rt, tol + half * np.abs(rt) + eps * row, f"{what} dtable from the inputs")
    assert np.all(got[tol == 0] == 0)  # buckets without pairs
    return O, lse, dq, dk_, dv_, dt


CASES = [  # B, H, Nq, Nk, mask, key_len, num, reach, both, table
    (1, 2, 1, 1, "none", None, 32, 128, True, F),
    (1, 1, 2, 3, "none", None, 4, 3, True, F),
    (2, 3, 37, 37, "none", None, 32, 128, True, BF),
    (1, 2, 128, 128, "causal", None, 32, 128, False, F),
    (2, 2, 300, 300, "causal", None, 32, 128, True, BF),
    (1, 2, 640, 640, "none", None, 32, 64, True, F),       # far tiles on both sides
    (1, 1, 900, 900, "causal", None, 32, 128, False, F),   # far tiles on one side
    (2, 2, 333, 333, "none", None, 128, 300, True, F),
    (1, 2, 520, 520, "none", None, 64, 4096, False, F),    # no tile within one segment but bucket 0
    (3, 1, 200, 390, "key_padding", [0, 1, 390], 32, 128, True, F),
    (3, 2, 257, 257, "key_padding", [256, 129, 3], 16, 50, False, BF),
    (2, 1, 100, 900, "none", None, 32, 128, True, F),      # more keys than queries
    (2, 1, 700, 65, "none", None, 32, 128, True, F),       # more queries than keys
    (1, 2, 513, 513, "none", None, 2, 2, False, F),        # one border: "at the query", "before it"
    (1, 1, 2300, 2300, "none", None, 32, 128, True, F),    # far sums over more than 16 tiles
]


@pytest.fixture(params=[False, True], ids=["fused_dq", "deterministic"])
def det_mode(request):
    before = mha.get_deterministic()
    mha.set_deterministic(request.param)
    yield request.param
    mha.set_deterministic(before)


@pytest.mark.parametrize("B,H,Nq,Nk,mask,kl,num,reach,both,table", CASES)
def test_bf16(B, H, Nq, Nk, mask, kl, num, reach, both, table, det_mode):
    check(B, H, Nq, Nk, mask, kl, BF, 700 + Nq + Nk, num, reach, both, table)


@pytest.mark.parametrize("B,H,Nq,Nk,mask,kl,num,reach,both,table", CASES[:-1])
def test_f32(B, H, Nq, Nk, mask, kl, num, reach, both, table):
    check(B, H, Nq, Nk, mask, kl, F, 800 + Nq + Nk, num, reach, both, table)


@pytest.mark.parametrize("dk,dv", [(1, 1), (17, 17), (32, 64), (40, 24), (65, 3), (100, 128),
                                   (128, 128), (63, 126)])
@pytest.mark.parametrize("mask", ["causal", "key_padding"])
def test_f32_head_sizes(dk, dv, mask):
    check(2, 2, 150, 150, mask, [150, 71] if mask == "key_padding" else None, F, dk * 7 + dv, 32,
          40, mask != "causal", dk=dk, dv=dv)


@pytest.mark.parametrize("dtype", [BF, F])
def test_scale_one(dtype):
    check(2, 2, 200, 200, "none", None, dtype, 901, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F])
def test_large_bias_far_away(dtype):
    # the largest scores come after many small ones: the running reference has to move
    def edit(Q, K, V, dO, T):
        T[31] = 180.0  # far keys after the query
        T[15] = -90.0

    check(1, 2, 500, 500, "none", None, dtype, 902, edit=edit)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("low", [-np.inf, -1e38, -1e9])
def test_excluded_buckets(dtype, low):
    # head 0: keys before the query are out, so a row's first tiles hold nothing; head 1: the query
    # itself and the keys after it are out, so row 0 holds nothing at all; head 2: all are out
    B, H, N = 2, 3, 300
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 903)
    Q, dO = 4 * Q, dO
    T[:, 0] -= 100.0  # and what is left lies far below 1
    T[1:16, 0] = low
    T[0, 1] = low
    T[16:, 1] = low
    T[:, 2] = low
    how = dict(max_distance=128, bidirectional=True)
    q, k, v, g = (dev(a, dtype) for a in (Q, K, V, dO))
    t = dev(np.maximum(T, -3.4e38) if low > -np.inf else T, F)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    Tr = np.where(T < -1e6, -np.inf, T)
    with np.errstate(invalid="ignore"):
        rO, rl = ref.sdpa_rel_ref(Q, K, V, Tr, **how)
    check_lse(lse.cpu().numpy(), rl, atol=1e-3)
    assert np.all(np.isinf(rl[:, 2])) and np.all(np.isinf(rl[:, 1, 0]))
    assert torch.all(O[:, 2] == 0) and torch.all(O[:, 1, 0] == 0)
    for det in (False, True):
        mha.set_deterministic(det)
        dq, dk, dv, dt = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)
        mha.set_deterministic(False)
        for x in (dq, dk, dv, dt):
            assert torch.all(torch.isfinite(x))
        assert torch.all(dt[t < -1e6] == 0) and torch.all(dq[:, 2] == 0) and torch.all(dv[:, 2] == 0)
        with np.errstate(invalid="ignore"):
            rq, rk, rv, _ = ref.sdpa_rel_bwd_ref(Q, K, V, Tr, dO, **how)
            near_enough(dtype, [(O, rO, "O"), (dq, rq, "dQ"), (dk, rk, "dK"), (dv, rv, "dV")], rl,
                        (Q, K, V, Tr, dO), how, "rel excluded", plain=False)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("bad", [np.nan, np.inf, 3e38])
def test_anything_in_padding(dtype, bad, det_mode):
    B, H, N = 3, 2, 300
    kl = [140, 0, 256]
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 904)
    how = dict(mask="key_padding", max_distance=128)
    clean = [dev(a, dtype) for a in (Q, K, V)]
    g, t = dev(dO, dtype), dev(T, F)
    dirty = [x.clone() for x in clean]
    for b, n in enumerate(kl):
        dirty[1][b, :, n:] = bad
        dirty[2][b, :, n:] = -bad
    outs = []
    for q, k, v in (clean, dirty):
        O, lse = mha.sdpa_rel_with_lse(q, k, v, t, key_len=i32(kl), **how)
        outs.append((O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, g, lse, key_len=i32(kl), **how))
    for n, (a, b) in enumerate(zip(*outs)):
        if n == 2 and dtype is BF and not det_mode:  # dQ's sums come in any order
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=1e-3)
        else:
            assert torch.equal(a, b), n
    O, lse, dq, dk, dv, dt = outs[1]
    for b, n in enumerate(kl):
        assert torch.all(dk[b, :, n:] == 0) and torch.all(dv[b, :, n:] == 0)
    assert torch.all(O[1] == 0) and torch.all(lse[1] == np.inf) and torch.all(dq[1] == 0)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_keys_to_come_may_hold_anything(dtype, bad):
    # under the causal mask: queries before the key keep their results, to the bit where none after it
    # shares their warp (a raised reference of the exponentials takes the warp's other rows along)
    B, H, N, j = 2, 2, 300, 137
    Q, K, V, _, T = draw(B, H, N, N, dtype, 907)
    K[:, :, j] = 0.0  # so that the row leaves the others' scales as they are
    q, k, v, t = dev(Q, dtype), dev(K, dtype), dev(V, dtype), dev(T, F)
    want = mha.sdpa_rel_with_lse(q, k, v, t, mask="causal")
    k[:, :, j] = bad
    got = mha.sdpa_rel_with_lse(q, k, v, t, mask="causal")
    for a, b in zip(want, got):
        assert torch.equal(a[:, :, :128], b[:, :, :128])
    # weights and outputs rounded to bf16 in both (each half a step of at most max |V|); fp32: 2^-22 of
    # a term, exponentials 2^-21
    tol = (4 * 2.0 ** -8 if dtype is BF else 2.0 ** -18) * float(v.abs().max())
    assert float((want[0] - got[0])[:, :, :j].abs().max()) <= tol
    assert float((want[1] - got[1])[:, :, :j].abs().max()) <= 1e-5  # logarithms of about 10
    if not bad == bad:
        assert torch.all(torch.isnan(got[0][:, :, j:]))
    # and in a step of several queries
    n, Nq = i32([N, 140]), 5
    step = [mha.sdpa_rel_decode(q[:, :, :Nq].contiguous(), c, v, t, n) for c in (dev(K, dtype), k)]
    assert float((step[0] - step[1])[1, :, :2].abs().max()) <= tol  # positions 135 and 136


def test_reproducible_and_determinism_switch(det_mode):
    Q, K, V, dO, T = draw(2, 3, 700, 700, BF, 905)
    q, k, v, g, t = (dev(a, BF) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    runs = [mha.sdpa_rel_backward(q, k, v, t, O, g, lse) for _ in range(5)]
    for r in runs[1:]:
        for i, (a, b) in enumerate(zip(runs[0], r)):
            if i > 0 or det_mode:
                assert torch.equal(a, b), i


def test_zero_table_is_plain_attention():
    Q, K, V, dO, T = draw(2, 2, 400, 400, BF, 906)
    q, k, v, g, t = (dev(a, BF) for a in (Q, K, V, dO, 0 * T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, "causal")
    O0, lse0 = mha.sdpa_with_lse(q, k, v, "causal")
    assert torch.allclose(O.float(), O0.float(), rtol=2.0 ** -7, atol=1e-3)
    assert torch.allclose(lse, lse0, rtol=0, atol=1e-5)


@pytest.mark.parametrize("dtype", [BF, F])
def test_packed_projection_layout(dtype):
    # Q|K|V inside one [B, N, 3, H, 64] buffer, O and dO as [B, N, H*64]
    B, H, N = 2, 4, 260
    g = np.random.Generator(np.random.PCG64(907))
    fin = si.round_bf16 if dtype is BF else (lambda a: np.asarray(a, np.float32))
    buf, dOb = fin(g.standard_normal((B, N, 3, H, 64))), fin(g.standard_normal((B, N, H * 64)))
    T = si.round_bf16(g.standard_normal((32, H)))
    tb, t = dev(buf, dtype), dev(T, F)
    q, k, v = (tb[:, :, i].permute(0, 2, 1, 3) for i in range(3))
    do = dev(dOb, dtype).view(B, N, H, 64).permute(0, 2, 1, 3)
    out = torch.full((B, N, H * 64 + 8), 7.0, dtype=dtype, device="cuda")
    view = out.as_strided((B, H, N, 64), (N * (H * 64 + 8), 64, H * 64 + 8, 1))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, "causal", bidirectional=False, out=view)
    assert O.data_ptr() == out.data_ptr() and torch.all(out[..., H * 64:] == 7)
    dq, dk, dv, dt = mha.sdpa_rel_backward(q, k, v, t, O, do, lse, "causal", bidirectional=False)
    Q, K, V = (np.moveaxis(np.asarray(buf[:, :, i], np.float64), 1, 2) for i in range(3))
    dO = np.moveaxis(np.asarray(dOb, np.float64).reshape(B, N, H, 64), 1, 2)
    how = dict(mask="causal", bidirectional=False)
    rO, rl = ref.sdpa_rel_ref(Q, K, V, T, **how)
    want = (rO,) + ref.sdpa_rel_bwd_ref(Q, K, V, T, dO, **how)[:3]
    near_enough(dtype, list(zip((O, dq, dk, dv), want, ("O", "dQ", "dK", "dV"))), rl,
                (Q, K, V, T, dO), how, "rel packed")
    same = mha.sdpa_rel_backward(*(x.contiguous() for x in (q, k, v)), t, O.contiguous(),
                                 do.contiguous(), lse, "causal", bidirectional=False)
    assert torch.equal(same[3], dt) and torch.equal(same[1], dk)


def test_fp32_rows_of_odd_strides_and_addresses():
    # rows 67 floats apart that start at an odd float: no 16-byte access fits
    B, H, N, d = 2, 3, 130, 40
    Q, K, V, dO, T = draw(B, H, N, N, F, 908, dk=d, dv=d)

    def odd(a):
        x = torch.zeros(B * H * N * 67 + 1, device="cuda")
        y = x[1:].as_strided((B, H, N, d), (H * N * 67, N * 67, 67, 1), 1)
        return y.copy_(dev(a, F))

    t = dev(T, F)
    args = [dev(a, F) for a in (Q, K, V)]
    O, lse = mha.sdpa_rel_with_lse(*args, t, "causal")
    O2, lse2 = mha.sdpa_rel_with_lse(*(odd(a) for a in (Q, K, V)), t, "causal")
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    a = mha.sdpa_rel_backward(*args, t, O, dev(dO, F), lse, "causal")
    b = mha.sdpa_rel_backward(*(odd(x) for x in (Q, K, V)), t, odd(host(O)), odd(dO), lse, "causal")
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    n = torch.tensor([130, 77], dtype=torch.int32, device="cuda")
    a = mha.sdpa_rel_decode(args[0][:, :, :3].contiguous(), args[1], args[2], t, n)
    b = mha.sdpa_rel_decode(odd(Q)[:, :, :3], odd(K), odd(V), t, n)
    assert torch.equal(a, b)


def test_fp32_keys_that_heads_share():
    # inputs may have a head stride of 0; gradients come per head
    B, H, N = 2, 4, 150
    Q, K, V, dO, T = draw(B, H, N, N, F, 909)
    q, g, t = dev(Q, F), dev(dO, F), dev(T, F)
    k, v = (dev(a[:, :1], F).expand(B, H, N, 64) for a in (K, V))
    assert k.stride(1) == 0
    runs = []
    for kk, vv in ((k, v), (k.contiguous(), v.contiguous())):
        O, lse = mha.sdpa_rel_with_lse(q, kk, vv, t, "causal")
        runs.append((O, lse) + mha.sdpa_rel_backward(q, kk, vv, t, O, g, lse, "causal") +
                    (mha.sdpa_rel_decode(q[:, :, :2], kk, vv, t, i32([150, 33])),))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F])
def test_two_backwards_at_once(dtype, det_mode):
    # on two streams, a workspace each
    B, H, N = 4, 4, 700
    Q, K, V, dO, T = draw(B, H, N, N, dtype, 943)
    q, k, v, g = (dev(a, dtype) for a in (Q, K, V, dO))
    t = dev(T, F)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, "causal")
    want = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, "causal")
    n = mha.sdpa_rel_bwd_workspace_size(B, H, N, N, dtype, 32)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mha.sdpa_rel_backward(q, k, v, t, O, g, lse, "causal",
                                                    workspace=ws[i]))
    torch.cuda.synchronize()
    for run in got[0] + got[1]:
        for i, (a, b) in enumerate(zip(run, want)):
            if i == 0 and dtype is BF and not det_mode:  # dQ's sums come in any order
                assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=1e-3)
            else:
                assert torch.equal(a, b)


def test_gradient_of_the_table_against_differences():
    # a loss sum(O dO) in fp32, differences of the fp32 forward in single buckets
    Q, K, V, dO, T = draw(2, 2, 120, 120, F, 909, num=8)
    q, k, v, g = (dev(a, F) for a in (Q, K, V, dO))
    t = dev(T, F)
    how = dict(mask="causal", max_distance=30, bidirectional=False)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    dt = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, **how)[3]
    h = 2.0 ** -6
    for u in range(8):
        up, down = t.clone(), t.clone()
        up[u, 1] += h
        down[u, 1] -= h
        diff = ((mha.sdpa_rel(q, k, v, up, **how).double()
                 - mha.sdpa_rel(q, k, v, down, **how).double()) * g.double())[:, 1].sum() / (2 * h)
        # a weight's third derivative in a bias is at most 6 times the weight (h^2 / 6 of it in the
        # difference); fp32 values of O are off by 2^-22 of themselves at most
        size = (O.double().abs() * g.double().abs())[:, 1].sum()
        tol = float(size) * (h * h + 2.0 ** -22 / h)
        assert abs(float(diff - dt[u, 1])) <= tol


def plain64(q, k, v, t, do, causal, reach, both, given=None):
    """(O, lse, dQ, dK, dV, dtable) in float64 on the GPU, elementary operations only."""
    q, k, v, t, do = (x.double() for x in (q, k, v, t, do))
    N, M = q.shape[2], k.shape[2]
    lo = -(N - 1)
    u = torch.tensor(ref.bucket_table(lo, M - 1, t.shape[0], reach, both), device="cuda")
    d = torch.arange(M, device="cuda") - torch.arange(N, device="cuda")[:, None]
    s = q.shape[3] ** -0.5
    x = q @ k.transpose(2, 3) * s + t[u[d - lo]].permute(2, 0, 1)
    if causal:
        x = x.masked_fill(d > 0, -float("inf"))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    del x
    O = p @ v
    base, weights = (O, p) if given is None else (given[0].double(), None)
    if weights is None:
        weights = p * torch.exp(lse - given[1].double())[..., None]
    dS = weights * (do @ v.transpose(2, 3) - (do * base).sum(-1, keepdim=True))
    dt = torch.zeros_like(t)
    for e in range(M + N - 1):
        dt[u[e]] += dS.diagonal(lo + e, 2, 3).sum((0, 2))
    return O, lse, s * dS @ k, s * dS.transpose(2, 3) @ q, weights.transpose(2, 3) @ do, dt


@pytest.mark.parametrize("dtype,N,causal", [(BF, 6001, False), (BF, 5000, True), (F, 2500, False)])
def test_long_sequences(dtype, N, causal):
    # hundreds of tiles per row: relative norms against 64 bits, the table's gradient element by element
    torch.manual_seed(N)
    q, k, v, do = (torch.randn(1, 2, N, 64, device="cuda").to(dtype) for _ in range(4))
    t = torch.randn(32, 2, device="cuda") * 1.5
    how = dict(mask="causal" if causal else "none", max_distance=128, bidirectional=not causal)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = (O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, do, lse, **how)
    want = plain64(q, k, v, t, do, causal, 128, not causal, given=(O, lse))
    most = BF16_REL_L2 if dtype is BF else 1e-5
    for i, (a, b) in enumerate(zip(got[:5], want[:5])):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= (1e-6 if i == 1 else most), (i, rel)
    # a sum of N N / 2 terms p (dP - D): fp32 arithmetic is off by 2^-15 of a weight's term (its
    # exponent's roundings), of random sign over the N rows, whose own weights sum to 1 at most
    size = float((do.double() ** 2).sum(-1).mean() ** 0.5) * 8 ** 0.5  # of dP, per row
    tol = 2.0 ** -15 * size * N ** 0.5 * 4
    assert float((got[5].double() - want[5]).abs().max()) <= tol


@pytest.mark.parametrize("dtype", [BF, F])
def test_many_short_sequences(dtype):
    B, H, N = 3000, 8, 5
    torch.manual_seed(1)
    q, k, v, do = (torch.randn(B, H, N, 64, device="cuda").to(dtype) for _ in range(4))
    t = torch.randn(8, H, device="cuda")
    how = dict(mask="causal", max_distance=20, bidirectional=False)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t, **how)
    got = (O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, do, lse, **how)
    want = plain64(q, k, v, t, do, True, 20, False, given=(O, lse))
    for i, (a, b) in enumerate(zip(got, want)):
        rel = float((a.double() - b).norm() / b.norm())
        # O, and gradients of a handful of terms each: at most two roundings of 2^-8, on average less
        assert rel <= (1e-6 if i == 1 else 2.0 ** -7 if dtype is BF and i < 5 else 1e-5), (i, rel)
    n = torch.randint(0, N + 1, (B,), device="cuda").to(torch.int32)
    a = mha.sdpa_rel_decode(q[:, :, :1], k, v, t, n, max_distance=20)
    for b in (0, 1, 777, B - 1):
        L = int(n[b])
        want = ref.sdpa_rel_decode_ref(*(host(x[b:b + 1]) for x in (q[:, :, :1], k, v)), host(t), [L],
                                       max_distance=20)
        close(dtype)(host(a[b:b + 1]), want, "rel decode of many")


def test_fp32_is_reproducible():
    Q, K, V, dO, T = draw(2, 3, 500, 500, F, 911)
    q, k, v, g, t = (dev(a, F) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    runs = [(O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, g, lse)]
    for _ in range(3):
        O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
        runs.append((O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, g, lse))
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12])
def test_fp32_values_of_any_size(size):
    # operands are scaled tile by tile: V and dO of any size, and rows of very different sizes, keep
    # fp32's relative accuracy
    Q, K, V, dO, T = draw(1, 2, 200, 200, F, 912)
    V = np.asarray(V * size, np.float32).astype(np.float64)
    g = np.random.Generator(np.random.PCG64(5))
    dO = np.asarray(dO * 10.0 ** g.integers(-6, 7, (1, 2, 200, 1)), np.float32).astype(np.float64)
    q, k, v, do, t = (dev(a, F) for a in (Q, K, V, dO, T))
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    rO, _ = ref.sdpa_rel_ref(Q, K, V, T)
    assert errors(O.double().cpu().numpy() / size, rO / size)[1] <= 1e-6
    dq, dk, dv, dt = mha.sdpa_rel_backward(q, k, v, t, O, do, lse)
    for a, b in zip((dq, dk, dv, dt), ref.sdpa_rel_bwd_ref(Q, K, V, T, dO)):
        unit = np.abs(b).max()
        assert errors(a.double().cpu().numpy() / unit, b / unit)[1] <= 1e-5
    # every row of dQ goes by its own row of dO: rows a million times smaller than their neighbours
    # are exact to 2^-22 of the tile's largest operand times their own
    want = ref.sdpa_rel_bwd_ref(Q, K, V, T, dO)[0]
    row = np.linalg.norm(dq.double().cpu().numpy() - want, axis=-1) / np.linalg.norm(want, axis=-1)
    assert row.max() <= 1e-4


# ------------------------------------------------------------------ generation step
def check_decode(B, H, Nq, Lmax, lens, dtype, causal=True, num=32, reach=128, both=False, table=F,
                 dk=64, dv=64, seed=0, poison=True, scale=None):
    Q, K, V, _, T = draw(B, H, Nq, Lmax, dtype, 1000 + seed + Lmax, num, dk, dv)
    q, k, v, t = dev(Q, dtype), dev(K, dtype), dev(V, dtype), dev(T, table)
    if poison:
        for b, n in enumerate(lens):
            k[b, :, max(n, 0):] = float("nan")
            v[b, :, max(n, 0):] = float("inf")
    O = mha.sdpa_rel_decode(q, k, v, t, i32(lens), causal=causal, max_distance=reach,
                            bidirectional=both, scale=scale)
    rO = ref.sdpa_rel_decode_ref(Q, K, V, T, lens, causal, scale, reach, both)
    close(dtype)(host(O), rO, f"rel decode {B}x{H} {Nq} of {Lmax}")
    return O


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("Nq", [1, 2, 5, 8, 9, 16])
@pytest.mark.parametrize("causal", [True, False])
def test_decode_lengths(dtype, Nq, causal):
    lens = [0, 1, Nq - 1, Nq, 15, 16, 17, 31, 63, 64, 65, 100]
    check_decode(len(lens), 3, Nq, 100, lens, dtype, causal, seed=Nq)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("num,reach,both,table", [(32, 128, False, F), (32, 1000, True, BF),
                                                  (128, 4096, False, F), (4, 3, True, F)])
def test_decode_long(dtype, num, reach, both, table):
    check_decode(2, 2, 3, 5000, [5000, 3777], dtype, True, num, reach, both, table, seed=num)


@pytest.mark.parametrize("dk,dv", [(1, 1), (17, 40), (64, 32), (96, 128), (128, 65), (126, 3)])
def test_decode_f32_head_sizes(dk, dv):
    check_decode(2, 2, 4, 900, [900, 333], F, dk=dk, dv=dv, seed=dk)


def test_decode_lengths_out_of_range_are_clamped():
    Q, K, V, _, T = draw(3, 2, 2, 50, BF, 920)
    q, k, v, t = (dev(a, BF) for a in (Q, K, V, T))
    a = mha.sdpa_rel_decode(q, k, v, t, i32([-3, 51, 2**31 - 1]))
    b = mha.sdpa_rel_decode(q, k, v, t, i32([0, 50, 50]))
    assert torch.equal(a, b) and torch.all(a[0] == 0)


def test_decode_strided_cache():
    # a cache kept as [B, Lmax, H, 64], queries inside a packed projection
    B, H, Lmax = 3, 5, 400
    Q, K, V, _, T = draw(B, H, 4, Lmax, BF, 921)
    t = dev(T, F)
    q, k, v = (dev(np.moveaxis(a, 1, 2), BF).permute(0, 2, 1, 3) for a in (Q, K, V))
    n = i32([400, 1, 200])
    assert not k.is_contiguous()
    a = mha.sdpa_rel_decode(q, k, v, t, n)
    b = mha.sdpa_rel_decode(*(x.contiguous() for x in (q, k, v)), t, n)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F])
def test_generation_follows_the_prompt(dtype):
    # as used: a prompt's forward, then steps of one and of several tokens against the cache give the
    # rows of the whole causal forward
    B, H, N, P = 2, 4, 200, 150
    Q, K, V, _, T = draw(B, H, N, N, dtype, 930)
    q, k, v, t = (dev(a, dtype) for a in (Q, K, V, T))
    how = dict(max_distance=64, bidirectional=False)
    whole = mha.sdpa_rel(q, k, v, t, "causal", **how)
    kc = torch.full((B, H, N + 30, 64), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    kc[:, :, :P], vc[:, :, :P] = k[:, :, :P], v[:, :, :P]
    first = mha.sdpa_rel(*(x[:, :, :P].contiguous() for x in (q, k, v)), t, "causal", **how)
    tol = dict(rtol=2.0 ** -7, atol=2e-2) if dtype is BF else dict(rtol=1e-5, atol=1e-5)
    assert torch.allclose(first.float(), whole[:, :, :P].float(), **tol)
    at = P
    for step in (1, 1, 4, 16, 1, 16, 11):
        new = slice(at, at + step)
        kc[:, :, new], vc[:, :, new] = k[:, :, new], v[:, :, new]
        at += step
        got = mha.sdpa_rel_decode(q[:, :, new], kc, vc, t, i32([at] * B), **how)
        assert torch.allclose(got.float(), whole[:, :, new].float(), **tol)
    assert at == N


def test_training_step_together():
    # as used: projections, attention with the bias, its backward, the bias updated
    B, N, H = 2, 96, 2
    g = np.random.Generator(np.random.PCG64(931))
    x = dev(g.standard_normal((B * N, 128)), F)
    W = dev(g.standard_normal((3 * H * 64, 128)) * 0.1, F)
    qkv = mha.linear(x, W).view(B, N, 3, H, 64)
    q, k, v = (qkv[:, :, i].permute(0, 2, 1, 3) for i in range(3))
    t = torch.zeros(32, H, device="cuda")
    target = dev(g.standard_normal((B, H, N, 64)), F)

    def loss_of(t):
        return 0.5 * ((mha.sdpa_rel(q, k, v, t).double() - target.double()) ** 2).sum()

    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    dt = mha.sdpa_rel_backward(q, k, v, t, O, O - target, lse)[3]
    # along the gradient the loss changes by |dt|^2 per unit; a bias moves by 0.05 at most, so terms
    # of third order are below 0.05^2 of the slope's parts
    h = 0.05 / float(dt.abs().max())
    want = float((dt.double() ** 2).sum())
    slope = float(loss_of(t + h * dt) - loss_of(t - h * dt)) / (2 * h)
    assert abs(slope - want) <= 0.02 * want


# ------------------------------------------------------------------ streams, graphs, memory
def test_captured_step_replayed_with_other_lengths():
    B, H, Lmax = 4, 3, 3000
    Q, K, V, _, T = draw(B, H, 2, Lmax, BF, 940)
    q, k, v = (dev(a, BF) for a in (Q, K, V))
    t = dev(T, F)
    n = i32([5, 3000, 1, 800])
    ws = [torch.empty(mha.sdpa_rel_decode_workspace_size(B, H, 2, Lmax, 64, 64, BF),
                      dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty_like(q) for _ in range(2)]
    mha.sdpa_rel_decode(q, k, v, t, n, workspace=ws[0], out=out[0])
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            mha.sdpa_rel_decode(q, k, v, t, n, workspace=ws[i], out=out[i])
        graphs.append(gr)
    for lens in ([5, 3000, 1, 800], [0, 17, 2999, 64], [3000] * 4):
        n.copy_(i32(lens))
        t.normal_()
        s = [torch.cuda.Stream() for _ in range(2)]
        for i in range(2):
            s[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        want = mha.sdpa_rel_decode(q, k, v, t, n)
        assert torch.equal(out[0], want) and torch.equal(out[1], want)


@pytest.mark.parametrize("dtype", [BF, F])
def test_captured_training_pass(dtype):
    Q, K, V, dO, T = draw(2, 2, 300, 300, dtype, 941)
    q, k, v, g = (dev(a, dtype) for a in (Q, K, V, dO))
    t, kl = dev(T, F), i32([300, 100])
    mha.set_deterministic(True)
    try:
        def both():
            O, lse = mha.sdpa_rel_with_lse(q, k, v, t, "key_padding", kl)
            return (O, lse) + mha.sdpa_rel_backward(q, k, v, t, O, g, lse, "key_padding", kl)

        both()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = both()
        for lens in ([300, 100], [0, 299]):
            kl.copy_(i32(lens))
            q.normal_()
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, both()):
                assert torch.equal(a, b)
    finally:
        mha.set_deterministic(False)


def test_side_stream():
    Q, K, V, dO, T = draw(2, 2, 500, 500, BF, 942)
    s = torch.cuda.Stream()
    q, k, v, g = (dev(a, BF) for a in (Q, K, V, dO))
    t = dev(T, F)
    want = mha.sdpa_rel(q, k, v, t)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        t2 = torch.zeros_like(t)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-3
        t2.copy_(t)  # the table is ready only behind the products
        got = mha.sdpa_rel(q, k, v, t2)
    s.synchronize()
    assert torch.equal(got, want)


def test_workspace_is_enough_and_nothing_else_is_written():
    B, H, N = 2, 2, 300
    Q, K, V, dO, T = draw(B, H, N, N, BF, 943)
    q, k, v, g = (dev(a, BF) for a in (Q, K, V, dO))
    t = dev(T, F)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    need = mha.sdpa_rel_bwd_workspace_size(B, H, N, N, BF, 32)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    a = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, workspace=ws[:need])
    assert torch.all(ws[need:] == 0xA5)
    ws[:need] = 0xFF  # NaNs
    b = mha.sdpa_rel_backward(q, k, v, t, O, g, lse, workspace=ws[:need])
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x, y)
    need = mha.sdpa_rel_decode_workspace_size(B, H, 2, 3000, 64, 64, BF)
    kc = torch.randn(B, H, 3000, 64, device="cuda", dtype=BF)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    x = mha.sdpa_rel_decode(q[:, :, :2], kc, kc, t, i32([3000, 10]), workspace=ws[:need])
    y = mha.sdpa_rel_decode(q[:, :, :2], kc, kc, t, i32([3000, 10]))
    assert torch.all(ws[need:] == 0xFF) and torch.equal(x, y)


def test_caches_past_32_bits():
    # heads 2^31 elements apart: the last one's offset does not fit 32 bits
    H, L, far = 2, 600, 2**31 + 64
    base = torch.empty(far + L * 64, dtype=BF, device="cuda")
    k = base.as_strided((1, H, L, 64), (2 * far, far, 64, 1))
    k.copy_(torch.randn(1, H, L, 64, device="cuda"))
    v = k
    q = torch.randn(1, H, 3, 64, device="cuda").to(BF)
    t = torch.randn(32, H, device="cuda")
    kc = k.contiguous()
    a = mha.sdpa_rel_decode(q, k, v, t, i32([L]))
    assert torch.equal(a, mha.sdpa_rel_decode(q, kc, kc, t, i32([L])))
    q = torch.randn(1, H, L, 64, device="cuda").to(BF)
    O, lse = mha.sdpa_rel_with_lse(q, k, v, t)
    O2, lse2 = mha.sdpa_rel_with_lse(q, kc, kc, t)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    a = mha.sdpa_rel_backward(q, k, v, t, O, O, lse)
    b = mha.sdpa_rel_backward(q, kc, kc, t, O, O, lse)
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x, y)


def test_wrapper_refusals():
    q = torch.zeros(1, 2, 4, 64, dtype=BF, device="cuda")
    t = torch.zeros(32, 2, device="cuda")
    n = i32([4])
    lse = torch.zeros(1, 2, 4, device="cuda")
    for bad in (lambda: mha.sdpa_rel(q, q[:, :1], q, t), lambda: mha.sdpa_rel(q, q, q.float(), t),
                lambda: mha.sdpa_rel(q, q, q, t[:, :1]), lambda: mha.sdpa_rel(q, q, q, t.t()),
                lambda: mha.sdpa_rel(q, q, q, t.cpu()),
                lambda: mha.sdpa_rel(q, q, q, t, "key_padding", n.long()),
                lambda: mha.sdpa_rel(q, q, q, t, out=q.float()),
                lambda: mha.sdpa_rel_backward(q, q, q, t, q, q[:, :, :3], lse),
                lambda: mha.sdpa_rel_backward(q, q, q, t, q, q, lse[..., :3]),
                lambda: mha.sdpa_rel_decode(q[:, :, :1], q, q, t, i32([4, 4])),
                lambda: mha.sdpa_rel_decode(q[:, :, :1], q, q, t, n, workspace=lse)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mha.sdpa_rel(q.half(), q.half(), q.half(), t)
    for bad in (lambda: mha.sdpa_rel(q, q, q, t, "key_padding"),
                lambda: mha.sdpa_rel(q, q, q, t, max_distance=8),
                lambda: mha.sdpa_rel(q, q, q, t[:31].contiguous()),
                lambda: mha.sdpa_rel(q, q[:, :, :3], q[:, :, :3], t, "causal"),
                lambda: mha.sdpa_rel_decode(q, q[:, :, :2], q[:, :, :2], t, n)):
        with pytest.raises(mha.MhaError):
            bad()
