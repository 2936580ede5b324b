"""Refusals of the entry points of the learned relative position bias, on the host: every call here
fails its checks, so nothing is launched and no GPU is needed."""
import ctypes

import pytest
import torch

import transformer_head_scaled_04_gb300 as mha
from transformer_head_scaled_04_gb300 import _capi as C
from transformer_head_scaled_04_gb300 import build as B

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = (C.MHA_ERR_INVALID, C.MHA_ERR_UNSUPPORTED,
                                          C.MHA_ERR_ALIGN, C.MHA_ERR_WORKSPACE)
F32, BF16 = C.MHA_F32, C.MHA_BF16


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def at(i):
    return ctypes.c_void_p(0x10000 + 0x1000 * i)  # never dereferenced


ODD = ctypes.c_void_p(0x10002)
ODDER = ctypes.c_void_p(0x10001)
EIGHT = ctypes.c_void_p(0x10008)


def strides(n, **changed):
    s = [4096, 1024, 64, 1] * n
    for k, v in changed.items():
        s[int(k[1:])] = v
    return ctypes.cast((ctypes.c_int64 * len(s))(*s), ctypes.c_void_p)


BIAS = [
    (dict(bias=None), INVALID), (dict(bt=2), INVALID), (dict(nb=1), INVALID),
    (dict(nb=129), UNSUPPORTED), (dict(reach=1 << 24), UNSUPPORTED), (dict(both=2), INVALID), (dict(both=-1), INVALID),
    (dict(nb=33), INVALID), (dict(nb=2), INVALID),           # both sides: even, 4 at least
    (dict(reach=8), INVALID), (dict(reach=0), INVALID), (dict(reach=-5), INVALID),
    (dict(nb=33, both=0, reach=16), INVALID),
    (dict(bias=ODD, bt=F32), ALIGN), (dict(bias=ODDER, bt=BF16), ALIGN),
]
SIZES = [
    (dict(Bn=0), INVALID), (dict(H=0), INVALID), (dict(Nq=0), INVALID), (dict(dk=0), INVALID),
    (dict(dt=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(Bn=65536), UNSUPPORTED),
    (dict(scale=1e-20), UNSUPPORTED), (dict(scale=1e20), UNSUPPORTED),
    (dict(H=65536), UNSUPPORTED), (dict(dk=32), UNSUPPORTED), (dict(dv=128), UNSUPPORTED),
    (dict(dt=F32, dk=129), UNSUPPORTED), (dict(dt=F32, dv=129), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(q=EIGHT), ALIGN), (dict(v=EIGHT), ALIGN), (dict(dt=F32, k=ODD), ALIGN),
]
MASKS = [
    (dict(mask=3), INVALID), (dict(mask=-1), INVALID), (dict(mask=1, Nk=65), INVALID),
    (dict(mask=2), INVALID), (dict(mask=2, kl=ODD), ALIGN), (dict(Nk=0), INVALID),
    (dict(Nk=(1 << 24) + 1), UNSUPPORTED),
]


def fwd(lib, Bn=1, H=2, Nq=64, Nk=64, dk=64, dv=64, dt=BF16, mask=0, kl=None, scale=0.0, q=at(1),
        k=at(2), v=at(3), bias=at(4), bt=F32, nb=32, reach=128, both=1, o=at(5), st=None, lse=None):
    return lib.mha_sdpa_rel_fwd(Bn, H, Nq, Nk, dk, dv, dt, mask, kl, scale, q, k, v, bias, bt, nb,
                                reach, both, o, st, lse, None)


@pytest.mark.parametrize("kw,code", BIAS + SIZES + MASKS + [
    (dict(o=None), INVALID), (dict(o=EIGHT), ALIGN), (dict(lse=ODD), ALIGN),
    (dict(st=strides(4, _0=-8)), INVALID), (dict(st=strides(4, _3=2)), UNSUPPORTED),
    (dict(st=strides(4, _7=2), dt=F32), UNSUPPORTED), (dict(st=strides(4, _2=68)), ALIGN),
    (dict(st=strides(4, _9=0)), ALIGN), (dict(st=strides(4, _14=0), dt=F32), ALIGN),
])
def test_forward_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code


def bwd(lib, Bn=1, H=2, Nq=64, Nk=64, dk=64, dv=64, dt=BF16, mask=0, kl=None, scale=0.0, q=at(1),
        k=at(2), v=at(3), bias=at(4), bt=F32, nb=32, reach=128, both=1, o=at(5), do=at(6),
        lse=at(7), dq=at(8), dkk=at(9), dvv=at(10), db=at(11), st=None, ws=at(16), n=1 << 30):
    return lib.mha_sdpa_rel_bwd(Bn, H, Nq, Nk, dk, dv, dt, mask, kl, scale, q, k, v, bias, bt, nb,
                                reach, both, o, do, lse, dq, dkk, dvv, db, st, ws, n, None)


@pytest.mark.parametrize("kw,code", BIAS + SIZES + MASKS + [
    (dict(o=None), INVALID), (dict(do=None), INVALID), (dict(lse=None), INVALID),
    (dict(dq=None), INVALID), (dict(dkk=None), INVALID), (dict(dvv=None), INVALID),
    (dict(db=None), INVALID), (dict(lse=ODD), ALIGN), (dict(db=ODD), ALIGN),
    (dict(dq=EIGHT), ALIGN), (dict(st=strides(8, _19=2)), UNSUPPORTED),
    (dict(st=strides(8, _16=0)), ALIGN), (dict(st=strides(8, _22=0), dt=F32), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=EIGHT), ALIGN),
])
def test_backward_refusals(lib, kw, code):
    assert bwd(lib, **kw) == code


def decode(lib, Bn=1, H=2, Nq=1, Lmax=64, dk=64, dv=64, dt=BF16, causal=1, cl=at(12), scale=0.0,
           q=at(1), k=at(2), v=at(3), bias=at(4), bt=F32, nb=32, reach=128, both=1, o=at(5),
           st=None, ws=at(16), n=1 << 30):
    return lib.mha_sdpa_rel_decode_fwd(Bn, H, Nq, Lmax, dk, dv, dt, causal, cl, scale, q, k, v, bias,
                                       bt, nb, reach, both, o, st, ws, n, None)


@pytest.mark.parametrize("kw,code", BIAS + SIZES + [
    (dict(Lmax=0), INVALID), (dict(causal=2), INVALID), (dict(Nq=9, Lmax=8), INVALID),
    (dict(Nq=17), UNSUPPORTED), (dict(Nq=17, dt=F32), UNSUPPORTED),
    (dict(Lmax=(1 << 24) + 1), UNSUPPORTED), (dict(cl=None), INVALID), (dict(cl=ODD), ALIGN),
    (dict(o=None), INVALID), (dict(o=EIGHT), ALIGN), (dict(st=strides(4, _6=68)), ALIGN),
    (dict(st=strides(4, _11=2)), UNSUPPORTED), (dict(st=strides(4, _13=0), dt=F32), ALIGN),
    (dict(Lmax=8192, ws=None), WORKSPACE), (dict(Lmax=8192, n=16), WORKSPACE),
    (dict(Lmax=8192, ws=EIGHT), ALIGN),
])
def test_decode_refusals(lib, kw, code):
    assert decode(lib, **kw) == code


def test_sizes_and_buckets(lib):
    n = ctypes.c_size_t(0)
    size = lib.mha_sdpa_rel_bwd_workspace_size
    assert size(2, 3, 200, 300, BF16, 32, ctypes.byref(n)) == 0 and n.value % 256 == 0
    assert n.value >= 2 * 3 * (2 * (1024 + 8192 + 32768) + 3 * 32 * 4)
    assert size(2, 3, 200, 300, BF16, 32, None) == INVALID
    assert size(2, 3, 200, 300, BF16, 1, ctypes.byref(n)) == INVALID
    assert size(2, 3, 200, 300, BF16, 129, ctypes.byref(n)) == UNSUPPORTED
    assert size(2, 3, 200, (1 << 24) + 1, F32, 32, ctypes.byref(n)) == UNSUPPORTED
    size = lib.mha_sdpa_rel_decode_workspace_size
    assert size(64, 16, 1, 128, 64, 64, BF16, ctypes.byref(n)) == 0 and n.value == 0
    assert size(1, 1, 1, 8192, 64, 64, BF16, ctypes.byref(n)) == 0 and n.value > 0
    assert size(1, 1, 17, 8192, 64, 64, BF16, ctypes.byref(n)) == UNSUPPORTED
    assert size(1, 1, 1, 8192, 32, 64, BF16, ctypes.byref(n)) == UNSUPPORTED
    assert lib.mha_rel_bucket(3, 33, 128, 1) == INVALID
    assert lib.mha_rel_bucket(3, 200, 128, 0) == UNSUPPORTED
    with pytest.raises(C.MhaError):
        mha.rel_bucket(1, 32, 8)


def test_numbers_past_an_int(lib):
    assert mha.rel_bucket(2 ** 32) == mha.rel_bucket(10 ** 6) == 31
    assert mha.rel_bucket(-2 ** 32 - 3) == mha.rel_bucket(-10 ** 6) == 15
    for kw in (dict(max_distance=2 ** 32 + 128), dict(num_buckets=2 ** 32 + 32),
               dict(max_distance=-2 ** 32 + 128)):
        with pytest.raises(C.MhaError):
            mha.rel_bucket(3, **kw)


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(1, 2, 4, 64)
    t = torch.zeros(32, 2)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: mha.sdpa_rel(x, x, x, t), lambda: mha.sdpa_rel_with_lse(x, x, x, t),
                 lambda: mha.sdpa_rel_backward(x, x, x, t, x, x, x[..., 0]),
                 lambda: mha.sdpa_rel_decode(x[:, :, :1], x, x, t, n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
