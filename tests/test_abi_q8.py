"""Refusals of the 8-bit cache's entry points, on the host: every call here fails its checks, so
nothing is launched and no GPU is needed."""
import ctypes

import pytest
import torch

from transformer_head_scaled_04_gb300 import KvCacheQ8, cache_q8, kv_cache_q8
from transformer_head_scaled_04_gb300 import _capi as C
from transformer_head_scaled_04_gb300 import build as B

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = (C.MHA_ERR_INVALID, C.MHA_ERR_UNSUPPORTED,
                                          C.MHA_ERR_ALIGN, C.MHA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def at(i):
    return ctypes.c_void_p(0x10000 + 0x1000 * i)  # never dereferenced


ODD = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x10008)


def strides(n, **changed):
    s = [4096, 1024, 64, 1] * n
    for k, v in changed.items():
        s[int(k[1:])] = v
    return ctypes.cast((ctypes.c_int64 * len(s))(*s), ctypes.c_void_p)


def append(lib, B=1, H=1, N=4, Lmax=16, dk=64, dv=64, dt=1, qt=0, block=16, new_len=None,
           cache_len=at(1), k=at(2), v=at(3), kc=at(4), vc=at(5), ks=at(6), vs=at(7), w=None,
           st=None):
    return lib.mha_kv_append_q8(B, H, N, Lmax, dk, dv, dt, qt, block, new_len, cache_len, k, v,
                                kc, vc, ks, vs, w, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Lmax=0), INVALID), (dict(dt=2), INVALID),
    (dict(qt=2), INVALID), (dict(qt=-1), INVALID), (dict(cache_len=None), INVALID),
    (dict(k=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID),
    (dict(kc=at(5)), INVALID), (dict(ks=at(7)), INVALID),      # K and V caches must differ
    (dict(dk=128), UNSUPPORTED), (dict(block=48), UNSUPPORTED), (dict(block=0), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED), (dict(Lmax=(1 << 30) + 1), UNSUPPORTED),
    (dict(k=EIGHT), ALIGN), (dict(vc=EIGHT), ALIGN), (dict(cache_len=ODD), ALIGN),
    (dict(w=ODD), ALIGN), (dict(new_len=ODD), ALIGN),
    (dict(st=strides(4, _0=-8)), INVALID), (dict(st=strides(4, _3=2)), UNSUPPORTED),
    (dict(st=strides(4, _2=68)), ALIGN), (dict(st=strides(4, _10=72)), ALIGN),
    (dict(st=strides(4, _9=0)), ALIGN), (dict(st=strides(4, _2=66), dt=0), ALIGN),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def decode(lib, B=1, H=4, Hkv=2, Nq=1, Lmax=16, dk=64, dv=64, dt=1, qt=0, block=16, causal=1,
           cache_len=at(1), scale=0.0, q=at(2), kc=at(4), vc=at(5), ks=at(6), vs=at(7), o=at(8),
           st=None, w=None, ws=at(16), n=1 << 30):
    return lib.mha_sdpa_decode_q8_fwd(B, H, Hkv, Nq, Lmax, dk, dv, dt, qt, block, causal,
                                      cache_len, scale, q, kc, vc, ks, vs, o, st, w, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=5), INVALID), (dict(Hkv=0), INVALID), (dict(Nq=0), INVALID),
    (dict(Nq=16, Lmax=15), INVALID), (dict(causal=2), INVALID), (dict(dt=5), INVALID),
    (dict(qt=3), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(vs=None), INVALID), (dict(cache_len=None), INVALID),
    (dict(dv=32), UNSUPPORTED), (dict(block=256), UNSUPPORTED), (dict(Nq=17, Lmax=99), UNSUPPORTED),
    (dict(q=EIGHT), ALIGN), (dict(kc=EIGHT), ALIGN), (dict(ks=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(st=strides(4, _13=-8)), INVALID), (dict(st=strides(4, _7=2)), UNSUPPORTED),
    (dict(st=strides(4, _6=24)), ALIGN), (dict(st=strides(4, _14=0)), ALIGN),
    (dict(ws=None, Lmax=4096), WORKSPACE), (dict(n=16, Lmax=4096), WORKSPACE),
    (dict(ws=EIGHT, Lmax=4096), ALIGN),
])
def test_decode_refusals(lib, kw, code):
    assert decode(lib, **kw) == code


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    size = lib.mha_decode_q8_workspace_size
    assert size(64, 16, 16, 1, 4096, 0, ctypes.byref(n)) == 0 and n.value % 256 == 0
    assert size(64, 16, 16, 1, 4096, 1, None) == INVALID
    assert size(64, 16, 5, 1, 4096, 1, ctypes.byref(n)) == INVALID
    assert size(64, 16, 16, 1, 4096, 2, ctypes.byref(n)) == INVALID
    assert size(64, 16, 16, 17, 4096, 1, ctypes.byref(n)) == UNSUPPORTED
    assert size(1, 256, 1, 16, 4096, 1, ctypes.byref(n)) == 0
    assert size(1, 257, 1, 16, 4096, 1, ctypes.byref(n)) == UNSUPPORTED      # rows of a head
    assert size(1, 1, 1, 1, (1 << 30) + 1, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(65535, 65535, 65535, 1, 16, 0, ctypes.byref(n)) == UNSUPPORTED  # rows of a batch
    assert size(64, 64, 64, 1, 1 << 30, 0, ctypes.byref(n)) == UNSUPPORTED   # tiles of a batch
    size = lib.mha_key_weights_workspace_size
    assert size(8, 16, 16, 4096, 4096, 1, ctypes.byref(n)) == 0 and n.value % 256 == 0
    assert size(8, 16, 16, 4096, 4096, 1, None) == INVALID
    assert size(8, 16, 3, 4096, 4096, 1, ctypes.byref(n)) == INVALID
    assert size(8, 16, 16, 4096, 4096, 2, ctypes.byref(n)) == INVALID
    assert size(65536, 1, 1, 1, 1, 1, ctypes.byref(n)) == UNSUPPORTED        # heads of a batch
    assert size(60000, 1, 1, 1, 1 << 30, 1, ctypes.byref(n)) == UNSUPPORTED  # key tiles
    assert size(1, 65535, 1, 1 << 30, 1, 0, ctypes.byref(n)) == UNSUPPORTED  # query tiles of a head


def keyw(lib, B=1, H=4, Hkv=2, Nq=8, Nk=8, dk=64, dt=1, mask=0, kl=None, ql=None, scale=0.0,
         q=at(1), k=at(2), lse=at(3), st=None, w=at(4), ld=8, ws=None, n=0):
    return lib.mha_sdpa_key_weights(B, H, Hkv, Nq, Nk, dk, dt, mask, kl, ql, scale, q, k, lse, st,
                                    w, ld, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(H=3), INVALID), (dict(Nk=0), INVALID), (dict(dt=2), INVALID),
    (dict(mask=3), INVALID), (dict(mask=1, Nq=7), INVALID), (dict(mask=2), INVALID),
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID),
    (dict(ld=7), INVALID), (dict(scale=float("nan")), INVALID), (dict(dk=32), UNSUPPORTED),
    (dict(H=70000, Hkv=70000), UNSUPPORTED), (dict(k=EIGHT), ALIGN), (dict(lse=ODD), ALIGN),
    (dict(ql=ODD), ALIGN), (dict(st=strides(2, _1=-64)), INVALID),
    (dict(st=strides(2, _7=3)), UNSUPPORTED), (dict(st=strides(2, _2=60)), ALIGN),
])
def test_key_weights_refusals(lib, kw, code):
    assert keyw(lib, **kw) == code


def evict(lib, B=1, H=1, Lmax=64, Lout=32, dk=64, dv=64, qt=0, block=16, keep=20, recent=0,
          cl=at(1), kc=at(2), vc=at(3), ks=at(4), vs=at(5), w=at(6), ko=at(7), vo=at(8),
          kso=at(9), vso=at(10), wo=at(11), n=at(12), kept=at(13), st=None):
    return lib.mha_kv_evict_q8(B, H, Lmax, Lout, dk, dv, qt, block, keep, recent, cl, kc, vc, ks,
                               vs, w, ko, vo, kso, vso, wo, n, kept, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(keep=0), INVALID), (dict(keep=33), INVALID),
    (dict(recent=-1), INVALID), (dict(qt=2), INVALID), (dict(w=None), INVALID),
    (dict(kept=None), INVALID), (dict(n=None), INVALID), (dict(ko=None), INVALID),
    (dict(ko=at(2)), INVALID), (dict(vo=at(7)), INVALID), (dict(n=at(1)), INVALID),
    (dict(wo=at(6)), INVALID), (dict(vso=at(5)), INVALID), (dict(dk=32), UNSUPPORTED),
    (dict(block=20), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
    (dict(B=65535, H=65535), UNSUPPORTED),
    (dict(vo=EIGHT), ALIGN),
    (dict(kept=ODD), ALIGN), (dict(st=strides(4, _8=-16)), INVALID),
    (dict(st=strides(4, _11=0)), UNSUPPORTED), (dict(st=strides(4, _14=8)), ALIGN),
])
def test_evict_refusals(lib, kw, code):
    assert evict(lib, **kw) == code


def test_wrappers_check_shapes_and_types():
    cpu = -1
    c = kv_cache_q8(2, 3, 50, 16, torch.int8, device="cpu")
    assert cache_q8._check_cache(c, cpu) == (2, 3, 50, C.MHA_Q8_I8)
    assert c.k_scale.shape == (2, 3, 4) and c.weights.shape == (2, 3, 50)
    assert kv_cache_q8(1, 1, 5, weights=False, device="cpu").weights is None
    for bad in (c._replace(k_scale=c.k_scale[:, :, :3]), c._replace(block=20),
                c._replace(v=c.v[:, :2]), c._replace(weights=c.weights.double()),
                c._replace(v_scale=c.v_scale.transpose(0, 1)),
                c._replace(v=c.v.view(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            cache_q8._check_cache(bad, cpu)
    with pytest.raises(TypeError):
        cache_q8._check_cache(c._replace(k=c.k.float(), v=c.v.float()), cpu)
    with pytest.raises(TypeError):
        kv_cache_q8(1, 1, 5, dtype=torch.uint8, device="cpu")
    with pytest.raises(ValueError):
        kv_cache_q8(1, 1, 5, block=8, device="cpu")
    n = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 3, 1, 64)
    for call in (lambda: cache_q8.sdpa_decode_q8(q, c, n),       # tensors on the host
                 lambda: cache_q8.kv_append_q8(c, q, q, n),
                 lambda: cache_q8.sdpa_key_weights(q, q, q[..., 0]),
                 lambda: cache_q8.kv_evict_q8(c, c, n, 5)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    assert isinstance(c, KvCacheQ8)
