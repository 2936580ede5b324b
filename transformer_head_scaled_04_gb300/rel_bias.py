"""torch-facing wrappers of attention with a learned relative position bias (argument checks and
marshalling only, as in ``api``): the forward, its backward with the gradient of the bias, and the
generation step against a key/value cache.

Every call takes ``rel_bias`` [num_buckets, H] (fp32 or bf16, like the weight of an embedding over
the buckets), ``max_distance`` and ``bidirectional``; ``rel_bucket`` says which bucket a distance
(the key's position minus the query's) falls into."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi as C
from .api import _DTYPES, _dt, _mask
from .cache_q8 import _call, _dense, _i32, _p, _same, _workspace


def _int(n):
    """n as the C ABI's int holds it: what lies past it is as good as its ends."""
    return max(-2 ** 31, min(2 ** 31 - 1, int(n)))


def rel_bucket(distance, num_buckets=32, max_distance=128, bidirectional=True) -> int:
    """The bucket of ``distance`` (key's position - query's position) via ``mha_rel_bucket``."""
    u = C.load().mha_rel_bucket(_int(distance), _int(num_buckets), _int(max_distance),
                                1 if bidirectional else 0)
    if u < 0:
        C.check(u, "mha_rel_bucket")
    return u


def _strides(*ts):
    """None where every tensor is contiguous, else their strides as the C ABI takes them (that of a
    dimension of one element, which nothing goes by, as a valid one)."""
    for t in ts:
        if not t.is_contiguous():
            return (ctypes.c_int64 * (4 * len(ts)))(
                *[s if n > 1 or i == 3 else 128
                  for t in ts for i, (n, s) in enumerate(zip(t.shape, t.stride()))])
    return None


def _qkv(what, q, k, v):
    """(device, dtype code, B, H, Nq, Nk, d_k, d_v) of tensors that fit together."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    dtype = q.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dt(q)  # raises
    try:
        (B, H, Nq, d_k), (Bk, Hk, Nk, dk), (Bv, Hv, Nv, d_v) = q.shape, k.shape, v.shape
    except ValueError:
        B, Bk = 0, 1
    if (Bk != B or Bv != B or Hk != H or Hv != H or Nv != Nk or dk != d_k or k.dtype is not dtype
            or v.dtype is not dtype or k.get_device() != dev or v.get_device() != dev):
        raise ValueError(f"{what}: q [B, H, Nq, d_k], k [B, H, Nk, d_k] and v [B, H, Nk, d_v] of "
                         "one type on one device expected")
    return dev, dt, B, H, Nq, Nk, d_k, d_v


def _new(like, B, H, N, d):
    """A contiguous tensor [B, H, N, d] of like's type and device."""
    if like.shape == (B, H, N, d) and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty((B, H, N, d), dtype=like.dtype, device=like.device)


def _table(what, rel_bias, H, dev):
    """(type code, num_buckets) of the bias."""
    shape = rel_bias.shape
    if (len(shape) != 2 or shape[1] != H or not rel_bias.is_contiguous()
            or rel_bias.get_device() != dev):
        raise ValueError(f"{what}: rel_bias must be a contiguous tensor [num_buckets, {H}] on the "
                         "device of the other tensors")
    return _dt(rel_bias), shape[0]


def _forward(what, q, k, v, rel_bias, mask, key_len, scale, max_distance, bidirectional, out, lse):
    dev, dt, B, H, Nq, Nk, d_k, d_v = _qkv(what, q, k, v)
    bt, nb = _table(what, rel_bias, H, dev)
    if key_len is not None:
        _dense(key_len, _i32, (B,), dev, "key_len")
    if out is None:
        out = _new(q, B, H, Nq, d_v)
    else:
        _same(out, q, (B, H, Nq, d_v), dev, f"{what}: out")
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse else None
    _call(dev, "mha_sdpa_rel_fwd", B, H, Nq, Nk, d_k, d_v, dt, _mask(mask), _p(key_len),
          float(scale or 0.0), q.data_ptr(), k.data_ptr(), v.data_ptr(), rel_bias.data_ptr(), bt,
          nb, _int(max_distance), 1 if bidirectional else 0, out.data_ptr(),
          _strides(q, k, v, out), _p(lse))
    return out, lse


def sdpa_rel(q, k, v, rel_bias, mask="none", key_len=None, scale=None, max_distance=128,
             bidirectional=True, out=None):
    """O = softmax(q k^T * scale + bias) v per (batch, head) via ``mha_sdpa_rel_fwd``: ``sdpa`` with
    rel_bias[bucket(j - i), h] added to the score of query i and key j.

    q [B,H,Nq,d_k], k [B,H,Nk,d_k], v [B,H,Nk,d_v] (any strides the kernels accept; d stride 1);
    mask "none", "causal" or "key_padding" (key_len int32 [B]); scale None: 1/sqrt(d_k)."""
    return _forward("sdpa_rel", q, k, v, rel_bias, mask, key_len, scale, max_distance,
                    bidirectional, out, False)[0]


def sdpa_rel_with_lse(q, k, v, rel_bias, mask="none", key_len=None, scale=None, max_distance=128,
                      bidirectional=True, out=None):
    """``sdpa_rel`` that returns (O, lse), lse fp32 [B,H,Nq] the natural log of each row's softmax
    denominator (what ``sdpa_rel_backward`` needs)."""
    return _forward("sdpa_rel_with_lse", q, k, v, rel_bias, mask, key_len, scale, max_distance,
                    bidirectional, out, True)


@functools.lru_cache(maxsize=1024)
def sdpa_rel_bwd_workspace_size(B, H, Nq, Nk, dtype, num_buckets) -> int:
    n = ctypes.c_size_t(0)
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    C.check(C.load().mha_sdpa_rel_bwd_workspace_size(B, H, Nq, Nk, dt, num_buckets,
                                                     ctypes.byref(n)),
            "mha_sdpa_rel_bwd_workspace_size")
    return n.value


def sdpa_rel_backward(q, k, v, rel_bias, o, do, lse, mask="none", key_len=None, scale=None,
                      max_distance=128, bidirectional=True, workspace=None):
    """(dq, dk, dv, drel_bias) via ``mha_sdpa_rel_bwd``: the gradients of ``sdpa_rel`` given
    do = dL/dO, from o and lse of ``sdpa_rel_with_lse`` with the same arguments.  drel_bias has the
    shape and type of rel_bias.  workspace: uint8 CUDA tensor of at least
    ``sdpa_rel_bwd_workspace_size(...)`` bytes, allocated here if None."""
    what = "sdpa_rel_backward"
    dev, dt, B, H, Nq, Nk, d_k, d_v = _qkv(what, q, k, v)
    bt, nb = _table(what, rel_bias, H, dev)
    _same(o, q, (B, H, Nq, d_v), dev, f"{what}: o")
    _same(do, q, (B, H, Nq, d_v), dev, f"{what}: do")
    _dense(lse, torch.float32, (B, H, Nq), dev, "lse")
    if key_len is not None:
        _dense(key_len, _i32, (B,), dev, "key_len")
    dq, dk, dv = _new(q, B, H, Nq, d_k), _new(k, B, H, Nk, d_k), _new(v, B, H, Nk, d_v)
    dbias = torch.empty_like(rel_bias)
    workspace = _workspace(workspace, sdpa_rel_bwd_workspace_size(B, H, Nq, Nk, dt, nb), q, dev,
                           what)
    _call(dev, "mha_sdpa_rel_bwd", B, H, Nq, Nk, d_k, d_v, dt, _mask(mask), _p(key_len),
          float(scale or 0.0), q.data_ptr(), k.data_ptr(), v.data_ptr(), rel_bias.data_ptr(), bt,
          nb, _int(max_distance), 1 if bidirectional else 0, o.data_ptr(), do.data_ptr(),
          lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dbias.data_ptr(),
          _strides(q, k, v, o, do, dq, dk, dv), workspace.data_ptr(), workspace.numel())
    return dq, dk, dv, dbias


@functools.lru_cache(maxsize=1024)
def sdpa_rel_decode_workspace_size(B, H, Nq, Lmax, d_k, d_v, dtype) -> int:
    n = ctypes.c_size_t(0)
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    C.check(C.load().mha_sdpa_rel_decode_workspace_size(B, H, Nq, Lmax, d_k, d_v, dt,
                                                        ctypes.byref(n)),
            "mha_sdpa_rel_decode_workspace_size")
    return n.value


def sdpa_rel_decode(q, k_cache, v_cache, rel_bias, cache_len, causal=True, scale=None,
                    max_distance=128, bidirectional=False, workspace=None, out=None):
    """One generation step against a key/value cache via ``mha_sdpa_rel_decode_fwd``:
    ``sdpa_decode`` with rel_bias[bucket(j - i), h] added to the score of cached position j, where
    query r of sequence b is at position i = cache_len[b] - Nq + r.

    q [B,H,Nq,d_k] (the new positions, already in the cache; Nq <= 16), k_cache / v_cache
    [B,H,Lmax,d], cache_len int32 CUDA tensor [B].  workspace: uint8 CUDA tensor of at least
    ``sdpa_rel_decode_workspace_size(...)`` bytes, allocated here if None."""
    what = "sdpa_rel_decode"
    dev, dt, B, H, Nq, Lmax, d_k, d_v = _qkv(what, q, k_cache, v_cache)
    bt, nb = _table(what, rel_bias, H, dev)
    _dense(cache_len, _i32, (B,), dev, "cache_len")
    if out is None:
        out = _new(q, B, H, Nq, d_v)
    else:
        _same(out, q, (B, H, Nq, d_v), dev, f"{what}: out")
    if workspace is None:
        need = sdpa_rel_decode_workspace_size(B, H, Nq, Lmax, d_k, d_v, dt)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _workspace(workspace, 0, q, dev, what)
    _call(dev, "mha_sdpa_rel_decode_fwd", B, H, Nq, Lmax, d_k, d_v, dt, 1 if causal else 0,
          cache_len.data_ptr(), float(scale or 0.0), q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), rel_bias.data_ptr(), bt, nb, _int(max_distance),
          1 if bidirectional else 0, out.data_ptr(), _strides(q, k_cache, v_cache, out),
          _p(workspace), 0 if workspace is None else workspace.numel())
    return out
