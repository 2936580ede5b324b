"""torch-facing wrappers of the 8-bit key/value cache (argument checks and marshalling only, as
in ``api``): quantised append, the generation step's attention, a prompt's attention weights
and eviction by accumulated weight."""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _capi as C
from .api import _DTYPES, _dt, _mask

_CODES = {torch.float8_e4m3fn: C.MHA_Q8_E4M3, torch.int8: C.MHA_Q8_I8}
_BLOCKS = (16, 32, 64, 128)


class KvCacheQ8(NamedTuple):
    """An 8-bit key/value cache: codes k, v [B, H, Lmax, 64] (torch.float8_e4m3fn or torch.int8,
    any strides the kernels accept), scales k_scale, v_scale fp32 [B, H, ceil(Lmax / block)],
    weights fp32 [B, H, Lmax] (the attention weight each position has received) or None, and
    block, the positions that share a scale.  The number of valid positions is kept by the
    caller, as an int32 tensor [B]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    weights: Optional[torch.Tensor]
    block: int


def kv_cache_q8(B, H, Lmax, block=64, dtype=torch.float8_e4m3fn, weights=True, device="cuda"):
    """An empty ``KvCacheQ8``: zero codes, scales of 1, zero weights (None if not asked for)."""
    if dtype not in _CODES:
        raise TypeError(f"unsupported code dtype {dtype}; use torch.float8_e4m3fn or torch.int8")
    if block not in _BLOCKS:
        raise ValueError(f"block must be one of {_BLOCKS}")
    codes = [torch.zeros((B, H, Lmax, 64), dtype=torch.int8, device=device).view(dtype)
             for _ in range(2)]
    scales = [torch.ones((B, H, -(-Lmax // block)), device=device) for _ in range(2)]
    return KvCacheQ8(*codes, *scales,
                     torch.zeros((B, H, Lmax), device=device) if weights else None, block)


# The calls here are as short as the kernels behind them (a generation step of one sequence takes
# 5 us on the GPU), so checks and marshalling are written for speed: devices are compared by index,
# sizes of workspaces are remembered by the numbers they follow from.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent without CUDA
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_f32, _i32 = torch.float32, torch.int32


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dense(t, dtype, shape, dev, what):
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != dev):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on the device "
                         "of the other tensors")


def _check_cache(c, dev, what="cache"):
    """(B, H, Lmax, code type) of a cache whose tensors fit together and live on device ``dev``
    (an index, -1 for the host)."""
    k, v, k_scale, v_scale, weights, block = c
    code = _CODES.get(k.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported code dtype {k.dtype}; use torch.float8_e4m3fn or "
                        "torch.int8")
    if block not in _BLOCKS:
        raise ValueError(f"{what}: block must be one of {_BLOCKS}")
    shape = k.shape
    if (len(shape) != 4 or shape[3] != 64 or v.shape != shape or v.dtype is not k.dtype
            or k.get_device() != dev or v.get_device() != dev):
        raise ValueError(f"{what}: k and v must be [B, H, Lmax, 64] codes of one type on the "
                         "device of the other tensors")
    B, H, Lmax, _ = shape
    nb = (B, H, -(-Lmax // block))
    _dense(k_scale, _f32, nb, dev, f"{what}.k_scale")
    _dense(v_scale, _f32, nb, dev, f"{what}.v_scale")
    if weights is not None:
        _dense(weights, _f32, (B, H, Lmax), dev, f"{what}.weights")
    return B, H, Lmax, code


def _same(t, like, shape, dev, what):
    if t.dtype is not like.dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{what} must be a {like.dtype} tensor {list(shape)} on {like.device}")


def _cuda_device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    return dev


def _strides(*ts):
    """None where every tensor is contiguous, else their strides as the C ABI takes them."""
    for t in ts:
        if not t.is_contiguous():
            return (ctypes.c_int64 * (4 * len(ts)))(*[x for t in ts for x in t.stride()])
    return None


def _p(t):
    return None if t is None else t.data_ptr()


def _call(dev, name, *args):
    """The entry point ``name`` on the current stream of device ``dev`` (appended to the
    arguments), with ``dev`` the current device."""
    fn = getattr(C.load(), name)
    if _current_device() == dev:
        code = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(dev))
    if code:
        C.check(code, name)


def _workspace(workspace, need, like, dev, what):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    _need(workspace.dtype is torch.uint8 and workspace.get_device() == dev
          and workspace.is_contiguous(),
          f"{what}: workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


def kv_append_q8(cache, k, v, cache_len, new_len=None):
    """Quantise new keys and values into the cache via ``mha_kv_append_q8``: token i of sequence
    b goes to position cache_len[b] + i.

    k, v [B, H, N, 64] bf16 or fp32; cache_len int32 [B], the positions there before the call
    (add the new ones to it afterwards); new_len int32 [B], how many of the N tokens are real in
    each sequence (None: all).  The cache is written in place; its weights, where it keeps them,
    are 0 for the new positions."""
    dev = _cuda_device(k)
    B, H, Lmax, qt = _check_cache(cache, dev)
    dt = _dt(k)
    shape = k.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != H or shape[3] != 64:
        raise ValueError(f"kv_append_q8: k must be [{B}, {H}, N, 64]")
    _same(v, k, shape, dev, "kv_append_q8: v")
    _dense(cache_len, _i32, (B,), dev, "cache_len")
    if new_len is not None:
        _dense(new_len, _i32, (B,), dev, "new_len")
    _call(dev, "mha_kv_append_q8", B, H, shape[2], Lmax, 64, 64, dt, qt, cache.block,
          _p(new_len), cache_len.data_ptr(), k.data_ptr(), v.data_ptr(), cache.k.data_ptr(),
          cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(),
          _p(cache.weights), _strides(k, v, cache.k, cache.v))


@functools.lru_cache(maxsize=1024)
def decode_q8_workspace_size(B, H, Hkv, Nq, Lmax, with_weights) -> int:
    n = ctypes.c_size_t(0)
    C.check(C.load().mha_decode_q8_workspace_size(B, H, Hkv, Nq, Lmax, int(bool(with_weights)),
                                                  ctypes.byref(n)),
            "mha_decode_q8_workspace_size")
    return n.value


def sdpa_decode_q8(q, cache, cache_len, causal=True, scale=None, add_weights=False,
                   workspace=None, out=None):
    """One generation step against an 8-bit cache via ``mha_sdpa_decode_q8_fwd``.

    q [B, Hq, Nq, 64] (the new positions, already appended; Hq a multiple of the cache's heads,
    query head h reading cache head h // (Hq // H)), cache_len int32 [B] (valid positions, the
    new ones included); causal and scale as for ``sdpa_decode``.  add_weights: add to
    cache.weights what each position received from these queries.  workspace: uint8 CUDA tensor
    of at least ``decode_q8_workspace_size(...)`` bytes, allocated here if None.  Returns O
    [B, Hq, Nq, 64] (``out`` if given)."""
    dev = _cuda_device(q)
    Bc, Hkv, Lmax, qt = _check_cache(cache, dev)
    dt = _dt(q)
    shape = q.shape
    if len(shape) != 4 or shape[0] != Bc or shape[3] != 64 or shape[1] % Hkv != 0:
        raise ValueError(f"sdpa_decode_q8: q must be [{Bc}, a multiple of {Hkv}, Nq, 64]")
    if add_weights and cache.weights is None:
        raise ValueError("sdpa_decode_q8: add_weights needs a cache with weights")
    B, H, Nq, _ = shape
    _dense(cache_len, _i32, (B,), dev, "cache_len")
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        _same(out, q, shape, dev, "sdpa_decode_q8: out")
    if workspace is None:
        need = decode_q8_workspace_size(B, H, Hkv, Nq, Lmax, bool(add_weights))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _workspace(workspace, 0, q, dev, "sdpa_decode_q8")
    _call(dev, "mha_sdpa_decode_q8_fwd", B, H, Hkv, Nq, Lmax, 64, 64, dt, qt, cache.block,
          1 if causal else 0, cache_len.data_ptr(), float(scale or 0.0), q.data_ptr(),
          cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
          cache.v_scale.data_ptr(), out.data_ptr(), _strides(q, cache.k, cache.v, out),
          cache.weights.data_ptr() if add_weights else None, _p(workspace),
          0 if workspace is None else workspace.numel())
    return out


@functools.lru_cache(maxsize=1024)
def key_weights_workspace_size(B, H, Hkv, Nq, Nk, dtype) -> int:
    n = ctypes.c_size_t(0)
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    C.check(C.load().mha_key_weights_workspace_size(B, H, Hkv, Nq, Nk, dt, ctypes.byref(n)),
            "mha_key_weights_workspace_size")
    return n.value


def sdpa_key_weights(q, k, lse, mask="none", key_len=None, query_len=None, scale=None,
                     weights=None, workspace=None):
    """The attention weight each key of a prompt received, added to ``weights`` via
    ``mha_sdpa_key_weights``.

    q [B, Hq, Nq, 64], k [B, H, Nk, 64] (Hq a multiple of H), lse fp32 [B, Hq, Nq] from
    ``sdpa_with_lse`` with the same mask and scale; query_len int32 [B]: rows from there on add
    nothing (the padding of a ragged batch).  weights fp32 [B, H, L], L >= Nk (the weights of an
    8-bit cache, say); zeros [B, H, Nk] are made if None.  Returns weights."""
    dev = _cuda_device(q)
    dt = _dt(q)
    shape, kshape = q.shape, k.shape
    if (len(shape) != 4 or len(kshape) != 4 or shape[3] != 64 or kshape[3] != 64
            or kshape[0] != shape[0] or kshape[1] < 1 or shape[1] % kshape[1] != 0
            or k.dtype is not q.dtype or k.get_device() != dev):
        raise ValueError("sdpa_key_weights: q [B, Hq, Nq, 64] and k [B, H, Nk, 64] of one type on "
                         "one device expected, Hq a multiple of H")
    B, H, Nq, _ = shape
    Hkv, Nk = kshape[1], kshape[2]
    _dense(lse, _f32, (B, H, Nq), dev, "lse")
    if key_len is not None:
        _dense(key_len, _i32, (B,), dev, "key_len")
    if query_len is not None:
        _dense(query_len, _i32, (B,), dev, "query_len")
    if weights is None:
        weights = torch.zeros((B, Hkv, Nk), device=q.device)
    else:
        _need(weights.dim() == 3 and weights.shape[2] >= Nk,
              f"sdpa_key_weights: weights must be [{B}, {Hkv}, at least {Nk}]")
        _dense(weights, _f32, (B, Hkv, weights.shape[2]), dev, "weights")
    need = key_weights_workspace_size(B, H, Hkv, Nq, Nk, dt)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, q, dev, "sdpa_key_weights")
    _call(dev, "mha_sdpa_key_weights", B, H, Hkv, Nq, Nk, 64, dt, _mask(mask), _p(key_len),
          _p(query_len), float(scale or 0.0), q.data_ptr(), k.data_ptr(), lse.data_ptr(),
          _strides(q, k), weights.data_ptr(), weights.shape[2], _p(workspace),
          0 if workspace is None else workspace.numel())
    return weights


def kv_evict_q8(cache, out, cache_len, keep, recent=0, len_out=None, kept=None):
    """Move the positions worth keeping from ``cache`` into the cache ``out`` via
    ``mha_kv_evict_q8``: every position of a head with at most ``keep`` of them, else the newest
    ``recent`` and those of the others with the largest ``cache.weights``, in their order.

    out: a ``KvCacheQ8`` of the same B, heads, code type and block, with room for ``keep``
    positions, sharing no memory with ``cache`` (its weights may be None).  Returns (len_out
    int32 [B], the valid positions of ``out``; kept int32 [B, H, keep], the old position of each,
    -1 behind the last)."""
    dev = _cuda_device(cache.k)
    B, H, Lmax, qt = _check_cache(cache, dev)
    B2, H2, Lout, qt2 = _check_cache(out, dev, "out")
    if (B2, H2, qt2, out.block) != (B, H, qt, cache.block):
        raise ValueError("kv_evict_q8: out must have the batch, heads, code type and block of "
                         "cache")
    if cache.weights is None:
        raise ValueError("kv_evict_q8: the cache keeps no weights to go by")
    _dense(cache_len, _i32, (B,), dev, "cache_len")
    keep, recent = int(keep), int(recent)
    _need(1 <= keep <= Lout and recent >= 0,
          f"kv_evict_q8: keep must be 1..{Lout} (the room in out) and recent not negative")
    if len_out is None:
        len_out = torch.empty(B, dtype=_i32, device=cache.k.device)
    else:
        _dense(len_out, _i32, (B,), dev, "len_out")
    if kept is None:
        kept = torch.empty((B, H, keep), dtype=_i32, device=cache.k.device)
    else:
        _dense(kept, _i32, (B, H, keep), dev, "kept")
    _call(dev, "mha_kv_evict_q8", B, H, Lmax, Lout, 64, 64, qt, cache.block, keep,
          min(recent, keep), cache_len.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(),
          cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), cache.weights.data_ptr(),
          out.k.data_ptr(), out.v.data_ptr(), out.k_scale.data_ptr(), out.v_scale.data_ptr(),
          _p(out.weights), len_out.data_ptr(), kept.data_ptr(),
          _strides(cache.k, cache.v, out.k, out.v))
    return len_out, kept
