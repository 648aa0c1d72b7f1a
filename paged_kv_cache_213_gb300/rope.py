"""ctypes binding of the norm/rotation append (``include/pagedkv_rope.h``).
Marshalling only; the work is in the library's CUDA kernels."""
from __future__ import annotations

import ctypes

import torch

from .binding import _check, _need, library

PKV_ERRBIT_POSITION = 0x40

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = library()
        c = ctypes
        p, i, l, f = c.c_void_p, c.c_int, c.c_int64, c.c_float
        lib.paged_qk_norm_rope_append.argtypes = [p, p, p, p, l, l, l, p, p, f, p, p, i, i, i, p,
                                                  p, p, i, i, i, i, i, l, p, p]
        lib.paged_qk_norm_rope_append.restype = i
        lib.paged_qk_norm_rope_append_fp8.argtypes = [p, p, p, p, l, l, l, p, p, f, p, p, i, i, i,
                                                      p, p, p, i, i, i, i, i, l, f, f, p, p]
        lib.paged_qk_norm_rope_append_fp8.restype = i
        _bound = lib
    return _bound


# the current device and its current stream's handle as plain integers: the
# wrapper objects of torch.cuda cost 2 us a call, a sixth of a small call's time
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _launch(dev, fn, *args):
    """fn(*args, current stream) with dev current; returns the status."""
    index = dev.index
    if _current_device() == index:
        return fn(*args, _current_stream(index))
    with torch.cuda.device(dev):
        return fn(*args, _current_stream(index))


def _need_cuda(t, name, dtype, dev):
    """_need without the contiguity check: the caller checks the strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _token_stride(t, name):
    """Elements between tokens of t [T, heads, d], whose heads are contiguous."""
    T, H, d = t.shape
    st, sh, se = t.stride()
    if (d > 1 and se != 1) or (H > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return st if T > 1 else H * d


def _append(scales, q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping, k_cache,
            v_cache, interleaved, q_out, err_word):
    fp8 = scales is not None
    dev = k_cache.device
    kind = torch.uint8 if fp8 else torch.float16
    _need(k_cache, "k_cache", kind)
    _need(v_cache, "v_cache", kind, dev)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache/v_cache must both be [num_blocks, n_kv_heads, block_size, head_dim]")
    NB, Hk, bs, d = k_cache.shape
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need_cuda(t, name, torch.float16, dev)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q must be [num_tokens, n_q_heads, head_dim]")
    T, H = q.shape[:2]
    if k.shape != (T, Hk, d) or v.shape != (T, Hk, d):
        raise ValueError("k/v must be [num_tokens, n_kv_heads, head_dim]")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, name, torch.float16, dev)
            if w.shape != (d,):
                raise ValueError(f"{name} must be [head_dim]")
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    table, rot = 0, 0
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", torch.float32, dev)
        _need(positions, "positions", torch.int32, dev)
        if cos_sin.dim() != 2 or positions.shape != (T,):
            raise ValueError("cos_sin must be [max_positions, rot_dim], positions [num_tokens]")
        table, rot = cos_sin.shape
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=torch.float16, device=dev)
    else:
        _need(q_out, "q_out", torch.float16, dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    lib = _lib()
    args = (_ptr(q_out), _ptr(q), _ptr(k), _ptr(v), _token_stride(q, "q"), _token_stride(k, "k"),
            _token_stride(v, "v"), _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(cos_sin),
            _ptr(positions) if rot else None, table, rot, int(bool(interleaved)),
            _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), T, H, Hk, d, bs, NB)
    if fp8:
        rc = _launch(dev, lib.paged_qk_norm_rope_append_fp8, *args, float(scales[0]),
                     float(scales[1]), _ptr(err_word))
        _check("paged_qk_norm_rope_append_fp8", rc)
    else:
        rc = _launch(dev, lib.paged_qk_norm_rope_append, *args, _ptr(err_word))
        _check("paged_qk_norm_rope_append", rc)
    return q_out


def paged_qk_norm_rope_append(q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping,
                              k_cache, v_cache, interleaved=False, q_out=None, err_word=None):
    """RMS norm of each query and key head, rotation by position and the append
    of K/V into their slots, in one kernel on the current stream.

    q [T, H, d], k, v [T, Hk, d] fp16: a token's heads contiguous, any stride
    between tokens (columns of a fused projection's output will do).  q_weight,
    k_weight [d] fp16 or None (no norm).  cos_sin [max_positions, rot_dim] fp32
    (cosines, then sines) and positions [T] int32, or None and None for no
    rotation; interleaved pairs (2i, 2i + 1) instead of split halves.
    slot_mapping [T] int64 (negative: padding, skipped); caches [NB, Hk, bs, d]
    fp16, in place.  Returns the queries [T, H, d] (q_out, which may be a
    contiguous q)."""
    return _append(None, q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping,
                   k_cache, v_cache, interleaved, q_out, err_word)


def paged_qk_norm_rope_append_fp8(q, k, v, q_weight, k_weight, eps, cos_sin, positions,
                                  slot_mapping, k_cache, v_cache, k_scale, v_scale,
                                  interleaved=False, q_out=None, err_word=None):
    """paged_qk_norm_rope_append into E4M3 caches (uint8 codes of value / scale)."""
    return _append((k_scale, v_scale), q, k, v, q_weight, k_weight, eps, cos_sin, positions,
                   slot_mapping, k_cache, v_cache, interleaved, q_out, err_word)
