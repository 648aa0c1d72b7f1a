"""ctypes binding of the norm/rotation append (``include/pagedkv_rope.h``).
Marshalling only; the work is in the library's CUDA kernels."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import warnings

import torch

from .binding import _check, _need, library, library_path

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


_calls = None


class _PythonOnly:
    """In the place of the native module where it is missing: takes no call."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_calls():
    from . import build as _build
    path = os.path.join(os.path.dirname(library_path()), "_pagedkv_calls.so")
    target, built = _build.calls_target(), _build.calls_built_for()
    why = "missing" if built is None else f"built for {built}, not for {target}"
    if built is not None and built == target:
        try:
            spec = importlib.util.spec_from_file_location("_pagedkv_calls", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            return module
        except (ImportError, OSError) as e:
            why = str(e)
    warnings.warn(f"{path}: {why}; the calls are marshalled in Python, about 10 us slower each "
                  "(build with python -m paged_kv_cache_213_gb300.build)", RuntimeWarning,
                  stacklevel=4)
    return _PythonOnly()


def _native():
    """The module of ``native/calls.cpp``, which marshals the plain case of each call:
    small calls take as long as the host needs for them, and this code needs 10 us more.
    Its functions return None, having launched nothing, for what they do not take; the
    code below then checks, and calls the library or raises.  Where the module is
    missing or was built for another torch, a warning says so once, and this code does
    all of it."""
    global _calls
    if _calls is None:
        library()
        _calls = _load_calls()
    return _calls


# Each tensor is looked at once (the full checks of _need run where that look fails, for
# the message), and device, stream and pointers are plain integers (the wrapper objects
# of torch.cuda cost 2 us a call).
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # None: a torch without CUDA
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_F16, _F32, _I32, _I64, _U8 = (torch.float16, torch.float32, torch.int32, torch.int64,
                               torch.uint8)


def _at(t, name, dtype, dev):
    """t's address; t must be a contiguous tensor of this type on the CUDA device dev."""
    try:
        if t.dtype is dtype and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, dev)
    raise ValueError(f"{name} must be on {dev}")


def _at_strided(t, name, dtype, dev):
    """t's address; the caller checks the strides."""
    try:
        if t.dtype is dtype and t.device == dev:
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _launch(dev, fn, *args):
    """fn(*args, current stream) with dev current; returns the status."""
    index = dev.index
    if _current_device() == index:
        return fn(*args, _current_stream(index))
    with torch.cuda.device(dev):
        return fn(*args, _current_stream(index))


def _token_stride(t, name, T, H, d):
    """Elements between tokens of t [T, H, d], whose heads are contiguous."""
    st, sh, se = t.stride()
    if (se != 1 and d > 1) or (sh != d and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return st if T > 1 else H * d


def _append(scales, q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping, k_cache,
            v_cache, interleaved, q_out, err_word):
    fp8 = scales is not None
    kind = _U8 if fp8 else _F16
    _need(k_cache, "k_cache", kind)
    dev = k_cache.device
    vc = _at(v_cache, "v_cache", kind, dev)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache/v_cache must both be [num_blocks, n_kv_heads, block_size, head_dim]")
    NB, Hk, bs, d = shape
    qp = _at_strided(q, "q", _F16, dev)
    kp = _at_strided(k, "k", _F16, dev)
    vp = _at_strided(v, "v", _F16, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [num_tokens, n_q_heads, head_dim]")
    T, H, _ = shape
    if k.shape != (T, Hk, d) or v.shape != (T, Hk, d):
        raise ValueError("k/v must be [num_tokens, n_kv_heads, head_dim]")
    qw = kw = None
    if q_weight is not None:
        qw = _at(q_weight, "q_weight", _F16, dev)
        if q_weight.shape != (d,):
            raise ValueError("q_weight must be [head_dim]")
    if k_weight is not None:
        kw = _at(k_weight, "k_weight", _F16, dev)
        if k_weight.shape != (d,):
            raise ValueError("k_weight must be [head_dim]")
    slots = _at(slot_mapping, "slot_mapping", _I64, dev)
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    table = rot = 0
    cs = pos = None
    if cos_sin is not None:
        cs = _at(cos_sin, "cos_sin", _F32, dev)
        pos = _at(positions, "positions", _I32, dev)
        shape = cos_sin.shape
        if len(shape) != 2 or positions.shape != (T,):
            raise ValueError("cos_sin must be [max_positions, rot_dim], positions [num_tokens]")
        table, rot = shape
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=_F16, device=dev)
        op = q_out.data_ptr()
    else:
        op = _at(q_out, "q_out", _F16, dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    lib = _lib()
    args = (op, qp, kp, vp, _token_stride(q, "q", T, H, d), _token_stride(k, "k", T, Hk, d),
            _token_stride(v, "v", T, Hk, d), qw, kw, float(eps), cs, pos, table, rot,
            1 if interleaved else 0, slots, k_cache.data_ptr(), vc, T, H, Hk, d, bs, NB)
    if fp8:
        rc = _launch(dev, lib.paged_qk_norm_rope_append_fp8, *args, float(scales[0]),
                     float(scales[1]), err)
        _check("paged_qk_norm_rope_append_fp8", rc)
    else:
        rc = _launch(dev, lib.paged_qk_norm_rope_append, *args, err)
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
    done = _native().qk_append(q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping,
                               k_cache, v_cache, interleaved, q_out, err_word)
    if done is not None:
        return done
    return _append(None, q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping,
                   k_cache, v_cache, interleaved, q_out, err_word)


def paged_qk_norm_rope_append_fp8(q, k, v, q_weight, k_weight, eps, cos_sin, positions,
                                  slot_mapping, k_cache, v_cache, k_scale, v_scale,
                                  interleaved=False, q_out=None, err_word=None):
    """paged_qk_norm_rope_append into E4M3 caches (uint8 codes of value / scale)."""
    done = _native().qk_append_fp8(q, k, v, q_weight, k_weight, eps, cos_sin, positions,
                                   slot_mapping, k_cache, v_cache, interleaved, q_out, err_word,
                                   k_scale, v_scale)
    if done is not None:
        return done
    return _append((k_scale, v_scale), q, k, v, q_weight, k_weight, eps, cos_sin, positions,
                   slot_mapping, k_cache, v_cache, interleaved, q_out, err_word)
