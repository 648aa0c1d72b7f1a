"""ctypes binding of latent attention over a paged cache
(``include/pagedkv_latent.h``).  Marshalling only; the work is in the library's
CUDA kernels."""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import _check, _need, library
from .rope import _F16, _F32, _I32, _I64, _U8, _at, _at_strided, _current_device, _launch, _native

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = library()
        c = ctypes
        p, i, l, f = c.c_void_p, c.c_int, c.c_int64, c.c_float
        lib.paged_latent_append.argtypes = [p, l, p, f, p, p, i, i, p, p, p, l, l, p, l, l, i, i,
                                            i, i, i, l, p, p]
        lib.paged_latent_append.restype = i
        lib.paged_latent_plan.argtypes = [i] * 9 + [c.POINTER(c.c_size_t)]
        lib.paged_latent_plan.restype = i
        lib.paged_latent_attention.argtypes = [p, p, p, p, p, p, i, i, i, i, l, f, i, i, i, i, i,
                                               p, c.c_size_t, p, p, p]
        lib.paged_latent_attention.restype = i
        lib.paged_latent_gather.argtypes = [p, p, p, p, p, i, l, i, l, i, i, i, p, p]
        lib.paged_latent_gather.restype = i
        lib.latent_prefill_attention.argtypes = [p, p, p, p, p, p, i, i, i, i, i, f, i, i, i, p,
                                                 p, p]
        lib.latent_prefill_attention.restype = i
        _bound = lib
    return _bound


def _cache(cache):
    """(device, address, blocks, block size, entries of a row) of a latent cache."""
    _need(cache, "cache", _F16)
    shape = cache.shape
    if len(shape) != 3:
        raise ValueError("cache must be [num_blocks, block_size, latent_dim + rope_dim]")
    return (cache.device, cache.data_ptr(), *shape)


def _strides(t, name, T, H, P):
    """(token stride, head stride) of t [T, H, P] with contiguous entries."""
    st, sh, se = t.stride()
    if se != 1 and P > 1:
        raise ValueError(f"{name}: the entries of a head must be contiguous")
    if H == 1:
        sh = P
    return (st if T > 1 else H * sh), sh


def paged_latent_append(kv, weight, eps, cos_sin, positions, slot_mapping, cache, q_rope=None,
                        q_out=None, interleaved=False, err_word=None):
    """Append new tokens to a latent cache [NB, bs, R + P] fp16, in place: the
    RMS norm of kv[:, :R] (weight [R] fp16, or None) and the rotation of
    kv[:, R:] (cos_sin [max_positions, P] fp32, positions [T] int32) go to
    slot_mapping [T] int64.  kv [T, R + P] fp16, any stride between tokens.
    With q_rope [T, H, P] the position part of the queries is rotated into
    q_out [T, H, P] (both with gaps between heads and tokens if need be, tokens
    outermost: q[..., d:] and absorbed[..., R:]; q_out may be q_rope)."""
    if _native().latent_append(kv, weight, eps, cos_sin, positions, slot_mapping, cache, q_rope,
                               q_out, interleaved, err_word):
        return
    dev, cp, NB, bs, E = _cache(cache)
    kp = _at_strided(kv, "kv", _F16, dev)
    shape = kv.shape
    if len(shape) != 2 or shape[1] != E or (E > 1 and kv.stride(1) != 1):
        raise ValueError("kv must be [num_tokens, latent_dim + rope_dim], entries contiguous")
    T = shape[0]
    cs = _at(cos_sin, "cos_sin", _F32, dev)
    pos = _at(positions, "positions", _I32, dev)
    slots = _at(slot_mapping, "slot_mapping", _I64, dev)
    shape = cos_sin.shape
    if len(shape) != 2 or positions.shape != (T,) or slot_mapping.shape != (T,):
        raise ValueError("cos_sin must be [max_positions, rope_dim], positions and slot_mapping [T]")
    table, P = shape
    R = E - P
    if R <= 0:
        raise ValueError("cos_sin is as wide as the cache rows: no latent entries")
    wp = None
    if weight is not None:
        wp = _at(weight, "weight", _F16, dev)
        if weight.shape != (R,):
            raise ValueError("weight must be [latent_dim]")
    H, qs, os, qp, op = 0, (0, 0), (0, 0), None, None
    if q_rope is not None and q_out is not None:
        qp = _at_strided(q_rope, "q_rope", _F16, dev)
        op = _at_strided(q_out, "q_out", _F16, dev)
        shape = q_rope.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != P or q_out.shape != shape:
            raise ValueError("q_rope and q_out must be [num_tokens, n_q_heads, rope_dim]")
        H = shape[1]
        qs, os = _strides(q_rope, "q_rope", T, H, P), _strides(q_out, "q_out", T, H, P)
    elif q_rope is not None or q_out is not None:
        raise ValueError("q_rope and q_out go together")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().paged_latent_append, kp, kv.stride(0) if T > 1 else E, wp,
                 float(eps), cs, pos, table, 1 if interleaved else 0, slots, cp, qp, *qs, op, *os, H, T, R, P, bs,
                 NB, err)
    _check("paged_latent_append", rc)


def latent_plan(num_seqs, total_q, max_q_len, n_q_heads, latent_dim, rope_dim, block_size,
                max_blocks_per_seq, max_context_len=0):
    """Workspace bytes of paged_latent_attention on the current device."""
    W = ctypes.c_size_t(0)
    _check("paged_latent_plan",
           _lib().paged_latent_plan(num_seqs, total_q, max_q_len, n_q_heads, latent_dim, rope_dim,
                                    block_size, max_blocks_per_seq, max_context_len,
                                    ctypes.byref(W)))
    return W.value


@functools.lru_cache(maxsize=4096)
def _plan_on(index, *sizes):
    """latent_plan on device `index`: a function of the sizes alone."""
    if _current_device() == index:
        return latent_plan(*sizes)
    with torch.cuda.device(index):
        return latent_plan(*sizes)


def paged_latent_attention(q, cache, block_tables, context_lens, scale, latent_dim,
                           query_start=None, max_q_len=1, max_context_len=None, out=None,
                           workspace=None, lse=None, err_word=None):
    """Absorbed latent attention over a paged latent cache [NB, bs, R + P] fp16.

    q [total_q, H, R + P] fp16 (the absorbed queries, then their rotated part);
    block_tables [B, MB] and context_lens [B] int32.  query_start [B + 1] int32:
    sequence b owns the rows [query_start[b], query_start[b + 1]), its newest
    tokens (causal; max_q_len bounds their number); None: one token a sequence.
    Returns out [total_q, H, R] fp16: the weighted latents of every head."""
    done = _native().latent_attention(q, cache, block_tables, context_lens, scale, latent_dim,
                                      query_start, max_q_len,
                                      0 if max_context_len is None else max_context_len, out,
                                      workspace, lse, err_word)
    if done is not None:
        return done
    dev, cp, NB, bs, E = _cache(cache)
    qp = _at(q, "q", _F16, dev)
    tables = _at(block_tables, "block_tables", _I32, dev)
    lens = _at(context_lens, "context_lens", _I32, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != E:
        raise ValueError("q must be [total_q, n_q_heads, latent_dim + rope_dim]")
    TQ, H, _ = shape
    R = int(latent_dim)
    if not 0 < R < E:
        raise ValueError("latent_dim must be positive and smaller than the cache rows")
    shape = block_tables.shape
    if len(shape) != 2 or context_lens.shape != (shape[0],):
        raise ValueError("block_tables must be [B, MB], context_lens [B]")
    B, MB = shape
    start = None
    if query_start is not None:
        start = _at(query_start, "query_start", _I32, dev)
        if query_start.shape != (B + 1,):
            raise ValueError("query_start must be [B + 1]")
    elif TQ != B or max_q_len != 1:
        raise ValueError("without query_start, q holds one token a sequence")
    mcl = 0 if max_context_len is None else int(max_context_len)
    max_q_len = int(max_q_len)
    if out is None:
        out = torch.empty((TQ, H, R), dtype=_F16, device=dev)
        op = out.data_ptr()
    else:
        op = _at(out, "out", _F16, dev)
        if out.shape != (TQ, H, R):
            raise ValueError("out must be [total_q, n_q_heads, latent_dim]")
    lp = None
    if lse is not None:
        lp = _at(lse, "lse", _F32, dev)
        if lse.shape != (TQ, H):
            raise ValueError("lse must be [total_q, n_q_heads]")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    if workspace is None:
        size = _plan_on(dev.index, B, TQ, max_q_len, H, R, E - R, bs, MB, mcl)
        workspace = torch.empty(size, dtype=_U8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp = _at(workspace, "workspace", _U8, dev)
        size = workspace.numel()
    rc = _launch(dev, _lib().paged_latent_attention, op, qp, cp, tables, lens, start, B, TQ,
                 max_q_len, MB, NB, float(scale), H, R, E - R, bs, mcl, wp, size, lp, err)
    _check("paged_latent_attention", rc)
    return out


def paged_latent_gather(cache, block_tables, start, total, latent_dim, latents=None, ropes=None,
                        err_word=None):
    """Cached rows in token order: rows [start[b], start[b + 1]) of the results
    are the first tokens of sequence b.  cache [NB, bs, R + P] fp16,
    block_tables [B, MB] and start [B + 1] int32, total: rows of the results.
    Returns (latents [total, R], ropes [total, P]) fp16."""
    done = _native().latent_gather(cache, block_tables, start, total, latent_dim, latents, ropes,
                                   err_word)
    if done is not None:
        return done
    dev, cp, NB, bs, E = _cache(cache)
    tables = _at(block_tables, "block_tables", _I32, dev)
    first = _at(start, "start", _I32, dev)
    R = int(latent_dim)
    if not 0 < R < E:
        raise ValueError("latent_dim must be positive and smaller than the cache rows")
    shape = block_tables.shape
    if len(shape) != 2 or start.shape != (shape[0] + 1,):
        raise ValueError("block_tables must be [B, MB], start [B + 1]")
    B, MB = shape
    total = int(total)
    if latents is None:
        latents = torch.empty((total, R), dtype=_F16, device=dev)
    elif latents.shape != (total, R):
        raise ValueError("latents must be [total, latent_dim]")
    if ropes is None:
        ropes = torch.empty((total, E - R), dtype=_F16, device=dev)
    elif ropes.shape != (total, E - R):
        raise ValueError("ropes must be [total, rope_dim]")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().paged_latent_gather, _at(latents, "latents", _F16, dev),
                 _at(ropes, "ropes", _F16, dev), cp, tables, first, B, total, MB, NB, R, E - R, bs,
                 err)
    _check("paged_latent_gather", rc)
    return latents, ropes


def latent_prefill_attention(q, kv, k_rope, q_start, kv_start, scale, max_q_len, max_kv_len,
                             out=None, lse=None, err_word=None):
    """Causal attention of prompts over keys and values expanded from latents.

    q [total_q, H, d + P], kv [total_kv, H, 2 d] (key, then value), k_rope
    [total_kv, P], fp16; q_start, kv_start [B + 1] int32: each sequence's query
    rows and key rows (its queries are the newest tokens of its keys).
    max_q_len, max_kv_len: host bounds.  Returns out [total_q, H, d] fp16."""
    done = _native().latent_prefill(q, kv, k_rope, q_start, kv_start, scale, max_q_len, max_kv_len,
                                    out, lse, err_word)
    if done is not None:
        return done
    _need(q, "q", _F16)
    dev = q.device
    kp = _at(kv, "kv", _F16, dev)
    rp = _at(k_rope, "k_rope", _F16, dev)
    qs = _at(q_start, "q_start", _I32, dev)
    ks = _at(kv_start, "kv_start", _I32, dev)
    if q.dim() != 3 or kv.dim() != 3 or k_rope.dim() != 2 or kv.shape[1] != q.shape[1] or \
            kv.shape[0] != k_rope.shape[0] or kv.shape[2] != 2 * (q.shape[2] - k_rope.shape[1]):
        raise ValueError("q must be [total_q, H, d + P], kv [total_kv, H, 2 d], k_rope [total_kv, P]")
    TQ, H, E = q.shape
    TK, P = k_rope.shape
    d = E - P
    if q_start.dim() != 1 or q_start.numel() < 1 or kv_start.shape != q_start.shape:
        raise ValueError("q_start and kv_start must be [B + 1]")
    if out is None:
        out = torch.empty((TQ, H, d), dtype=_F16, device=dev)
    elif out.shape != (TQ, H, d):
        raise ValueError("out must be [total_q, H, d]")
    lp = None
    if lse is not None:
        lp = _at(lse, "lse", _F32, dev)
        if lse.shape != (TQ, H):
            raise ValueError("lse must be [total_q, H]")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().latent_prefill_attention, _at(out, "out", _F16, dev), q.data_ptr(), kp,
                 rp, qs, ks, q_start.numel() - 1, TQ, TK, int(max_q_len),
                 int(max_kv_len), float(scale), H, d, P, lp, err)
    _check("latent_prefill_attention", rc)
    return out
