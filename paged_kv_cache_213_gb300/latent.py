"""ctypes binding of latent attention over a paged cache
(``include/pagedkv_latent.h``).  Marshalling only; the work is in the library's
CUDA kernels."""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import _check, _need, library
from .rope import _current_device, _launch, _need_cuda, _ptr

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


def _need_cache(cache):
    _need(cache, "cache", torch.float16)
    if cache.dim() != 3:
        raise ValueError("cache must be [num_blocks, block_size, latent_dim + rope_dim]")


def _strides(t, name, per):
    """(token stride, head stride) of t [T, H, P] with contiguous entries."""
    T, H, P = t.shape
    st, sh, se = t.stride()
    if P > 1 and se != 1:
        raise ValueError(f"{name}: the entries of a head must be contiguous")
    sh = sh if H > 1 else per
    return (st if T > 1 else H * sh), sh


def paged_latent_append(kv, weight, eps, cos_sin, positions, slot_mapping, cache, q_rope=None,
                        q_out=None, interleaved=False, err_word=None):
    """Append new tokens to a latent cache [NB, bs, R + P] fp16, in place: the
    RMS norm of kv[:, :R] (weight [R] fp16, or None) and the rotation of
    kv[:, R:] (cos_sin [max_positions, P] fp32, positions [T] int32) go to
    slot_mapping [T] int64.  kv [T, R + P] fp16, any stride between tokens.
    With q_rope [T, H, P] the position part of the queries is rotated into
    q_out [T, H, P] (both any strides between tokens and heads, e.g.
    q[..., d:] and absorbed[..., R:]; q_out may be q_rope)."""
    _need_cache(cache)
    dev = cache.device
    NB, bs, E = cache.shape
    _need_cuda(kv, "kv", torch.float16, dev)
    if kv.dim() != 2 or kv.shape[1] != E or (E > 1 and kv.stride(1) != 1):
        raise ValueError("kv must be [num_tokens, latent_dim + rope_dim], entries contiguous")
    T = kv.shape[0]
    _need(cos_sin, "cos_sin", torch.float32, dev)
    _need(positions, "positions", torch.int32, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if cos_sin.dim() != 2 or positions.shape != (T,) or slot_mapping.shape != (T,):
        raise ValueError("cos_sin must be [max_positions, rope_dim], positions and slot_mapping [T]")
    table, P = cos_sin.shape
    R = E - P
    if R <= 0:
        raise ValueError("cos_sin is as wide as the cache rows: no latent entries")
    if weight is not None:
        _need(weight, "weight", torch.float16, dev)
        if weight.shape != (R,):
            raise ValueError("weight must be [latent_dim]")
    if (q_rope is None) != (q_out is None):
        raise ValueError("q_rope and q_out go together")
    H, qs, os = 0, (0, 0), (0, 0)
    if q_rope is not None:
        for t, name in ((q_rope, "q_rope"), (q_out, "q_out")):
            _need_cuda(t, name, torch.float16, dev)
            if t.dim() != 3 or t.shape[0] != T or t.shape[2] != P:
                raise ValueError(f"{name} must be [num_tokens, n_q_heads, rope_dim]")
        if q_rope.shape != q_out.shape:
            raise ValueError("q_out must have q_rope's shape")
        H = q_rope.shape[1]
        qs, os = _strides(q_rope, "q_rope", P), _strides(q_out, "q_out", P)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    rc = _launch(dev, _lib().paged_latent_append, _ptr(kv), kv.stride(0) if T > 1 else E,
                 _ptr(weight), float(eps), _ptr(cos_sin), _ptr(positions), table,
                 int(bool(interleaved)), _ptr(slot_mapping), _ptr(cache), _ptr(q_rope), *qs,
                 _ptr(q_out), *os, H, T, R, P, bs, NB, _ptr(err_word))
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
    _need_cache(cache)
    dev = cache.device
    NB, bs, E = cache.shape
    _need(q, "q", torch.float16, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(context_lens, "context_lens", torch.int32, dev)
    if q.dim() != 3 or q.shape[2] != E:
        raise ValueError("q must be [total_q, n_q_heads, latent_dim + rope_dim]")
    TQ, H = q.shape[:2]
    R = int(latent_dim)
    if not 0 < R < E:
        raise ValueError("latent_dim must be positive and smaller than the cache rows")
    if block_tables.dim() != 2 or context_lens.shape != (block_tables.shape[0],):
        raise ValueError("block_tables must be [B, MB], context_lens [B]")
    B, MB = block_tables.shape
    if query_start is not None:
        _need(query_start, "query_start", torch.int32, dev)
        if query_start.shape != (B + 1,):
            raise ValueError("query_start must be [B + 1]")
    elif TQ != B or max_q_len != 1:
        raise ValueError("without query_start, q holds one token a sequence")
    mcl = 0 if max_context_len is None else int(max_context_len)
    if out is None:
        out = torch.empty((TQ, H, R), dtype=torch.float16, device=dev)
    else:
        _need(out, "out", torch.float16, dev)
        if out.shape != (TQ, H, R):
            raise ValueError("out must be [total_q, n_q_heads, latent_dim]")
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
        if lse.shape != (TQ, H):
            raise ValueError("lse must be [total_q, n_q_heads]")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    if workspace is None:
        ws = _plan_on(dev.index, B, TQ, max_q_len, H, R, E - R, bs, MB, mcl)
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    rc = _launch(dev, _lib().paged_latent_attention, _ptr(out), _ptr(q), _ptr(cache),
                 _ptr(block_tables), _ptr(context_lens), _ptr(query_start), B, TQ, int(max_q_len),
                 MB, NB, float(scale), H, R, E - R, bs, mcl, _ptr(workspace), workspace.numel(),
                 _ptr(lse), _ptr(err_word))
    _check("paged_latent_attention", rc)
    return out


def paged_latent_gather(cache, block_tables, start, total, latent_dim, latents=None, ropes=None,
                        err_word=None):
    """Cached rows in token order: rows [start[b], start[b + 1]) of the results
    are the first tokens of sequence b.  cache [NB, bs, R + P] fp16,
    block_tables [B, MB] and start [B + 1] int32, total: rows of the results.
    Returns (latents [total, R], ropes [total, P]) fp16."""
    _need_cache(cache)
    dev = cache.device
    NB, bs, E = cache.shape
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(start, "start", torch.int32, dev)
    R = int(latent_dim)
    if not 0 < R < E:
        raise ValueError("latent_dim must be positive and smaller than the cache rows")
    if block_tables.dim() != 2 or start.shape != (block_tables.shape[0] + 1,):
        raise ValueError("block_tables must be [B, MB], start [B + 1]")
    B, MB = block_tables.shape
    total = int(total)
    if latents is None:
        latents = torch.empty((total, R), dtype=torch.float16, device=dev)
    if ropes is None:
        ropes = torch.empty((total, E - R), dtype=torch.float16, device=dev)
    for t, name, w in ((latents, "latents", R), (ropes, "ropes", E - R)):
        _need(t, name, torch.float16, dev)
        if t.shape != (total, w):
            raise ValueError(f"{name} must be [total, {w}]")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    rc = _launch(dev, _lib().paged_latent_gather, _ptr(latents), _ptr(ropes), _ptr(cache),
                 _ptr(block_tables), _ptr(start), B, total, MB, NB, R, E - R, bs, _ptr(err_word))
    _check("paged_latent_gather", rc)
    return latents, ropes


def latent_prefill_attention(q, kv, k_rope, q_start, kv_start, scale, max_q_len, max_kv_len,
                             out=None, lse=None, err_word=None):
    """Causal attention of prompts over keys and values expanded from latents.

    q [total_q, H, d + P], kv [total_kv, H, 2 d] (key, then value), k_rope
    [total_kv, P], fp16; q_start, kv_start [B + 1] int32: each sequence's query
    rows and key rows (its queries are the newest tokens of its keys).
    max_q_len, max_kv_len: host bounds.  Returns out [total_q, H, d] fp16."""
    dev = q.device
    _need(q, "q", torch.float16)
    _need(kv, "kv", torch.float16, dev)
    _need(k_rope, "k_rope", torch.float16, dev)
    _need(q_start, "q_start", torch.int32, dev)
    _need(kv_start, "kv_start", torch.int32, dev)
    if q.dim() != 3 or kv.dim() != 3 or k_rope.dim() != 2 or kv.shape[1] != q.shape[1] or \
            kv.shape[0] != k_rope.shape[0] or kv.shape[2] != 2 * (q.shape[2] - k_rope.shape[1]):
        raise ValueError("q must be [total_q, H, d + P], kv [total_kv, H, 2 d], k_rope [total_kv, P]")
    TQ, H = q.shape[:2]
    TK, P = k_rope.shape
    d = q.shape[2] - P
    if q_start.dim() != 1 or q_start.numel() < 1 or kv_start.shape != q_start.shape:
        raise ValueError("q_start and kv_start must be [B + 1]")
    if out is None:
        out = torch.empty((TQ, H, d), dtype=torch.float16, device=dev)
    else:
        _need(out, "out", torch.float16, dev)
        if out.shape != (TQ, H, d):
            raise ValueError("out must be [total_q, H, d]")
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
        if lse.shape != (TQ, H):
            raise ValueError("lse must be [total_q, H]")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    rc = _launch(dev, _lib().latent_prefill_attention, _ptr(out), _ptr(q), _ptr(kv), _ptr(k_rope),
                 _ptr(q_start), _ptr(kv_start), q_start.numel() - 1, TQ, TK, int(max_q_len),
                 int(max_kv_len), float(scale), H, d, P, _ptr(lse), _ptr(err_word))
    _check("latent_prefill_attention", rc)
    return out
