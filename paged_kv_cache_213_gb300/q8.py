"""ctypes binding of the 8-bit caches with block scales (``include/pagedkv_q8.h``).
Marshalling only; the work is in the library's CUDA kernels.

Caches are [num_blocks, n_kv_heads, block_size, head_dim], uint8 (E4M3 codes) or
int8, with k_scales and v_scales [num_blocks, n_kv_heads] fp32."""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import _check, _need, library
from .rope import (_F16, _F32, _I32, _U8, _at, _at_strided, _current_device, _launch, _native,
                   _token_stride)

_KINDS = {torch.uint8: 0, torch.int8: 1}  # PKV_Q8_E4M3, PKV_Q8_INT8

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = library()
        c = ctypes
        p, i, l, f, z = c.c_void_p, c.c_int, c.c_int64, c.c_float, c.c_size_t
        lib.paged_kv_append_q8.argtypes = [p, p, l, l, p, p, p, i, i, i, i, p, p, p, p, i, i, i, i,
                                           l, p, p]
        lib.paged_kv_append_q8.restype = i
        lib.paged_decode_q8_plan.argtypes = [i] * 9 + [c.POINTER(z)]
        lib.paged_decode_q8_plan.restype = i
        lib.paged_decode_attention_q8.argtypes = [p, p, l, p, p, p, p, i, p, p, p, i, i, i, i, l, f,
                                                  i, i, i, i, i, p, z, p, p, p, c.c_uint32]
        lib.paged_decode_attention_q8.restype = i
        lib.paged_kv_gather_q8.argtypes = [p, p, p, p, p, p, i, p, p, i, l, i, l, i, i, i, p, p]
        lib.paged_kv_gather_q8.restype = i
        lib.paged_kv_copy_blocks_q8.argtypes = [p, p, p, p, p, p, p, i, i, i, i, l, p, p]
        lib.paged_kv_copy_blocks_q8.restype = i
        _bound = lib
    return _bound


def _cache(k_cache, v_cache, k_scales, v_scales):
    """(device, addresses of the four, kind, blocks, KV heads, block size, head size)."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    if k_cache.dtype not in _KINDS:
        raise TypeError(f"k_cache must be torch.uint8 (E4M3) or torch.int8, got {k_cache.dtype}")
    _need(k_cache, "k_cache", k_cache.dtype)
    dev = k_cache.device
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache/v_cache must both be [num_blocks, n_kv_heads, block_size, head_dim]")
    vp = _at(v_cache, "v_cache", k_cache.dtype, dev)
    ks, vs = _at(k_scales, "k_scales", _F32, dev), _at(v_scales, "v_scales", _F32, dev)
    if k_scales.shape != shape[:2] or v_scales.shape != shape[:2]:
        raise ValueError("k_scales/v_scales must be [num_blocks, n_kv_heads]")
    return dev, (k_cache.data_ptr(), vp, ks, vs), _KINDS[k_cache.dtype], *shape


def _tables(block_tables, context_lens, query_start, total, max_q_len, dev):
    """(addresses of tables, lengths and query starts, sequences, blocks a sequence)."""
    tables = _at(block_tables, "block_tables", _I32, dev)
    lens = _at(context_lens, "context_lens", _I32, dev)
    shape = block_tables.shape
    if len(shape) != 2 or context_lens.shape != (shape[0],):
        raise ValueError("block_tables must be [B, MB], context_lens [B]")
    B, MB = shape
    start = None
    if query_start is not None:
        start = _at(query_start, "query_start", _I32, dev)
        if query_start.shape != (B + 1,):
            raise ValueError("query_start must be [B + 1]")
    elif total != B or max_q_len != 1:
        raise ValueError("without query_start there is one token a sequence")
    return tables, lens, start, B, MB


def paged_kv_append_q8(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables,
                       context_lens, query_start=None, max_q_len=1, err_word=None):
    """Quantise each sequence's newest tokens into its blocks, in place.

    k_new, v_new [T, Hk, d] fp16: a token's heads contiguous, any stride between
    tokens.  block_tables [B, MB] and context_lens [B] int32, the new tokens
    included.  query_start [B + 1] int32: sequence b's new tokens are the rows
    [query_start[b], query_start[b + 1]) and go to its last positions (max_q_len
    bounds their number); None: one token a sequence.  A block's scale covers what
    the call and the calls before put into it: it is set when the block's first
    tokens come, and doubled as often as a later token needs."""
    if _native().append_q8(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables,
                           context_lens, query_start, max_q_len, err_word):
        return
    dev, cache, kind, NB, Hk, bs, d = _cache(k_cache, v_cache, k_scales, v_scales)
    kp = _at_strided(k_new, "k_new", _F16, dev)
    vp = _at_strided(v_new, "v_new", _F16, dev)
    shape = k_new.shape
    if len(shape) != 3 or shape[1:] != (Hk, d) or v_new.shape != shape:
        raise ValueError("k_new/v_new must be [num_tokens, n_kv_heads, head_dim]")
    T = shape[0]
    max_q_len = int(max_q_len)
    tables, lens, start, B, MB = _tables(block_tables, context_lens, query_start, T, max_q_len, dev)
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().paged_kv_append_q8, kp, vp, _token_stride(k_new, "k_new", T, Hk, d),
                 _token_stride(v_new, "v_new", T, Hk, d), start, tables, lens, B, T, max_q_len, MB,
                 *cache, kind, Hk, d, bs, NB, err)
    _check("paged_kv_append_q8", rc)


def q8_plan(num_seqs, total_q, max_q_len, n_q_heads, n_kv_heads, head_dim, block_size,
            max_blocks_per_seq, max_context_len=0):
    """Workspace bytes of paged_decode_attention_q8 on the current device, for calls of
    these sizes and of smaller ones."""
    W = ctypes.c_size_t(0)
    _check("paged_decode_q8_plan",
           _lib().paged_decode_q8_plan(num_seqs, total_q, max_q_len, n_q_heads, n_kv_heads,
                                       head_dim, block_size, max_blocks_per_seq, max_context_len,
                                       ctypes.byref(W)))
    return W.value


@functools.lru_cache(maxsize=4096)
def _plan_on(index, *sizes):
    """q8_plan on device `index`: a function of the sizes alone."""
    if _current_device() == index:
        return q8_plan(*sizes)
    with torch.cuda.device(index):
        return q8_plan(*sizes)


def paged_decode_attention_q8(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                              scale, query_start=None, max_q_len=1, max_context_len=None, out=None,
                              workspace=None, lse=None, err_word=None, flags=0):
    """softmax(q K^T * scale) V over each sequence's 8-bit K/V -> out [T, H, d] fp16.

    q [T, H, d] fp16: a token's heads contiguous, any stride between tokens.
    block_tables [B, MB] and context_lens [B] int32.  query_start [B + 1] int32:
    sequence b owns the rows [query_start[b], query_start[b + 1]), its newest
    tokens (causal; max_q_len bounds their number); None: one token a sequence.
    lse: optional fp32 [T, H] output.  workspace: uint8, q8_plan bytes, zero-filled
    before its first use (calls leave it ready for the next); None: a new one.
    flags: 0 or PKV_TABLES_READY."""
    done = _native().attention_q8(q, k_cache, v_cache, k_scales, v_scales, block_tables,
                                  context_lens, scale, query_start, max_q_len,
                                  0 if max_context_len is None else max_context_len, out,
                                  workspace, lse, err_word, flags)
    if done is not None:
        return done
    dev, cache, kind, NB, Hk, bs, d = _cache(k_cache, v_cache, k_scales, v_scales)
    qp = _at_strided(q, "q", _F16, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d or Hk == 0 or shape[1] % Hk:
        raise ValueError("q must be [total_q, n_q_heads, head_dim], n_q_heads a multiple of n_kv_heads")
    TQ, H, _ = shape
    max_q_len = int(max_q_len)
    tables, lens, start, B, MB = _tables(block_tables, context_lens, query_start, TQ, max_q_len, dev)
    mcl = 0 if max_context_len is None else int(max_context_len)
    if out is None:
        out = torch.empty((TQ, H, d), dtype=_F16, device=dev)
        op = out.data_ptr()
    else:
        op = _at(out, "out", _F16, dev)
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    lp = None
    if lse is not None:
        lp = _at(lse, "lse", _F32, dev)
        if lse.shape != (TQ, H):
            raise ValueError("lse must be [total_q, n_q_heads]")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    if workspace is None:
        size = _plan_on(dev.index, B, TQ, max_q_len, H, Hk, d, bs, MB, mcl)
        # zero-filled: it starts with arrival counters
        workspace = torch.zeros(size, dtype=_U8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp = _at(workspace, "workspace", _U8, dev)
        size = workspace.numel()
    stride = _token_stride(q, "q", TQ, H, d)

    def call(*args):  # flags come behind the stream
        return _lib().paged_decode_attention_q8(*args, int(flags))

    rc = _launch(dev, call, op, qp, stride, *cache, kind, tables, lens, start, B, TQ, max_q_len, MB,
                 NB, float(scale), H, Hk, d, bs, mcl, wp, size, lp, err)
    _check("paged_decode_attention_q8", rc)
    return out


def paged_kv_gather_q8(k_cache, v_cache, k_scales, v_scales, block_tables, start, total, k=None,
                       v=None, err_word=None):
    """Cached tokens back in fp16, in token order: rows [start[b], start[b + 1])
    of the results are the first tokens of sequence b.  block_tables [B, MB] and
    start [B + 1] int32, total: rows of the results.  Returns (k, v), both
    [total, Hk, d]."""
    done = _native().gather_q8(k_cache, v_cache, k_scales, v_scales, block_tables, start, total, k,
                               v, err_word)
    if done is not None:
        return done
    dev, cache, kind, NB, Hk, bs, d = _cache(k_cache, v_cache, k_scales, v_scales)
    tables = _at(block_tables, "block_tables", _I32, dev)
    first = _at(start, "start", _I32, dev)
    shape = block_tables.shape
    if len(shape) != 2 or start.shape != (shape[0] + 1,):
        raise ValueError("block_tables must be [B, MB], start [B + 1]")
    B, MB = shape
    total = int(total)
    if total < 0:
        raise ValueError("total must not be negative")
    if k is None:
        k = torch.empty((total, Hk, d), dtype=_F16, device=dev)
    if v is None:
        v = torch.empty((total, Hk, d), dtype=_F16, device=dev)
    kp, vp = _at(k, "k", _F16, dev), _at(v, "v", _F16, dev)
    if k.shape != (total, Hk, d) or v.shape != (total, Hk, d):
        raise ValueError("k and v must be [total, n_kv_heads, head_dim]")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().paged_kv_gather_q8, kp, vp, *cache, kind, tables, first, B, total, MB,
                 NB, Hk, d, bs, err)
    _check("paged_kv_gather_q8", rc)
    return k, v


def paged_kv_copy_blocks_q8(k_cache, v_cache, k_scales, v_scales, src, dst, tokens=None,
                            err_word=None):
    """Copy rows [0, tokens[i]) (all rows if None) and the scales of block src[i]
    to dst[i], all KV heads, in both caches, on the current stream (int32 tensors
    of one length)."""
    dev, cache, _, NB, Hk, bs, d = _cache(k_cache, v_cache, k_scales, v_scales)
    sp, dp = _at(src, "src", _I32, dev), _at(dst, "dst", _I32, dev)
    tp = None if tokens is None else _at(tokens, "tokens", _I32, dev)
    n = src.numel()
    if dst.numel() != n or (tokens is not None and tokens.numel() != n):
        raise ValueError("src, dst, tokens must have the same length")
    err = None if err_word is None else _at(err_word, "err_word", _I32, dev)
    rc = _launch(dev, _lib().paged_kv_copy_blocks_q8, *cache, sp, dp, tp, n, Hk, d, bs, NB, err)
    _check("paged_kv_copy_blocks_q8", rc)
