"""The 8-bit caches with block scales on the GPU, where a batch's shape, values or tables
are at the edge of what the header allows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv

from q8_util import Paged, append64, assert_attention, attend64, values
from test_q8_gpu import KINDS, OnGpu, queries, same_state, starts, t

pytestmark = pytest.mark.gpu

NAN = 127  # an E4M3 code


# --- NaN --------------------------------------------------------------------

@pytest.mark.parametrize("news", [1, 5, 40])
@pytest.mark.parametrize("L", [17, 129, 257, 385, 401, 3009])
def test_a_cached_nan_in_a_part_of_its_own(news, L):
    """The key of the last token, alone in its tile, is NaN, or the keys of a whole tile:
    where a warp holds that tile alone it has no finite logit.  The queries that attend it
    are NaN, with their lse, those of the other sequence are not."""
    Hk, g, d = 1, 4, 128
    news = min(news, L)
    for tile in (L - 1) // 16, 0, 3:
        p = Paged([L, 40], Hk, d, 16, "e4m3", seed=L)
        at = min(tile, (L - 1) // 16)
        p.codes[0][p.tables[0, at], :, :, 7] = NAN
        gpu = OnGpu(p)
        q = queries(p, news + 1, Hk * g)
        out, lse = gpu.attend(t(q), 0.1, [news, 1])
        sees = L - news + np.arange(news) >= at * 16
        want = np.concatenate([sees, [False]])[:, None].repeat(Hk * g, 1)
        assert np.array_equal(np.isnan(lse), want), (tile, at)
        assert np.isnan(out[want]).all() and np.isfinite(out[~want]).all()
        gpu.near(1, q, out, lse, 0.1, starts([news, 1]))


@pytest.mark.parametrize("news", [1, 5, 40])
@pytest.mark.parametrize("L", [40, 385, 3009])
def test_a_nan_query_has_a_nan_lse(news, L):
    p = Paged([L, 90], 2, 128, 16, "int8", seed=4)
    q = queries(p, news + 1, 8)
    q[news - 1, 3, 9] = np.nan
    out, lse = OnGpu(p).attend(t(q), 0.1, [news, 1])
    want = np.zeros(lse.shape, bool)
    want[news - 1, 3] = True
    assert np.array_equal(np.isnan(lse), want)
    assert np.array_equal(np.isnan(out), want[..., None].repeat(128, 2))


# --- steps without a wait between them ----------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("news,bs", [(1, 16), (1, 256), (3, 16), (3, 64), (12, 16), (12, 128)])
def test_flagged_attention_right_behind_an_append_that_grows_scales(kind, news, bs):
    """Steps of append (each with larger tokens than the blocks hold, so that scales grow
    and held codes are written anew) and attention under PKV_TABLES_READY, one behind the
    other in a stream and in a replayed graph: every step's results, and the cache in the
    end, by the definitions."""
    Hk, g, d, steps = 2, 4, 128, 8
    held = [0, 3, 15, 100, 40, 700, 17, 250]
    B = len(held)
    p = Paged([m + news * steps for m in held], Hk, d, bs, kind, seed=news + bs)
    first = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    kv = [x.clone() for x in first]
    gain = 2.0 ** np.arange(steps)
    x = [[(gain[i] * p.rng.standard_normal((B * news, Hk, d))).astype(np.float16) for _ in "kv"] for i in range(steps)]
    q = [queries(p, B * news, Hk * g) for _ in range(steps)]
    lens = [[m + news * (i + 1) for m in held] for i in range(steps)]
    at = starts([news] * B)
    many = {} if news == 1 else dict(query_start=t(at), max_q_len=news)
    ws = torch.zeros(pkv.q8_plan(B, B * news, news, Hk * g, Hk, d, bs, p.MB), dtype=torch.uint8, device="cuda")
    tables, err = t(p.tables), torch.zeros(1, dtype=torch.int32, device="cuda")
    tx, tq = [[t(y) for y in pair] for pair in x], [t(y) for y in q]
    tl = [t(np.array(y, np.int32)) for y in lens]
    out = [torch.empty_like(y) for y in tq]
    lse = [torch.empty(y.shape[:2], device="cuda") for y in tq]
    scale = 0.002

    def chain():
        for i in range(steps):
            pkv.paged_kv_append_q8(*tx[i], *kv, tables, tl[i], err_word=err, **many)
            pkv.paged_decode_attention_q8(tq[i], *kv, tables, tl[i], scale, out=out[i], lse=lse[i], workspace=ws,
                                          err_word=err, flags=pkv.PKV_TABLES_READY, **many)

    def results():
        torch.cuda.synchronize()
        assert pkv.get_error(err) == 0
        return [[y.view(torch.uint8).cpu().numpy() for y in group] for group in (out, lse, kv)]

    chain()
    eager = results()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            chain()
        for _ in range(3):
            for a, b in zip(kv, first):
                a.copy_(b)
            graph.replay()
            again = results()
            for a, b in zip(eager, again):
                assert all(np.array_equal(y, z) for y, z in zip(a, b))
    keys = 64 if news * g > 32 else 16
    for i in range(steps):
        for side in range(2):
            append64(kind, x[i][side], at, lens[i], p.tables, p.codes[side], p.scales[side])
        o, e = out[i].cpu().numpy(), lse[i].cpu().numpy()
        for b, L in enumerate(lens[i]):
            rows = slice(at[b], at[b + 1])
            k, v = (p.tokens(s, b, L) for s in range(2))
            ref = attend64(q[i][rows], k, v, scale, p.spread_in_steps(b, L, keys))
            assert_attention(o[rows], e[rows], ref, f"step {i}, sequence {b}")
    same_state(p, kv)


# --- starts that decrease -------------------------------------------------------

def _append_with(p, start, total, most, kind):
    """Appends with these starts to a copy of p's tensors (five times, each the same), and
    to p by the definition: sequences in bounds alone."""
    x = [p.rng.standard_normal((total, *p.codes[0].shape[1::2])).astype(np.float16) for _ in "kv"]
    first = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    for side in range(2):
        for b, (s, e) in enumerate(zip(start[:-1], start[1:])):
            L = int(p.lens[b])
            if 0 <= s <= e <= total and e - s <= min(most, L) and L <= p.MB * p.codes[0].shape[2]:
                append64(kind, x[side], [s, e], [L], p.tables[b:b + 1], p.codes[side], p.scales[side])
    for _ in range(5):
        kv, err = [y.clone() for y in first], torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.paged_kv_append_q8(t(x[0]), t(x[1]), *kv, t(p.tables), t(p.lens.astype(np.int32)),
                               query_start=t(np.array(start, np.int32)), max_q_len=most, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT
        same_state(p, kv)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs,start", [
    (16, [0, 200, 100, 200]),
    (16, [0, 150, 40, 90, 10, 200, 200]),
    (64, [50, 200, 0, 60, 300, 10]),
    (128, [100, 0, 150, 20, 199, -1, 3]),
    (256, [0, 200, 0, 200, 0, 200]),
])
def test_sequences_in_bounds_are_written_where_others_are_not(kind, bs, start):
    """Starts that decrease, so that several sequences have rows in common, and entries that
    are out of bounds: those sequences are flagged and nothing of them is written; all
    others are, the same each time."""
    p = Paged([230 + 7 * b for b in range(len(start) - 1)], 3, 64, bs, kind, seed=bs)
    _append_with(p, start, 200, 200, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("most", [1, 2, 40])
def test_many_sequences_in_no_order(kind, most):
    rng = np.random.default_rng(most)
    B, total = 400, 300
    start = rng.integers(0, total, B + 1)
    start[1::2] = np.minimum(start[::2][:B // 2] + rng.integers(0, most + 2, B // 2), total + 2)
    p = Paged(rng.integers(1, 90, B), 2, 128, 16, kind, seed=most)
    p.lens[::37] = 10 ** 6
    _append_with(p, start, total, most, kind)


@pytest.mark.parametrize("news", [[3, 0, 2], [1, 0, 1]])
@pytest.mark.parametrize("length", [-1, 49, 10 ** 6])
def test_a_length_out_of_bounds_is_flagged_without_new_tokens_too(news, length):
    """In the kernel for single tokens and in the one for several; the others are written."""
    p = Paged([40, 20, 41], 2, 64, 16, "int8", seed=5)
    x = [p.rng.standard_normal((sum(news), 2, 64)).astype(np.float16) for _ in "kv"]
    kv, lens = [t(c) for c in p.codes] + [t(s) for s in p.scales], np.array([40, length, 41], np.int32)
    for side in range(2):
        append64("int8", x[side], starts(news), p.lens, p.tables, p.codes[side], p.scales[side])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_kv_append_q8(t(x[0]), t(x[1]), *kv, t(p.tables), t(lens), query_start=t(starts(news)),
                           max_q_len=max(news), err_word=err)
    assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT
    same_state(p, kv)


# --- plans ----------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
def test_a_plan_never_falls_as_its_sizes_grow(d):
    def plan(**change):
        base = dict(num_seqs=9, total_q=300, max_q_len=1, n_q_heads=8, n_kv_heads=2, head_dim=d, block_size=16,
                    max_blocks_per_seq=500, max_context_len=700)
        return pkv.q8_plan(**{**base, **change})

    for name, values in (("max_q_len", range(1, 301)), ("total_q", range(1, 301)), ("num_seqs", range(1, 60)),
                         ("max_context_len", range(1, 8000, 61)), ("n_q_heads", range(2, 257, 2))):
        for other in ({}, dict(max_q_len=5), dict(max_q_len=40)):
            if name == "total_q":
                other = dict(max_q_len=300)
            got = [plan(**{**other, name: v}) for v in values]
            assert got == sorted(got), (name, other)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g,most", [(4, 5), (4, 8), (1, 17), (8, 16), (2, 33)])
def test_a_workspace_for_the_largest_call_serves_smaller_ones(kind, g, most):
    Hk, d = 2, 128
    p = Paged([700, 90, 333], Hk, d, 16, kind, seed=most)
    gpu = OnGpu(p)
    ws = torch.zeros(pkv.q8_plan(3, 3 * most, most, Hk * g, Hk, d, 16, p.MB), dtype=torch.uint8, device="cuda")
    for n in range(1, most + 1):
        gpu.check(queries(p, 3 * n, Hk * g), 0.1, [n] * 3, workspace=ws)
        if n == 1:
            gpu.check(queries(p, 3, Hk * g), 0.1, workspace=ws)


# --- scales at the ends of their range ---------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("news", [1, 5, 40])
@pytest.mark.parametrize("large", ["zeros", "values"])
def test_v_scales_from_the_least_to_the_largest(kind, d, news, large):
    """Blocks of 64 tokens (a step of the kernel for many rows) of V scale 2^64 and 2^-100 next
    to ordinary ones, in many orders.  Where the large ones hold zeros the result is that
    of the others; where they hold numbers it is infinite and of the right sign."""
    Hk, g, bs, n = 2, 4, 64, 12
    p = Paged([n * bs] * 8 + [50 * bs], Hk, d, bs, kind, seed=d + news)
    tiny, huge = np.float32(2.0 ** -100), np.float32(2.0 ** 64)
    for b in range(9):
        for j in range(n):
            ids = p.tables[b, j]
            pick = p.rng.integers(0, 4)
            if pick == 0:
                p.scales[1][ids] = tiny
            elif pick == 1:
                p.scales[1][ids] *= np.float32(2.0 ** -12)
            elif pick == 2 and large == "zeros":
                p.scales[1][ids] = huge
                p.codes[1][ids] = 0
    if large == "values":  # one block: sums of one sign or the other in each column
        for b in range(8):
            p.scales[1][p.tables[b, b]] = huge
            p.codes[1][p.tables[b, b]] = np.abs(p.codes[1][p.tables[b, b]].astype(np.int16) % 100) + 1
            if kind == "e4m3":
                p.codes[1][p.tables[b, b], :, :, ::2] |= 128
            else:
                p.codes[1][p.tables[b, b], :, :, ::2] *= -1
    times = 40  # the same sequences again and again, so that a warp goes through several blocks
    p.tables, p.lens = np.tile(p.tables, (times, 1)), np.tile(p.lens, times)
    gpu = OnGpu(p)
    B = len(p.lens)
    q, at = queries(p, B * news, Hk * g), starts([news] * B)
    out, lse = gpu.attend(t(q), 0.1, None if news == 1 else [news] * B)
    gpu.keys = 64 if news * g > 32 else 16
    for b in range(0, B, 7 if news == 1 else 31):
        if large == "zeros" or b % 9 == 8:
            gpu.near(b, q, out, lse, 0.1, at)
    if large == "values":
        want = np.full((news, Hk * g, d), np.inf)
        want[..., ::2] = -np.inf
        for b in range(B):
            if b % 9 < 8:
                assert np.array_equal(out[at[b]:at[b + 1]].astype(np.float64), want), b
        assert np.isfinite(lse).all()


# --- the read-back's roundings ------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_read_back_rounds_to_fp32_and_then_to_fp16(kind):
    """Every code at scales for some of whose products the two roundings end elsewhere than
    one would, and at others."""
    d, bs, n = 64, 16, 40
    p = Paged([n * bs], 1, d, bs, kind, seed=1)
    codes = np.array([c for c in range(256) if not (kind == "e4m3" and c & 127 == 127)]).astype(p.codes[0].dtype)
    p.codes[0][:] = np.resize(codes, (bs, d))
    some = np.exp2(p.rng.uniform(-20, 5, 200000)).astype(np.float32)
    products = values(kind, codes) * some.astype(np.float64)[:, None]
    apart = products.astype(np.float32).astype(np.float16) != products.astype(np.float16)
    few = some[apart.any(1)][:n // 2]
    p.scales[0][:] = p.rng.permutation(np.concatenate([few, some[:p.NB - len(few)]]))[:, None]
    want = p.tokens(0, 0, n * bs)
    twice, once = want.astype(np.float32).astype(np.float16), want.astype(np.float16)
    assert (twice != once).sum() >= 10
    k, _ = pkv.paged_kv_gather_q8(*OnGpu(p).kv, t(p.tables), t(starts([n * bs])), n * bs)
    assert np.array_equal(k.cpu().numpy().view(np.uint16), twice.view(np.uint16))
