"""The latent cache's operators against their 64-bit statements: append,
absorbed attention, gather, expanded attention, and a run of them together."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from latent_util import (Paged, assert_attention, assert_once_rounded, attend64, norm64, table,
                         turn64)
from paged_kv_cache_213_gb300.blocks import paged_kv_copy_blocks

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.library()


def _t(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# --- append ------------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,R,P,bs,norm", [
    (1, 1, 512, 64, 16, True), (9, 16, 512, 64, 64, False), (21, 3, 256, 64, 16, True),
    (5, 0, 512, 64, 32, True), (4, 33, 1024, 128, 16, True), (3, 5, 24, 16, 1, True),
    (2, 2, 8, 48, 16, True), (70, 128, 512, 64, 128, True)])
def test_latent_append(T, H, R, P, bs, norm, interleaved):
    rng = np.random.default_rng(T + H + R)
    wide = rng.standard_normal((T, R + P + 8)).astype(np.float16)
    w = (1 + 0.2 * rng.standard_normal(R)).astype(np.float16) if norm else None
    cs, pos = table(P, 300), rng.integers(0, 300, T).astype(np.int32)
    NB = -(-T // bs) + 2
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    cache = rng.standard_normal((NB, bs, R + P)).astype(np.float16)
    q = rng.standard_normal((T, H, 40 + P)).astype(np.float16)
    o = rng.standard_normal((T, H, R + P)).astype(np.float16)
    c, qo, err = _t(cache), _t(o), _err()
    pkv.paged_latent_append(_t(wide)[:, :R + P], _t(w), EPS, _t(cs), _t(pos), _t(slots), c,
                            q_rope=_t(q)[..., 40:] if H else None,
                            q_out=qo[..., R:] if H else None, interleaved=interleaved,
                            err_word=err)
    assert pkv.get_error(err) == 0
    got = c.cpu().numpy()
    n = norm64(wide[:, :R], w, EPS)
    r, mag = turn64(wide[:, None, R:R + P].astype(np.float64), cs[pos], interleaved)
    flat = got.reshape(-1, R + P)
    assert_once_rounded(flat[slots, :R], n, np.abs(n), "latent")
    assert_once_rounded(flat[slots, R:], r[:, 0], mag[:, 0], "rope")
    others = np.setdiff1d(np.arange(NB * bs), slots)
    assert np.array_equal(flat[others], cache.reshape(-1, R + P)[others])
    if H:
        y, mag = turn64(q[..., 40:].astype(np.float64), cs[pos], interleaved)
        assert_once_rounded(qo.cpu().numpy()[..., R:], y, mag, "q")
        assert np.array_equal(qo.cpu().numpy()[..., :R], o[..., :R])


def test_latent_append_bad_tokens_and_in_place():
    T, H, R, P, bs = 6, 4, 512, 64, 16
    rng = np.random.default_rng(5)
    kv = rng.standard_normal((T, R + P)).astype(np.float16)
    cs = table(P, 50)
    pos = np.array([0, 1, 50, 3, -1, 49], np.int32)
    slots = np.array([3, -1, 5, 32, 7, 8], np.int64)
    q = rng.standard_normal((T, H, P)).astype(np.float16)
    qd, err = _t(q), _err()
    c = torch.zeros(2, bs, R + P, dtype=torch.float16, device="cuda")
    pkv.paged_latent_append(_t(kv), None, EPS, _t(cs), _t(pos), _t(slots), c, q_rope=qd, q_out=qd,
                            err_word=err)
    assert pkv.get_error(err) == pkv.PKV_ERRBIT_SLOT | pkv.PKV_ERRBIT_POSITION
    flat = c.cpu().numpy().reshape(-1, R + P)
    assert np.array_equal(flat[[3, 8], :R], kv[[0, 5], :R])
    assert not np.any(np.delete(flat, [3, 8], 0))
    y, mag = turn64(q.astype(np.float64), cs[np.clip(pos, 0, 49)], False)
    got = qd.cpu().numpy()
    assert_once_rounded(got[[0, 5]], y[[0, 5]], mag[[0, 5]], "q in place")
    assert np.array_equal(got[1:5], q[1:5])


# --- absorbed attention --------------------------------------------------------

def _problem(lens, nq, H, R, bs, seed, spread=1.7):
    p = Paged(lens, R, 64, bs, seed)
    rng = np.random.default_rng(seed + 1)
    qs = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = rng.standard_normal((int(qs[-1]), H, R + 64)).astype(np.float16)
    return p, q, qs, spread / np.sqrt(R + 64)


def _attend(p, q, qs, scale, nq, out=None, **kw):
    err = _err()
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    if out is None:
        out = torch.full((*q.shape[:2], p.R), 7.0, dtype=torch.float16, device="cuda")
    pkv.paged_latent_attention(_t(q), _t(p.cache), _t(p.tables), _t(p.lens.astype(np.int32)),
                               scale, p.R, query_start=None if qs is None else _t(qs),
                               max_q_len=max(1, max(nq)), out=out, lse=lse, err_word=err,
                               **{"max_context_len": int(max(1, p.lens.max())), **kw})
    return out.cpu().numpy(), lse.cpu().numpy(), pkv.get_error(err)


def _check(p, q, qs, scale, nq, what, got=None, skip=()):
    out, lse, bits = _attend(p, q, qs, scale, nq) if got is None else got
    if got is None:
        assert bits == 0, what
    for b, n in enumerate(nq):
        if n == 0 or b in skip:
            continue
        L, r = int(p.lens[b]), slice(int(qs[b]), int(qs[b + 1]))
        ref = attend64(q[r], p.rows[b], p.rows[b][:, :p.R], L - n + np.arange(n) + 1, scale)
        assert_attention(out[r], lse[r], *ref, f"{what}: sequence {b}")


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("H", [1, 5, 16, 20, 40, 72, 128])
def test_decode(H, bs, R):
    lens = [1, 15, 16, 17, 63, 64, 65, 127, 200, 129]
    p, q, qs, scale = _problem(lens, [1] * len(lens), H, R, bs, H + bs + R)
    _check(p, q, qs, scale, [1] * len(lens), "decode")


@pytest.mark.parametrize("H,nq", [(16, [1, 3, 0, 8, 2]), (7, [9, 1, 1, 0, 33]),
                                  (128, [2, 1, 4, 1, 3]), (1, [100, 1, 0, 7, 65])])
def test_several_tokens(H, nq):
    lens = [150, 3, 70, 8, 333]
    nq = [min(n, m) for n, m in zip(nq, lens)]
    p, q, qs, scale = _problem(lens, nq, H, 512, 32, 40 + H)
    _check(p, q, qs, scale, nq, "several tokens")


@pytest.mark.parametrize("H", [16, 128])
def test_long_contexts_are_split_and_joined(H):
    lens = [9000, 1, 4097, 20]
    p, q, qs, scale = _problem(lens, [1] * 4, H, 512, 64, 50 + H)
    _check(p, q, qs, scale, [1] * 4, "long")


@pytest.mark.parametrize("B", [1, 40, 700])
def test_many_and_few_sequences(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 90, B)
    p, q, qs, scale = _problem(lens, [1] * B, 8, 512, 16, 60 + B)
    _check(p, q, qs, scale, [1] * B, "batch")


@pytest.mark.parametrize("spread", [0.0, 60.0, -1.7, -40.0])
def test_flat_and_peaked_weights(spread):
    """All weights equal (scale 0), one weight near 1 with logits far apart, and
    negative scales."""
    lens = [300, 77, 1, 129]
    p, q, qs, scale = _problem(lens, [1] * 4, 16, 512, 16, 70, spread)
    _check(p, q, qs, scale, [1] * 4, "peaked")


@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_rising_logits(H):
    """Keys that grow along the sequence: the running maximum moves in every tile."""
    lens = [900]
    p, q, qs, scale = _problem(lens, [1], H, 512, 16, 71)
    grow = np.linspace(0.01, 3.0, 900)[:, None]
    sign = np.sign(q[0, 0].astype(np.float64))
    p.rows[0] = (grow * sign * np.abs(p.rows[0])).astype(np.float16)
    t = np.arange(900)
    p.cache[p.tables[0, t // 16], t % 16] = p.rows[0]
    _check(p, q, qs, scale, [1], "rising")


def test_decode_form_with_an_empty_sequence():
    """Without query_start a context length of 0 gives out 0 and lse -inf."""
    p, q, qs, scale = _problem([20, 0, 130], [1, 1, 1], 16, 512, 16, 80)
    out, lse, bits = _attend(p, q, None, scale, [1])
    assert bits == 0 and not np.any(out[1]) and np.all(np.isneginf(lse[1]))
    _check(p, q, qs, scale, [1, 0, 1], "empty", (out, lse, bits))


def test_all_sequences_empty():
    p, q, qs, scale = _problem([0, 0], [1, 1], 16, 512, 16, 81)
    out, lse, bits = _attend(p, q, None, scale, [1])
    assert bits == 0 and not np.any(out) and np.all(np.isneginf(lse))


def test_bad_sequences_are_flagged_and_left_unwritten():
    """More tokens than cached, a length beyond the table, more tokens than
    max_q_len: flagged, rows as they were; the other sequences are right."""
    nq = [2, 1, 1, 3]
    p, q, qs, scale = _problem([50, 30, 40, 64], nq, 16, 512, 16, 90)
    keep = p.lens.copy()
    p.lens = np.array([1, 30, p.MB * 16 + 1, 64])
    out, lse, bits = _attend(p, q, qs, scale, [2], max_context_len=64)
    assert bits == pkv.PKV_ERRBIT_CONTEXT
    for r in (slice(0, 2), slice(3, 4), slice(4, 7)):
        assert np.all(out[r] == 7.0) and np.all(lse[r] == 7.0)
    p.lens = keep
    _check(p, q, qs, scale, nq, "bad", (out, lse, bits), skip=(0, 2, 3))


def test_a_bad_block_id_is_flagged():
    p, q, qs, scale = _problem([100, 100], [1, 1], 16, 512, 16, 91)
    p.tables[0, 3] = p.NB
    out, lse, bits = _attend(p, q, qs, scale, [1, 1])
    assert bits == pkv.PKV_ERRBIT_BLOCK_ID
    _check(p, q, qs, scale, [1, 1], "bad id", (out, lse, bits), skip=(0,))


def test_repeated_calls_are_bit_identical_and_graph_replay():
    """One workspace over calls of other shapes; captured once and replayed on
    changed lengths, with the maximum as the host's bound."""
    p, q, qs, scale = _problem([700, 1300, 5, 90], [1] * 4, 32, 512, 32, 92)
    one = _attend(p, q, qs, scale, [1])
    ws = torch.randint(0, 256, (pkv.latent_plan(4, 4, 1, 32, 512, 64, 32, p.MB, 1300) + 4096,),
                       dtype=torch.uint8, device="cuda")
    two = _attend(p, q, qs, scale, [1], workspace=ws)
    assert np.array_equal(one[0], two[0]) and np.array_equal(one[1], two[1])
    args = [_t(x) for x in (q, p.cache, p.tables, p.lens.astype(np.int32))]
    out = torch.zeros(4, 32, 512, dtype=torch.float16, device="cuda")
    lse = torch.zeros(4, 32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_latent_attention(*args, scale, 512, max_context_len=1300, out=out, lse=lse,
                                   workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), one[0])
    short = np.array([33, 1, 5, 64])
    args[3].copy_(_t(short.astype(np.int32)))
    g.replay()
    torch.cuda.synchronize()
    p.rows = [x[:n] for x, n in zip(p.rows, short)]
    p.lens = short
    _check(p, q, qs, scale, [1] * 4, "replayed", (out.cpu().numpy(), lse.cpu().numpy(), 0))


def test_two_streams_at_once_and_other_than_the_inputs():
    """Two calls in flight on two streams, each with its own workspace, on tensors
    that a third stream made."""
    a = _problem([3000, 40], [1, 1], 16, 512, 16, 95)
    b = _problem([2000, 900], [1, 1], 128, 512, 64, 96)
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    made = []
    for p, q, qs, scale in (a, b):
        made.append([_t(x) for x in (q, p.cache, p.tables, p.lens.astype(np.int32))])
    torch.cuda.synchronize()
    for rep in range(3):
        outs = []
        for (p, q, qs, scale), t, s in zip((a, b), made, streams):
            with torch.cuda.stream(s):
                lse = torch.empty(q.shape[:2], device="cuda")
                outs.append((pkv.paged_latent_attention(*t, scale, 512, lse=lse), lse))
    torch.cuda.synchronize()
    for (p, q, qs, scale), (o, l) in zip((a, b), outs):
        _check(p, q, qs, scale, [1, 1], "streams", (o.cpu().numpy(), l.cpu().numpy(), 0))


def test_shared_blocks_and_one_block_twice():
    """Two sequences that share leading blocks, and one whose table names a block
    twice."""
    p, q, qs, scale = _problem([64, 50, 48], [1, 1, 1], 16, 512, 16, 97)
    p.tables[1, :2] = p.tables[0, :2]
    p.rows[1] = np.concatenate([p.rows[0][:32], p.rows[1][32:]])
    p.tables[2, 1] = p.tables[2, 0]
    p.rows[2] = np.concatenate([p.rows[2][:16], p.rows[2][:16], p.rows[2][32:]])
    _check(p, q, qs, scale, [1, 1, 1], "shared")


def test_caches_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes and 2^31 values: append, gather and attention on
    its last blocks."""
    R, P, bs, NB = 512, 64, 64, 60000
    E = R + P
    assert NB * bs * E > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    cache = torch.empty(NB, bs, E, dtype=torch.float16, device="cuda")
    n, H = 130, 16
    rng = np.random.default_rng(12)
    rows = rng.standard_normal((n, E)).astype(np.float16)
    bt = torch.tensor([[NB - 1, 0, NB - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = bt[0, pos.long() // bs].long() * bs + pos.long() % bs
    cs = torch.cat([torch.ones(200, 32), torch.zeros(200, 32)], 1).cuda()   # no turn
    err = _err()
    pkv.paged_latent_append(_t(rows), None, EPS, cs, pos, slots, cache, err_word=err)
    st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lat, rop = pkv.paged_latent_gather(cache, bt, st, n, R, err_word=err)
    assert np.array_equal(lat.cpu().numpy(), rows[:, :R])
    assert np.array_equal(rop.cpu().numpy(), rows[:, R:])
    q = rng.standard_normal((1, H, E)).astype(np.float16)
    lse = torch.empty(1, H, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = pkv.paged_latent_attention(_t(q), cache, bt, lens, 0.07, R, lse=lse, err_word=err)
    assert pkv.get_error(err) == 0
    ref = attend64(q, rows, rows[:, :R], [n], 0.07)
    assert_attention(out.cpu().numpy(), lse.cpu().numpy(), *ref, "far blocks")


# --- gather --------------------------------------------------------------------

@pytest.mark.parametrize("R,P,bs", [(512, 64, 16), (256, 64, 64), (24, 8, 5)])
def test_gather(R, P, bs):
    lens = [1, 40, 0, 17, 129]
    p = Paged(lens, R, P, bs, 7)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    lat = torch.full((200, R), 5.0, dtype=torch.float16, device="cuda")
    rop = torch.full((200, P), 5.0, dtype=torch.float16, device="cuda")
    err = _err()
    pkv.paged_latent_gather(_t(p.cache), _t(p.tables), _t(start), 200, R, latents=lat, ropes=rop,
                            err_word=err)
    assert pkv.get_error(err) == 0
    rows = np.concatenate(p.rows)
    assert np.array_equal(lat.cpu().numpy()[:187], rows[:, :R])
    assert np.array_equal(rop.cpu().numpy()[:187], rows[:, R:])
    assert torch.all(lat[187:] == 5.0) and torch.all(rop[187:] == 5.0)


def test_gather_flags():
    p = Paged([40, 20], 64, 16, 16, 8)
    p.tables[0, 1] = -1
    start = np.array([0, 40, 40 + 49], np.int32)   # 49 > 3 blocks of 16
    lat = torch.full((89, 64), 5.0, dtype=torch.float16, device="cuda")
    err = _err()
    p.tables[1] = [p.tables[1, 0], p.tables[1, 1], 0]
    got, _ = pkv.paged_latent_gather(_t(p.cache), _t(p.tables), _t(start), 89, 64, latents=lat,
                                     err_word=err)
    assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID | pkv.PKV_ERRBIT_CONTEXT
    got = got.cpu().numpy()
    assert np.array_equal(got[:16], p.rows[0][:16, :64]) and np.all(got[16:32] == 5.0)
    assert np.array_equal(got[40:60], p.rows[1][:, :64]) and np.all(got[88] == 5.0)


# --- expanded attention ----------------------------------------------------------

def _prefill_problem(nq, nk, H, d, seed):
    rng = np.random.default_rng(seed)
    TQ, TK = sum(nq), sum(nk)
    qs = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    ks = np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)
    q = rng.standard_normal((TQ, H, d + 64)).astype(np.float16)
    kv = rng.standard_normal((TK, H, 2 * d)).astype(np.float16)
    kr = rng.standard_normal((TK, 64)).astype(np.float16)
    return q, kv, kr, qs, ks


def _prefill(q, kv, kr, qs, ks, scale, mq, mk):
    err = _err()
    d = q.shape[2] - 64
    out = torch.full((q.shape[0], q.shape[1], d), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pkv.latent_prefill_attention(_t(q), _t(kv), _t(kr), _t(qs), _t(ks), scale, mq, mk, out=out,
                                 lse=lse, err_word=err)
    return out.cpu().numpy(), lse.cpu().numpy(), pkv.get_error(err)


def _check_prefill(q, kv, kr, qs, ks, scale, got, what, skip=()):
    out, lse, _ = got
    d, H = q.shape[2] - 64, q.shape[1]
    for b in range(len(qs) - 1):
        n, m = int(qs[b + 1] - qs[b]), int(ks[b + 1] - ks[b])
        if n == 0 or b in skip:
            continue
        r, s = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
        k = np.concatenate([kv[s][..., :d], np.repeat(kr[s][:, None], H, 1)], -1)
        ref = attend64(q[r], k, kv[s][..., d:], m - n + np.arange(n) + 1, scale)
        assert_attention(out[r], lse[r], *ref, f"{what}: sequence {b}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk,H", [
    ([1], [1], 1), ([1, 5, 0, 64], [1, 5, 3, 64], 3), ([128, 129, 127], [128, 129, 127], 2),
    ([257], [257], 5), ([3, 100, 1], [200, 333, 1], 4), ([130], [1000], 2), ([600], [600], 1)])
def test_prefill(nq, nk, H, d):
    q, kv, kr, qs, ks = _prefill_problem(nq, nk, H, d, sum(nq) + d + H)
    scale = 1.0 / np.sqrt(d + 64)
    got = _prefill(q, kv, kr, qs, ks, scale, max(nq), max(nk))
    assert got[2] == 0
    _check_prefill(q, kv, kr, qs, ks, scale, got, "prefill")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("empty", [0, 20, 60, 500])
def test_prefill_beside_empty_sequences(empty, d):
    """The same sequences with ever more places in the batch that have none: few
    places split each tile's keys over a cluster's CTAs, many do not."""
    nq, nk = [200, 1, 129, 40], [420, 96, 129, 97]
    q, kv, kr, qs, ks = _prefill_problem(nq, nk, 3, d, 71)
    qs = np.concatenate([qs, np.full(empty, qs[-1])]).astype(np.int32)
    ks = np.concatenate([ks, np.full(empty, ks[-1])]).astype(np.int32)
    got = _prefill(q, kv, kr, qs, ks, 0.09, 200, 420)
    assert got[2] == 0
    _check_prefill(q, kv, kr, qs, ks, 0.09, got, f"{empty} empty")


@pytest.mark.parametrize("factor", [1.0, 20.0, -20.0])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_single_tiles_among_others(d, factor):
    """Sequences whose last (or only) rows fill no more than one tile, with an odd and
    an even number of key steps, between others: 40 heads, so that CTAs take over
    several in any order."""
    nq, nk = [1, 128, 40, 129, 300, 7, 100, 384], [500, 128, 1000, 129, 395, 193, 290, 384]
    q, kv, kr, qs, ks = _prefill_problem(nq, nk, 40, d, 81)
    scale = factor / np.sqrt(d + 64)
    got = _prefill(q, kv, kr, qs, ks, scale, 384, 1000)
    assert got[2] == 0
    _check_prefill(q, kv, kr, qs, ks, scale, got, "single tiles")


@pytest.mark.parametrize("factor", [0.0, 20.0, -1.0, -20.0])
def test_prefill_flat_and_peaked(factor):
    q, kv, kr, qs, ks = _prefill_problem([300, 40], [300, 200], 2, 128, 5)
    scale = factor / np.sqrt(192)
    _check_prefill(q, kv, kr, qs, ks, scale, _prefill(q, kv, kr, qs, ks, scale, 300, 300), "peaked")


def test_prefill_rising_logits():
    """Keys that grow along the sequence: O follows the reference in every step."""
    q, kv, kr, qs, ks = _prefill_problem([700], [700], 2, 128, 8)
    grow = np.linspace(0.01, 4.0, 700)[:, None, None]
    sign = np.sign(q[600, :, :128].astype(np.float64))
    kv[..., :128] = (grow * sign * np.abs(kv[..., :128].astype(np.float64))).astype(np.float16)
    _check_prefill(q, kv, kr, qs, ks, 0.07, _prefill(q, kv, kr, qs, ks, 0.07, 700, 700), "rising")


def test_prefill_many_items():
    """More work than CTAs: each takes over several (sequence, head, rows) items,
    some of them empty."""
    nq = [300, 0, 17, 513, 1, 256]
    nk = [300, 9, 17, 600, 700, 300]
    q, kv, kr, qs, ks = _prefill_problem(nq, nk, 61, 64, 9)
    got = _prefill(q, kv, kr, qs, ks, 0.09, 1024, 1024)
    assert got[2] == 0
    _check_prefill(q, kv, kr, qs, ks, 0.09, got, "many items")


def test_prefill_captured_and_replayed():
    """Captured with the largest lengths as bounds, replayed on shorter ones, after a
    kernel on the same stream that writes its inputs."""
    q, kv, kr, qs, ks = _prefill_problem([200, 130], [260, 130], 3, 128, 10)
    dev = [_t(x) for x in (q, kv, kr, qs, ks)]
    src = dev[0].clone()
    out = torch.zeros(330, 3, 128, dtype=torch.float16, device="cuda")
    lse = torch.zeros(330, 3, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev[0].copy_(src)
        pkv.latent_prefill_attention(*dev, 0.07, 330, 390, out=out, lse=lse)
    dev[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    _check_prefill(q, kv, kr, qs, ks, 0.07, (out.cpu().numpy(), lse.cpu().numpy(), 0), "replay")
    qs2, ks2 = np.array([0, 30, 330], np.int32), np.array([0, 30, 390], np.int32)
    dev[3].copy_(_t(qs2))
    dev[4].copy_(_t(ks2))
    g.replay()
    torch.cuda.synchronize()
    _check_prefill(q, kv, kr, qs2, ks2, 0.07, (out.cpu().numpy(), lse.cpu().numpy(), 0), "replay 2")


def test_prefill_with_the_largest_bounds():
    """Host bounds far above the lengths, up to the largest int."""
    q, kv, kr, qs, ks = _prefill_problem([130, 1], [200, 90], 2, 64, 12)
    top = 2 ** 31 - 1
    _check_prefill(q, kv, kr, qs, ks, 0.09, _prefill(q, kv, kr, qs, ks, 0.09, top, top), "bounds")


def test_prefill_neighbours_do_not_leak():
    """NaN in the rows of another sequence and beyond the last one stays there."""
    nq, nk = [70, 33, 200], [70, 150, 200]
    q, kv, kr, qs, ks = _prefill_problem(nq, nk, 2, 128, 6)
    kv = np.concatenate([kv, np.full((200, 2, 256), np.nan, np.float16)])
    kr = np.concatenate([kr, np.full((200, 64), np.nan, np.float16)])
    kv[ks[1]:ks[2]] = np.nan
    out, lse, bits = _prefill(q, kv, kr, qs, ks, 0.07, 200, 200)
    assert bits == 0
    kv[ks[1]:ks[2]] = 0
    _check_prefill(q, kv, kr, qs, ks, 0.07, (out, lse, 0), "neighbours", skip=(1,))


def test_prefill_bad_sequences():
    """More queries than keys, rows beyond the tensors, a longer sequence than the
    host's bound: flagged and left unwritten."""
    q, kv, kr, qs, ks = _prefill_problem([40, 30, 20, 10], [40, 30, 20, 10], 2, 128, 7)
    ks2 = ks.copy()
    ks2[2] = ks2[1] + 29        # 30 queries, 29 keys; the next sequence has 21 keys
    ks2[4] = 101                # 11 keys, one beyond the tensor
    out, lse, bits = _prefill(q, kv, kr, qs, ks2, 0.07, 39, 40)
    assert bits == pkv.PKV_ERRBIT_CONTEXT
    for b in (0, 1, 3):
        assert np.all(out[qs[b]:qs[b + 1]] == 7.0) and np.all(lse[qs[b]:qs[b + 1]] == 7.0)
    _check_prefill(q, kv, kr, qs, ks2, 0.07, (out, lse, 0), "bad", skip=(0, 1, 3))


# --- together --------------------------------------------------------------------

def test_prompt_then_decode_expanded_equals_absorbed():
    """A layer's run over a latent cache: the prompt is appended, gathered and
    attended in the expanded form; the next tokens are appended and attended in the
    absorbed form; both against the 64-bit formula on the cache's values."""
    H, d, R, P, bs, n, more = 4, 128, 512, 64, 16, 75, 3
    g = torch.Generator().manual_seed(3)

    def rnd(*s, f=1.0):
        return (f * torch.randn(*s, generator=g)).half().cuda()

    wk, wv = rnd(H, d, R, f=R ** -0.5), rnd(H, d, R, f=R ** -0.5)
    kv, q, w = rnd(n + more, R + P), rnd(n + more, H, d + P), rnd(R, f=0.1) + 1
    cs = torch.from_numpy(table(P, 200)).cuda()
    pos = torch.arange(n + more, dtype=torch.int32, device="cuda")
    bt = torch.tensor([[4, 1, 6, 0, 2]], dtype=torch.int32, device="cuda")
    slots = bt[0, pos.long() // bs].long() * bs + pos.long() % bs
    cache = torch.full((7, bs, R + P), float("nan"), dtype=torch.float16, device="cuda")
    err, scale = _err(), (d + P) ** -0.5
    qt = q.clone()
    absorbed = torch.empty(more, H, R + P, dtype=torch.float16, device="cuda")
    # the prompt
    pkv.paged_latent_append(kv[:n], w, EPS, cs, pos[:n], slots[:n], cache, q_rope=qt[:n, :, d:],
                            q_out=qt[:n, :, d:], err_word=err)
    st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lat, rop = pkv.paged_latent_gather(cache, bt, st, n, R, err_word=err)
    ex = torch.cat([torch.einsum("tr,hdr->thd", lat.float(), wk.float()),
                    torch.einsum("tr,hdr->thd", lat.float(), wv.float())], -1).half()
    out = pkv.latent_prefill_attention(qt[:n], ex, rop, st, st, scale, n, n, err_word=err)
    # the next tokens
    pkv.paged_latent_append(kv[n:], w, EPS, cs, pos[n:], slots[n:], cache, q_rope=q[n:, :, d:],
                            q_out=absorbed[..., R:], err_word=err)
    absorbed[..., :R] = torch.einsum("thd,hdr->thr", q[n:, :, :d].float(), wk.float()).half()
    lens = torch.tensor([n + more], dtype=torch.int32, device="cuda")
    o2 = pkv.paged_latent_attention(absorbed, cache, bt, lens, scale, R,
                                    query_start=torch.tensor([0, more], dtype=torch.int32,
                                                             device="cuda"),
                                    max_q_len=more, max_context_len=n + more, err_word=err)
    o2 = torch.einsum("thr,hdr->thd", o2.float(), wv.float())
    assert pkv.get_error(err) == 0
    # the formula in 64 bits on the cache's values
    rows = cache.view(-1, R + P)[slots].double().cpu().numpy()
    k = np.einsum("tr,hdr->thd", rows[:, :R], wk.double().cpu().numpy())
    v = np.einsum("tr,hdr->thd", rows[:, :R], wv.double().cpu().numpy())
    qr, _ = turn64(q[..., d:].double().cpu().numpy(), cs.cpu().numpy()[:n + more], False)
    q64 = np.concatenate([q[..., :d].double().cpu().numpy(), qr], -1)
    k = np.concatenate([k, np.repeat(rows[:, None, R:], H, 1)], -1)
    ref, mag, _, _ = attend64(q64, k, v, np.arange(n + more) + 1, scale)
    got = np.concatenate([out.double().cpu().numpy(), o2.double().cpu().numpy()])
    # fp16 roundings of k, v, q' and the rotated queries (2^-11 each, on logits of
    # size about 10: 0.02 of a weight at most), weights and results
    assert np.max(np.abs(got - ref)) <= 0.02 * np.max(mag)
    assert np.linalg.norm(got - ref) <= 2e-3 * np.linalg.norm(ref)


def test_copy_on_write_of_a_latent_block():
    """The block manager's copy on a latent cache, as one head of R + P entries."""
    R, P, bs = 512, 64, 16
    c = torch.randn(4, bs, R + P).half().cuda()
    was = c.clone()
    view = c.view(4, 1, bs, R + P)
    i32 = dict(dtype=torch.int32, device="cuda")
    paged_kv_copy_blocks(view, view, torch.tensor([2], **i32), torch.tensor([0], **i32),
                         torch.tensor([5], **i32))
    assert torch.equal(c[0, :5], was[2, :5]) and torch.equal(c[0, 5:], was[0, 5:])
    assert torch.equal(c[1:], was[1:])


class _Calls:
    """The native marshalling, which has to take every call; or none of them."""

    def __init__(self, real, native):
        self.real, self.native, self.taken = real, native, 0

    def __getattr__(self, name):
        def call(*a):
            if not self.native:
                return None
            r = getattr(self.real, name)(*a)
            assert r is not None, name
            self.taken += 1
            return r
        return call


def _one_of_each_call():
    """Results of every call, with and without what the caller may give."""
    g = torch.Generator().manual_seed(5)

    def rnd(*s):
        return torch.randn(*s, generator=g).half().cuda()

    i32 = dict(dtype=torch.int32, device="cuda")
    T, H, Hk, d, R, P, bs = 5, 4, 2, 128, 512, 64, 16
    cs, pos = torch.rand(50, P, generator=g).cuda(), torch.arange(T, **i32)
    slots, err = torch.arange(T, device="cuda") + 3, _err()
    q, k, v, w = rnd(T, H, d), rnd(T, Hk, d), rnd(T, Hk, d), rnd(d)
    results = []
    for out in (None, torch.empty_like(q)):
        kc, vc = torch.zeros(2, 3, Hk, bs, d, dtype=torch.float16, device="cuda")
        r = pkv.paged_qk_norm_rope_append(q, k, v, w, None, EPS, cs, pos, slots, kc, vc, q_out=out,
                                          err_word=err)
        assert out is None or r is out
        k8, v8 = torch.zeros(2, 3, Hk, bs, d, dtype=torch.uint8, device="cuda")
        r8 = pkv.paged_qk_norm_rope_append_fp8(q, k, v, None, w, EPS, None, None, slots, k8, v8, 0.02,
                                               0.03, interleaved=True, q_out=out)
        results += [kc, vc, k8, v8, r8.clone()] + ([r] if out is None else [])
    cache, kv, lw = torch.zeros(4, bs, R + P, dtype=torch.float16, device="cuda"), rnd(40, R + P), rnd(R)
    pos, slots = torch.arange(40, **i32), torch.arange(40, device="cuda")
    qr, ab = rnd(40, H, P + 8), torch.zeros(40, H, R + P, dtype=torch.float16, device="cuda")
    pkv.paged_latent_append(kv, lw, EPS, cs, pos, slots, cache, q_rope=qr[..., 8:], q_out=ab[..., R:])
    pkv.paged_latent_append(kv[7:8], None, EPS, cs, pos[3:4], slots[:1] + 60, cache, interleaved=True,
                            err_word=err)
    results += [cache, ab]
    bt, lens = torch.tensor([[0, 1, 2]], **i32), torch.tensor([40], **i32)
    lse = torch.zeros(2, H, device="cuda")
    ql = rnd(2, H, R + P)
    ws = torch.empty(pkv.latent_plan(1, 2, 2, H, R, P, bs, 3, 40), dtype=torch.uint8, device="cuda")
    results += [pkv.paged_latent_attention(ql, cache, bt, lens, 0.05, R, torch.tensor([0, 2], **i32), 2,
                                           max_context_len=40, workspace=ws, lse=lse), lse]
    out = torch.empty(1, H, R, dtype=torch.float16, device="cuda")
    assert pkv.paged_latent_attention(ql[:1], cache, bt, lens, 1, R, out=out, err_word=err) is out
    st = torch.tensor([0, 40], **i32)
    lat, rop = pkv.paged_latent_gather(cache, bt, st, 40, R)
    l2 = torch.empty_like(lat)
    assert pkv.paged_latent_gather(cache, bt, st, 40, R, latents=l2, err_word=err)[0] is l2
    ex, qp = rnd(40, H, 2 * d), rnd(40, H, d + P)
    plse = torch.zeros(40, H, device="cuda")
    results += [out, lat, rop, l2, pkv.latent_prefill_attention(qp, ex, rop, st, st, 0.07, 40, 40, lse=plse),
                plse]
    po = torch.empty_like(ex[..., :d])
    assert pkv.latent_prefill_attention(qp, ex, rop, st, st, 0.07, 40, 40, out=po, err_word=err) is po
    assert pkv.get_error(err) == 0
    return [x.contiguous().cpu().numpy().tobytes() for x in results + [po]]


def test_both_marshallings_make_the_same_calls(monkeypatch):
    """Every call through the native marshalling and through the Python one: the same
    bits."""
    from paged_kv_cache_213_gb300 import rope
    native, python = _Calls(rope._native(), True), _Calls(rope._native(), False)
    monkeypatch.setattr(rope, "_calls", native)
    one = _one_of_each_call()
    monkeypatch.setattr(rope, "_calls", python)
    other = _one_of_each_call()
    assert native.taken == 12 and one == other


def test_native_marshalling_leaves_the_rest():
    """What the native marshalling does not take it leaves alone: it returns None."""
    from paged_kv_cache_213_gb300 import rope
    f = rope._native().latent_gather
    c = torch.zeros(4, 16, 576, dtype=torch.float16, device="cuda")
    bt = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    plain = [c, bt, st, 40, 512, None, None, None]
    assert f(*plain) is not None
    for at, x in ((0, c.float()), (0, c.cpu()), (0, None), (0, "c"), (0, c[0]), (0, c.transpose(0, 1)),
                  (1, bt.long()), (2, st[:1]), (3, 40.0), (3, 1 << 40), (3, -1), (4, 576), (4, None),
                  (5, c), (6, torch.zeros(40, 64)), (7, c)):
        assert f(*plain[:at], x, *plain[at + 1:]) is None, at
    assert f(*plain[:-1]) is None and f(*plain, 1) is None and f() is None


def test_python_calls_refuse_what_does_not_fit():
    """Types, shapes, strides and devices that the calls do not take."""
    p, q, qs, scale = _problem([20, 30], [1, 1], 4, 512, 16, 98)
    q, c, bt, cl = (_t(x) for x in (q, p.cache, p.tables, p.lens.astype(np.int32)))

    def bad(error, f, *a, **k):
        with pytest.raises(error):
            f(*a, **k)

    f = pkv.paged_latent_attention
    bad(TypeError, f, q.float(), c, bt, cl, scale, 512)
    bad(TypeError, f, q, c, bt.long(), cl, scale, 512)
    bad(TypeError, f, None, c, bt, cl, scale, 512)
    bad(ValueError, f, q, c, bt.cpu(), cl, scale, 512)
    bad(ValueError, f, q, c, bt.t().contiguous().t(), cl, scale, 512)   # not contiguous
    bad(ValueError, f, q[:1], c, bt, cl, scale, 512)
    bad(ValueError, f, q, c, bt, cl, scale, 576)
    bad(ValueError, f, q, c, bt, cl, scale, 512, max_q_len=2)
    bad(ValueError, f, q, c, bt, cl, scale, 512, lse=torch.empty(2, 5, device="cuda"))
    bad(ValueError, f, q, c, bt, cl, scale, 512, out=torch.empty_like(q))
    bad(pkv.PagedKVError, f, q, c, bt, cl, scale, 512,
        workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    bad(pkv.PagedKVError, f, q, c, bt, cl, float("inf"), 512)
    bad(pkv.PagedKVError, f, q, c, bt, cl, scale, 500)
    st = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    bad(ValueError, pkv.paged_latent_gather, c, bt, st[:2], 50, 512)
    bad(ValueError, pkv.paged_latent_gather, c, bt, st, 50, 512, latents=q)
    h = torch.zeros(3, 2, 192, dtype=torch.float16, device="cuda")
    bad(ValueError, pkv.latent_prefill_attention, h, h, h[:, 0, :64].contiguous(), st, st, 1.0, 3, 3)
    cs = torch.zeros(9, 64, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv = torch.zeros(2, 576, dtype=torch.float16, device="cuda")
    bad(ValueError, pkv.paged_latent_append, kv, None, EPS, cs, i, i.long(), c, q_rope=q[..., :64])
    bad(ValueError, pkv.paged_latent_append, kv[:, ::2], None, EPS, cs, i, i.long(), c)
    bad(TypeError, pkv.paged_latent_append, kv, None, EPS, cs, i.long(), i.long(), c)
