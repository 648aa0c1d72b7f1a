"""The 8-bit caches with block scales on the GPU: append, attention, read-back and
block copy against their definitions in 64 bits (tests/q8_util.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from paged_kv_cache_213_gb300 import q8, rope

from q8_util import LIMIT, U32, Paged, append64, assert_attention, attend64, values

pytestmark = pytest.mark.gpu
KINDS = ["e4m3", "int8"]


def t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def starts(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


@pytest.fixture(params=["native", "python"])
def marshalled(request, monkeypatch):
    """Every call through the native module and through the ctypes code."""
    if request.param == "python":
        monkeypatch.setattr(q8, "_native", lambda: rope._PythonOnly())
    return request.param


class OnGpu:
    """A Paged problem's tensors."""

    def __init__(self, p):
        self.p, self.keys = p, 16  # keys that share a V reference at least
        self.kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
        self.tables, self.lens = t(p.tables), t(p.lens.astype(np.int32))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def attend(self, q, scale, news=None, **kw):
        TQ, H, d = q.shape
        lse = torch.full((TQ, H), float("nan"), device="cuda")
        many = {} if news is None else dict(query_start=t(starts(news)), max_q_len=max(news))
        kw.setdefault("max_context_len", int(self.p.lens.max()))
        out = pkv.paged_decode_attention_q8(q, *self.kv, self.tables, self.lens, scale, lse=lse,
                                            err_word=self.err, **many, **kw)
        assert pkv.get_error(self.err) == 0
        return out.cpu().numpy(), lse.cpu().numpy()

    def check(self, q16, scale, news=None, **kw):
        out, lse = self.attend(t(q16), scale, news, **kw)
        if max(news or [1]) * (q16.shape[1] // self.p.codes[0].shape[1]) > 32:
            self.keys = 64
        at = starts([1] * len(self.p.lens) if news is None else news)
        for b in range(len(self.p.lens)):
            self.near(b, q16, out, lse, scale, at)
        return out, lse

    def near(self, b, q16, out, lse, scale, at):
        """Sequence b's rows against the formula."""
        rows, L = slice(at[b], at[b + 1]), int(self.p.lens[b])
        if L == 0:
            assert np.all(out[rows] == 0) and np.all(np.isneginf(lse[rows]))
        elif at[b] < at[b + 1]:
            k, v = (self.p.tokens(side, b, L) for side in range(2))
            spread = self.p.spread_in_steps(b, L, self.keys)
            assert_attention(out[rows], lse[rows], attend64(q16[rows], k, v, scale, spread), f"sequence {b} of {L}")


def queries(p, T, H, gain=1.0):
    return (gain * p.rng.standard_normal((T, H, p.codes[0].shape[3]))).astype(np.float16)


# --- append -----------------------------------------------------------------

def run_append(p, kv, news, x, views=False, err_bits=0, **kw):
    """One append of x = (k, v) on tensors kv and on the numpy state."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if views:  # columns of a wider matrix
        wide = torch.cat([t(x[0]).flatten(1), torch.full((len(x[0]), 8), 9.0, dtype=torch.float16,
                                                         device="cuda"), t(x[1]).flatten(1)], 1)
        w = x[0].shape[1] * x[0].shape[2]
        k = wide[:, :w].unflatten(1, x[0].shape[1:])
        v = wide[:, w + 8:].unflatten(1, x[0].shape[1:])
    else:
        k, v = t(x[0]), t(x[1])
    many = {} if news is None else dict(query_start=t(starts(news)), max_q_len=max(news))
    pkv.paged_kv_append_q8(k, v, *kv, t(p.tables), t(p.lens.astype(np.int32)), err_word=err, **many, **kw)
    assert pkv.get_error(err) == err_bits


def same_state(p, kv):
    for got, want, what in zip(kv, p.codes + p.scales, ("k codes", "v codes", "k scales", "v scales")):
        got = got.cpu().numpy()
        bad = got.view(np.uint8) != want.view(np.uint8)
        assert not bad.any(), f"{what}: {np.argwhere(bad)[:4].tolist()} of {bad.sum()}"


APPENDS = [  # kv heads, d, block size, cached tokens, new tokens
    (8, 128, 16, [0, 1, 15, 16, 17, 31, 500], [1] * 7),
    (1, 64, 16, [0, 7], [1, 1]),
    (3, 64, 32, [0, 31, 32, 33, 5], [1, 2, 3, 40, 0]),
    (8, 128, 16, [0, 3, 16, 30], [5, 5, 5, 5]),
    (2, 128, 64, [0, 63, 64, 100], [200, 1, 64, 37]),
    (5, 64, 128, [0, 127, 300], [129, 2, 1]),
    (1, 128, 256, [0, 250, 13], [257, 7, 600]),
    (12, 128, 32, [77], [1000]),
    (17, 128, 16, [9, 0], [33, 16]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,d,bs,held,news", APPENDS)
def test_append(kind, Hk, d, bs, held, news, marshalled):
    p = Paged([m + n for m, n in zip(held, news)], Hk, d, bs, kind, seed=len(held) + d + bs)
    for b, (m, n) in enumerate(zip(held, news)):  # what comes is poison yet
        for i in range(m, m + n):
            for side in range(2):
                p.codes[side][p.tables[b, i // bs], :, i % bs] = 127
                if i % bs == 0 or m == 0:
                    p.scales[side][p.tables[b, i // bs]] = np.nan
    x = [p.rng.standard_normal((sum(news), Hk, d)).astype(np.float16) for _ in "kv"]
    # sizes from far below to far above what is held: no growth, and growth by many doublings
    x[0] *= (2.0 ** p.rng.integers(-6, 7, (sum(news), Hk, 1))).astype(np.float16)
    kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    one = all(n == 1 for n in news)
    run_append(p, kv, None if one else news, x, views=bs != 16)
    for side in range(2):
        append64(kind, x[side], starts(news), p.lens, p.tables, p.codes[side], p.scales[side])
    same_state(p, kv)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [1, 3])
def test_append_special_values(kind, new):
    """Zeros, infinities, NaN, subnormals and the largest numbers, into blocks that are
    empty, of zeros, or of ordinary values."""
    rows = [[0.0], [-0.0], [np.inf], [-np.inf], [np.nan], [6e-8], [65504.0], [1.0, np.inf, np.nan],
            [np.nan, 3e-7], [-65504.0, 2.0], [1e-4, -1e-3]]
    held = [0, 5, 5] * len(rows)
    Hk, d, bs = 2, 64, 16
    p = Paged([m + new for m in held], Hk, d, bs, kind, seed=3)
    for b, m in enumerate(held):
        if m == 0:
            p.scales[0][p.tables[b, 0]] = p.scales[1][p.tables[b, 0]] = np.nan
        elif b % 3 == 2:  # a block of zeros
            for side in range(2):
                p.codes[side][p.tables[b, 0], :, :m] = 0
                p.scales[side][p.tables[b, 0]] = 0
    x = np.zeros((2, len(held) * new, Hk, d), np.float16)
    for b in range(len(held)):
        pattern = rows[b // 3]
        x[:, b * new:(b + 1) * new] = np.resize(np.array(pattern, np.float16), (new, Hk, d))
    kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    run_append(p, kv, None if new == 1 else [new] * len(held), list(x))
    for side in range(2):
        append64(kind, x[side], starts([new] * len(held)), p.lens, p.tables, p.codes[side], p.scales[side])
    same_state(p, kv)


@pytest.mark.parametrize("kind", KINDS)
def test_every_fp16_value_gets_its_code(kind):
    """All finite fp16 numbers at scales that they set themselves and at one that is given."""
    every = np.arange(65536, dtype=np.uint16).view(np.float16)
    every = every[np.isfinite(every)]
    every = every[np.argsort(np.abs(every.astype(np.float64)), kind="stable")]
    d, bs = 64, 16
    n = -(-len(every) // (bs * d)) * bs
    x = np.resize(every, (n, 1, d))
    p = Paged([n], 1, d, bs, kind, seed=0)
    p.scales[0][:] = p.scales[1][:] = np.nan
    kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    run_append(p, kv, [n], [x, x[::-1].copy()])
    for side, y in enumerate((x, x[::-1])):
        append64(kind, y, starts([n]), p.lens, p.tables, p.codes[side], p.scales[side])
    same_state(p, kv)


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_one_by_one_are_off_by_little(kind):
    """40 tokens of growing size one by one: what is read back is off by the bounds that
    the header states (E4M3: one rounding, and half a step of the subnormals a doubling;
    int8: one step of the final scale)."""
    Hk, d, bs, n = 2, 128, 16, 40
    p = Paged([n], Hk, d, bs, kind, seed=11)
    x = (p.rng.standard_normal((n, Hk, d)) * 1.3 ** np.arange(n)[:, None, None] * 1e-3).astype(np.float16)
    kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    for i in range(n):
        pkv.paged_kv_append_q8(t(x[i:i + 1]), t(-x[i:i + 1]), *kv, t(p.tables),
                               torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
    k, v = pkv.paged_kv_gather_q8(*kv, t(p.tables), t(starts([n])), n)
    step = kv[2].cpu().numpy()[p.tables[0, np.arange(n) // bs]][..., None].astype(np.float64)
    if kind == "int8":
        bound = step
    else:  # subnormal codes lie 2^-9 apart; a doubling halves the earlier errors too
        bound = 2.0 ** -4 * np.abs(x.astype(np.float64)) + 2.0 ** -9 * step
    bound = bound * (1 + 4 * U32) + 2.0 ** -11 * np.abs(x.astype(np.float64))
    for got, want in ((k, x), (v, -x)):
        err = np.abs(got.cpu().numpy().astype(np.float64) - want.astype(np.float64))
        assert np.all(err <= bound), np.max(err / bound)


# --- attention --------------------------------------------------------------

ATTENDS = [  # kv heads, group, d, block size, lengths
    (8, 4, 128, 16, [1, 2, 15, 16, 17, 31, 33, 64, 130, 700]),
    (1, 1, 64, 16, [1]),
    (2, 8, 128, 32, [300, 1, 0, 31, 999, 32]),
    (3, 1, 64, 16, [0, 0, 5, 77]),
    (1, 3, 128, 64, [65, 64, 63]),
    (12, 1, 64, 128, [1000, 129, 128, 1]),
    (2, 2, 64, 256, [2000, 255, 257]),
    (1, 16, 128, 16, [400, 33]),
    (1, 71, 64, 16, [90, 800]),
    (4, 5, 128, 32, [2500]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,bs,lens", ATTENDS)
def test_attend(kind, Hk, g, d, bs, lens, marshalled):
    p = Paged(lens, Hk, d, bs, kind, seed=7 * Hk + g)
    OnGpu(p).check(queries(p, len(lens), Hk * g), 1.3 / d ** 0.5)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,bs,lens,news", [
    (2, 4, 128, 16, [5, 20, 33, 700], [5, 4, 1, 3]),
    (8, 4, 128, 16, [400, 90, 16], [5, 5, 5]),
    (1, 1, 64, 32, [9, 300], [9, 8]),
    (2, 8, 64, 16, [64, 130, 40, 7], [16, 0, 40, 1]),
    (1, 4, 128, 64, [333, 70], [100, 70]),
    (2, 3, 128, 16, [150], [150]),
    (1, 6, 64, 128, [1200, 31], [37, 31]),
])
def test_attend_several_tokens(kind, Hk, g, d, bs, lens, news, marshalled):
    p = Paged(lens, Hk, d, bs, kind, seed=5 * Hk + g)
    OnGpu(p).check(queries(p, sum(news), Hk * g), 1.1 / d ** 0.5, news)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,lens", [(8, 4, [9000, 3, 12345]), (1, 8, [70001]), (2, 2, [1] * 300),
                                       (4, 4, list(range(1, 900, 7)))])
def test_attend_many_pieces(kind, Hk, g, lens):
    """Segments over many CTAs, and many segments in one warp."""
    p = Paged(lens, Hk, 128, 16, kind, seed=len(lens))
    gpu = OnGpu(p)
    q = queries(p, len(lens), Hk * g)
    ws = torch.zeros(pkv.q8_plan(len(lens), len(lens), 1, Hk * g, Hk, 128, 16, p.MB), dtype=torch.uint8,
                     device="cuda")
    a = gpu.check(q, 0.1, workspace=ws)
    assert not ws[:pkv.PKV_WORKSPACE_COUNTER_BYTES].any()
    for flags in (0, pkv.PKV_TABLES_READY):  # the same again, from the used workspace
        b = gpu.attend(t(q), 0.1, workspace=ws, flags=flags)
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
    assert not ws[:pkv.PKV_WORKSPACE_COUNTER_BYTES].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", [3, 12])
@pytest.mark.parametrize("gain", [0.0, 1.0, 30.0])
def test_block_scales_that_differ(kind, spread, gain):
    """V references that move up and down, logits that make the rows' references move
    often, and logits that are all the same."""
    lens = [500, 37, 2000]
    p = Paged(lens, 2, 128, 16, kind, seed=spread, spread=spread)
    p.scales[0][p.tables[0, 0]] *= 2.0 ** 4
    OnGpu(p).check(queries(p, 3, 8, gain), 0.05)


@pytest.mark.parametrize("kind", KINDS)
def test_logits_that_climb(kind):
    """Keys that grow along the sequence: every tile moves the references."""
    Hk, d, L = 2, 128, 1600
    p = Paged([L], Hk, d, 16, kind, seed=2)
    for j in range(L // 16):
        p.scales[0][p.tables[0, j]] = 0.002 * (j + 1) / LIMIT[kind] * 4
        p.codes[0][p.tables[0, j], :, :, :] = np.abs(p.codes[0][p.tables[0, j]].astype(np.int16) % 100)
    q = np.abs(queries(p, 1, Hk * 4))
    OnGpu(p).check(q, 0.3)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-20])
def test_scales_of_the_softmax(scale):
    p = Paged([130, 1, 60], 2, 64, 16, "int8", seed=1)
    OnGpu(p).check(queries(p, 3, 4), scale)


def test_blocks_of_zeros():
    """Scale 0: keys of no effect, values of 0; first in a sequence, and all of it."""
    p = Paged([100, 40], 2, 128, 16, "e4m3", seed=4)
    for b, js in ((0, (0, 3)), (1, (0, 1, 2))):
        for j in js:
            for side in range(2):
                p.codes[side][p.tables[b, j]] = 0
                p.scales[side][p.tables[b, j]] = 0
    OnGpu(p).check(queries(p, 2, 8), 0.2)


def test_a_cached_nan_reaches_its_sequence_alone():
    p = Paged([100, 100, 50], 2, 128, 16, "e4m3", seed=4)
    p.codes[1][p.tables[1, 2], 0, 3, 5] = 127
    gpu = OnGpu(p)
    out, _ = gpu.attend(t(queries(p, 3, 4)), 0.1)
    want = np.zeros(out.shape, bool)
    want[1, :2, 5] = True
    assert np.array_equal(np.isnan(out), want)


def test_queries_with_gaps_and_outputs_given():
    p = Paged([70, 300], 2, 128, 16, "int8", seed=9)
    gpu = OnGpu(p)
    q = queries(p, 2, 8)
    want = gpu.check(q, 0.1)
    wide = torch.full((2, 8 * 128 + 520), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 1024] = t(q).flatten(1)
    view = wide[:, 8:8 + 1024].unflatten(1, (8, 128))
    out = torch.empty(2, 8, 128, dtype=torch.float16, device="cuda")
    got = gpu.attend(view, 0.1, out=out)
    assert np.array_equal(got[0], want[0]) and np.array_equal(out.cpu().numpy(), want[0])


def test_rows_and_sequences_out_of_bounds():
    """Flagged, their rows left as they were, the others computed."""
    lens = [40, 50, 60, 70]
    p = Paged(lens, 2, 64, 16, "e4m3", seed=6)
    gpu = OnGpu(p)
    news = [2, 3, 1, 2]
    q = queries(p, sum(news), 4)
    good = gpu.check(q, 0.1, news)[0]
    at = starts(news)
    for change in (dict(lens=[40, 10 ** 6, 60, 70]), dict(lens=[40, -3, 60, 70]), dict(lens=[40, 2, 60, 70])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((sum(news), 4, 64), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((sum(news), 4), 7.0, device="cuda")
        pkv.paged_decode_attention_q8(t(q), *gpu.kv, gpu.tables,
                                      torch.tensor(change["lens"], dtype=torch.int32, device="cuda"), 0.1,
                                      query_start=t(at), max_q_len=3, max_context_len=70, out=out, lse=lse,
                                      err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT
        out, lse = out.cpu().numpy(), lse.cpu().numpy()
        assert np.all(out[at[1]:at[2]] == 7) and np.all(lse[at[1]:at[2]] == 7)
        for b in (0, 2, 3):  # in another split of the work: not bit for bit
            gpu.near(b, q, out, lse, 0.1, at)
    # more new tokens than the host's bound
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_decode_attention_q8(t(q), *gpu.kv, gpu.tables, gpu.lens, 0.1, query_start=t(at), max_q_len=2,
                                  err_word=err)
    assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT
    # rows behind the last sequence are left as they were
    out = torch.full((sum(news) + 4, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    more = np.concatenate([q, q[:4]])
    pkv.paged_decode_attention_q8(t(more), *gpu.kv, gpu.tables, gpu.lens, 0.1, query_start=t(at), max_q_len=3,
                                  max_context_len=70, out=out)
    out = out.cpu().numpy()
    assert np.all(out[sum(news):] == 7) and np.array_equal(out[:sum(news)], good)


def test_bad_blocks_are_flagged_everywhere():
    p = Paged([40, 50], 2, 128, 16, "int8", seed=6)
    gpu = OnGpu(p)
    q = queries(p, 2, 4)
    good = gpu.check(q, 0.1)[0]
    for bad in (-1, p.NB, 2 ** 31 - 1):
        tables = p.tables.copy()
        tables[0, 1] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pkv.paged_decode_attention_q8(t(q), *gpu.kv, t(tables), gpu.lens, 0.1, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID
        assert np.array_equal(out.cpu().numpy()[1], good[1])
        err.zero_()
        k = torch.full((90, 2, 128), 7.0, dtype=torch.float16, device="cuda")
        pkv.paged_kv_gather_q8(*gpu.kv, t(tables), t(starts([40, 50])), 90, k=k, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID
        assert torch.all(k[16:32] == 7) and not torch.any((k[32:] == 7).all(-1))
        err.zero_()
        kv = [x.clone() for x in gpu.kv]
        x = t(queries(p, 2, 2))
        pkv.paged_kv_append_q8(x, x, *kv, t(tables), torch.tensor([20, 50], dtype=torch.int32, device="cuda"),
                               err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID
        err.zero_()
        many = torch.cat([x, x, x])
        pkv.paged_kv_append_q8(many, many, *kv, t(tables),
                               torch.tensor([20, 50], dtype=torch.int32, device="cuda"),
                               query_start=t(starts([3, 3])), max_q_len=3, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID
        for got, want in zip(kv[:2], gpu.kv[:2]):  # nothing beyond the second sequence's tokens
            changed = {int(i) for i in torch.nonzero((got != want).flatten(1).any(1))}
            assert changed <= set(map(int, p.tables[1, 2:4]))


@pytest.mark.parametrize("news", [None, [1, 2]])
def test_append_out_of_bounds(news):
    p = Paged([40, 50], 2, 64, 16, "e4m3", seed=6)
    kv = [t(c) for c in p.codes] + [t(s) for s in p.scales]
    T = 2 if news is None else 3
    x = t(np.ones((T, 2, 64), np.float16))
    for lens in ([40, 10 ** 6], [40, -1]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        many = {} if news is None else dict(query_start=t(starts(news)), max_q_len=2)
        pkv.paged_kv_append_q8(x, x, *kv, t(p.tables), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               err_word=err, **many)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT
    if news is not None:
        for start in ([0, 1, 9], [0, 2, 1], [-1, 1, 3], [0, 3, 3]):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            pkv.paged_kv_append_q8(x, x, *kv, t(p.tables), t(p.lens.astype(np.int32)), err_word=err,
                                   query_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                                   max_q_len=2)
            assert pkv.get_error(err) == pkv.PKV_ERRBIT_CONTEXT


# --- read-back and copy -----------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,d,bs,lens", [(8, 128, 16, [17, 600, 0, 1]), (3, 64, 64, [64, 65]), (1, 128, 256, [700]),
                                          (12, 64, 32, [5] * 40)])
def test_gather(kind, Hk, d, bs, lens, marshalled):
    p = Paged([n + 3 for n in lens], Hk, d, bs, kind, seed=Hk)
    gpu = OnGpu(p)
    first = 2  # rows before the first sequence and behind the last stay
    total = sum(lens) + first + 5
    k = torch.full((total, Hk, d), 7.0, dtype=torch.float16, device="cuda")
    v = torch.full_like(k, 7.0)
    got = pkv.paged_kv_gather_q8(*gpu.kv, gpu.tables, t(starts(lens) + first), total, k=k, v=v,
                                 err_word=gpu.err)
    assert pkv.get_error(gpu.err) == 0 and got[0] is k and got[1] is v
    for side, x in enumerate((k, v)):
        x = x.cpu().numpy()
        assert np.all(x[:first] == 7) and np.all(x[-5:] == 7)
        want = np.concatenate([p.tokens(side, b, n) for b, n in enumerate(lens)])
        assert np.array_equal(x[first:-5], want.astype(np.float32).astype(np.float16))


def test_gather_saturates():
    p = Paged([32], 1, 64, 16, "e4m3", seed=0)
    p.scales[0][p.tables[0]] = 200.0
    p.codes[0][p.tables[0, 0], 0, 0, :2] = 126, 254
    k, _ = pkv.paged_kv_gather_q8(*OnGpu(p).kv, t(p.tables), t(starts([32])), 32)
    k = k.cpu().numpy()
    want = np.clip(p.tokens(0, 0, 32), -65504, 65504).astype(np.float16)
    assert np.array_equal(k, want) and k[0, 0, 0] == 65504 and k[0, 0, 1] == -65504


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,d,bs", [(8, 128, 16), (3, 64, 64), (1, 128, 256)])
def test_copy_blocks(kind, Hk, d, bs):
    p = Paged([5 * bs], Hk, d, bs, kind, seed=1, extra=6)
    gpu = OnGpu(p)
    free = [i for i in range(p.NB) if i not in p.tables[0]]
    src, dst, rows = p.tables[0, :4], np.array(free[:4], np.int32), np.array([bs, 1, 0, bs - 1], np.int32)
    bad = np.array([p.NB, -1, 0, 0], np.int32), np.array([0, 0, -1, p.NB], np.int32)
    pkv.paged_kv_copy_blocks_q8(*gpu.kv, t(src), t(dst), t(rows), err_word=gpu.err)
    assert pkv.get_error(gpu.err) == 0
    for side in range(2):
        for s, e, n in zip(src, dst, rows):
            p.codes[side][e, :, :n] = p.codes[side][s, :, :n]
            p.scales[side][e] = p.scales[side][s]
    same_state(p, gpu.kv)
    pkv.paged_kv_copy_blocks_q8(*gpu.kv, t(bad[0]), t(bad[1]), err_word=gpu.err)
    assert pkv.get_error(gpu.err) == pkv.PKV_ERRBIT_SLOT
    same_state(p, gpu.kv)


# --- together ---------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_prompts_then_steps(kind):
    """A serving loop: prompts appended in chunks and attended, tokens one by one, drafts,
    a fork with copy-on-write; what the attention sees is what the read-back gives."""
    from paged_kv_cache_213_gb300.blocks import BlockManager

    Hk, g, d, bs = 2, 4, 128, 16
    rng = np.random.default_rng(0)
    m = BlockManager(64, bs)
    kv = [torch.full((64, Hk, bs, d), 127, dtype=torch.uint8 if kind == "e4m3" else torch.int8, device="cuda")
          for _ in "kv"] + [torch.full((64, Hk), float("nan"), device="cuda") for _ in "kv"]
    lens = {}

    def step(ids, news):
        for i, n in zip(ids, news):
            if i not in lens:
                m.add_sequence(i)
                lens[i] = 0
            for _ in range(n):
                _, copy = m.append_slot(i)
                if copy:
                    a = [torch.tensor([y], dtype=torch.int32, device="cuda") for y in copy]
                    pkv.paged_kv_copy_blocks_q8(*kv, *a)
            lens[i] += n
        most = max(-(-lens[i] // bs) for i in ids)
        tables = np.full((len(ids), most), -1, np.int32)
        for r, i in enumerate(ids):
            tb = m.block_table(i)
            tables[r, :len(tb)] = tb
        total = [lens[i] for i in ids]
        x = [(rng.standard_normal((sum(news), Hk, d)) * 1.5 ** rng.integers(-3, 4)).astype(np.float16) for _ in "kv"]
        q = rng.standard_normal((sum(news), Hk * g, d)).astype(np.float16)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        many = {} if max(news) == 1 else dict(query_start=t(starts(news)), max_q_len=max(news))
        cl = torch.tensor(total, dtype=torch.int32, device="cuda")
        pkv.paged_kv_append_q8(t(x[0]), t(x[1]), *kv, t(tables), cl, err_word=err, **many)
        lse = torch.empty(sum(news), Hk * g, device="cuda")
        out = pkv.paged_decode_attention_q8(t(q), *kv, t(tables), cl, 0.1, lse=lse, err_word=err, **many)
        k, v = pkv.paged_kv_gather_q8(*kv, t(tables), t(starts(total)), sum(total), err_word=err)
        assert pkv.get_error(err) == 0
        at, of = starts(news), starts(total)
        codes = [c.cpu().numpy() for c in kv]
        for r in range(len(ids)):
            tok = np.arange(total[r])
            full = [values(kind, codes[s][tables[r, tok // bs], :, tok % bs]) *
                    codes[s + 2][tables[r, tok // bs]][..., None].astype(np.float64) for s in range(2)]
            for got, want in zip((k, v), full):
                assert np.array_equal(got[of[r]:of[r + 1]].cpu().numpy(), want.astype(np.float32).astype(np.float16))
            rows = slice(at[r], at[r + 1])
            assert_attention(out[rows].cpu().numpy(), lse[rows].cpu().numpy(),
                             attend64(q[rows], *full, 0.1), f"sequence {ids[r]}")

    step([0, 1], [37, 5])
    step([0, 1], [1, 20])
    for _ in range(3):
        step([0, 1], [1, 1])
    m.fork(0, 2)
    lens[2] = lens[0]
    step([0, 1, 2], [1, 1, 1])
    step([2, 0, 1], [4, 2, 3])
    step([2, 1, 0], [1, 1, 1])


def test_side_stream_and_replayed_graph():
    """A captured step (append, attention, read-back) replayed with other inputs, on a
    stream of its own, its workspace used by eager calls between the replays."""
    Hk, g, d, bs, L = 2, 4, 128, 16, 333
    p = Paged([L, 50], Hk, d, bs, "e4m3", seed=8)
    gpu = OnGpu(p)
    H = Hk * g
    ws = torch.zeros(pkv.q8_plan(2, 2, 1, H, Hk, d, bs, p.MB), dtype=torch.uint8, device="cuda")
    x = torch.zeros(2, Hk, d, dtype=torch.float16, device="cuda")
    q = torch.zeros(2, H, d, dtype=torch.float16, device="cuda")
    lse, out = torch.empty(2, H, device="cuda"), torch.empty(2, H, d, dtype=torch.float16, device="cuda")
    at = t(starts([L, 50]))

    def step():
        pkv.paged_kv_append_q8(x, x, *gpu.kv, gpu.tables, gpu.lens, err_word=gpu.err)
        pkv.paged_decode_attention_q8(q, *gpu.kv, gpu.tables, gpu.lens, 0.1, out=out, lse=lse, workspace=ws,
                                      max_context_len=L, err_word=gpu.err)
        return pkv.paged_kv_gather_q8(*gpu.kv, gpu.tables, at, L + 50, err_word=gpu.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            k, v = step()
        for i in range(3):
            new, qs = (p.rng.standard_normal(s.shape).astype(np.float16) for s in (x, q))
            x.copy_(torch.from_numpy(new))
            q.copy_(torch.from_numpy(qs))
            graph.replay()
            side.synchronize()
            assert pkv.get_error(gpu.err) == 0
            got = [y.cpu().numpy().copy() for y in (out, lse, k, v)]
            for side_, kept in enumerate(gpu.kv[:2]):
                p.codes[side_], p.scales[side_] = kept.cpu().numpy(), gpu.kv[2 + side_].cpu().numpy()
            for b, n in enumerate((L, 50)):
                kk, vv = (p.tokens(s, b, n) for s in range(2))
                assert_attention(got[0][b:b + 1], got[1][b:b + 1], attend64(qs[b:b + 1], kk, vv, 0.1), f"replay {i}")
            eager = [y.cpu().numpy() for y in step()]
            assert np.array_equal(eager[0], got[2]) and np.array_equal(out.cpu().numpy(), got[0])


def test_a_workspace_that_was_not_cleared_is_reported():
    """Counters full of ones: flagged (nothing faults or hangs: no one waits on them);
    after the clear the call is right again."""
    p = Paged([5000], 1, 128, 16, "int8", seed=8)
    gpu = OnGpu(p)
    q = queries(p, 1, 8)
    ws = torch.full((pkv.q8_plan(1, 1, 1, 8, 1, 128, 16, p.MB),), 255, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        err.zero_()
        pkv.paged_decode_attention_q8(t(q), *gpu.kv, gpu.tables, gpu.lens, 0.1, workspace=ws, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_WORKSPACE
    pkv.paged_decode_workspace_clear(ws)
    gpu.check(q, 0.1, workspace=ws)


def test_calls_with_nothing_to_do():
    p = Paged([40], 2, 64, 16, "int8", seed=6)
    gpu = OnGpu(p)
    none = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    before = [x.clone() for x in gpu.kv]
    lens, tables = gpu.lens[:0], gpu.tables[:0]
    pkv.paged_kv_append_q8(none, none, *gpu.kv, tables, lens)
    pkv.paged_kv_append_q8(none, none, *gpu.kv, gpu.tables, gpu.lens, query_start=t(starts([0])), max_q_len=4)
    assert pkv.paged_decode_attention_q8(torch.empty(0, 4, 64, dtype=torch.float16, device="cuda"), *gpu.kv,
                                         tables, lens, 0.1).shape == (0, 4, 64)
    assert pkv.paged_kv_gather_q8(*gpu.kv, gpu.tables, t(starts([0])), 0)[0].shape == (0, 2, 64)
    pkv.paged_kv_copy_blocks_q8(*gpu.kv, lens, lens)
    for x, y in zip(before, gpu.kv):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# --- sizes at the edges -----------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_one_token_or_none_by_query_start(kind, marshalled):
    """max_q_len 1 with query_start: sequences with a token and without, cached or empty."""
    held, news = [0, 31, 16, 0, 700, 5], [1, 1, 0, 0, 1, 0]
    Hk, d, bs = 2, 128, 16
    p = Paged([m + n for m, n in zip(held, news)], Hk, d, bs, kind, seed=12)
    for b, (m, n) in enumerate(zip(held, news)):
        if n:
            for side in range(2):
                p.codes[side][p.tables[b, m // bs], :, m % bs] = 127
                if m % bs == 0:
                    p.scales[side][p.tables[b, m // bs]] = np.nan
    x = [p.rng.standard_normal((sum(news), Hk, d)).astype(np.float16) for _ in "kv"]
    gpu = OnGpu(p)
    run_append(p, gpu.kv, news, x)
    for side in range(2):
        append64(kind, x[side], starts(news), p.lens, p.tables, p.codes[side], p.scales[side])
    same_state(p, gpu.kv)
    at, q = starts(news), queries(p, sum(news), 8)
    out, lse = gpu.attend(t(q), 0.1, news)
    for b, n in enumerate(news):
        if n:
            gpu.near(b, q, out, lse, 0.1, at)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("most", [1, 3])
def test_as_many_sequences_as_there_may_be(kind, most):
    held = [5 * i % 37 for i in range(2048)]
    news = [1 + i % most for i in range(2048)]
    p = Paged([m + n for m, n in zip(held, news)], 1, 64, 16, kind, seed=most)
    for b, (m, n) in enumerate(zip(held, news)):
        for i in range(m, m + n):
            for side in range(2):
                p.codes[side][p.tables[b, i // 16], :, i % 16] = 127
                if i % 16 == 0:
                    p.scales[side][p.tables[b, i // 16]] = np.nan
    x = [p.rng.standard_normal((sum(news), 1, 64)).astype(np.float16) for _ in "kv"]
    gpu = OnGpu(p)
    run_append(p, gpu.kv, None if most == 1 else news, x)
    for side in range(2):
        append64(kind, x[side], starts(news), p.lens, p.tables, p.codes[side], p.scales[side])
    same_state(p, gpu.kv)
    total = int(p.lens.sum())
    got = pkv.paged_kv_gather_q8(*gpu.kv, gpu.tables, t(starts(p.lens)), total, err_word=gpu.err)
    assert pkv.get_error(gpu.err) == 0
    for side in range(2):
        want = np.concatenate([p.tokens(side, b, int(n)) for b, n in enumerate(p.lens)])
        assert np.array_equal(got[side].cpu().numpy(), want.astype(np.float32).astype(np.float16))


@pytest.mark.parametrize("kind", KINDS)
def test_a_pool_beyond_32_bits(kind):
    """Blocks behind 4 GB of codes: what every call does there is, bit for bit, what it does
    in a small pool."""
    Hk, d, bs, lens, news = 8, 128, 16, [700, 90], [1, 1]
    small = Paged(lens, Hk, d, bs, kind, seed=13)
    NB = 290000
    assert NB * Hk * bs * d > 2 ** 32
    far = np.full(small.NB, -1, np.int32)  # block of the small pool -> of the large one
    used = sorted({int(i) for b, n in enumerate(lens) for i in small.tables[b, :-(-n // bs)]})
    far[used] = NB - 1 - 3 * np.arange(len(used))
    tables = np.where((small.tables >= 0) & (small.tables < small.NB), far[np.clip(small.tables, 0, small.NB - 1)],
                      NB + 7).astype(np.int32)
    a = OnGpu(small)
    large = [torch.empty(NB, *x.shape[1:], dtype=x.dtype, device="cuda") for x in a.kv]
    to, frm = torch.from_numpy(far[used].astype(np.int64)).cuda(), torch.tensor(used, device="cuda")
    for x, y in zip(large, a.kv):
        x[to] = y[frm]
    pools = ((a.kv, a.tables), (large, t(tables)))
    q, many = queries(small, 2, 32), queries(small, 150, 32)
    x = [queries(small, 2, Hk) for _ in "kv"]
    y = [queries(small, 150, Hk) for _ in "kv"]
    results = []
    for kv, tb in pools:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cut = dict(query_start=t(starts([90, 60])), max_q_len=90)
        pkv.paged_kv_append_q8(t(y[0]), t(y[1]), *kv, tb, a.lens, err_word=err, **cut)
        pkv.paged_kv_append_q8(t(x[0]), t(x[1]), *kv, tb, a.lens, err_word=err)
        one = pkv.paged_decode_attention_q8(t(q), *kv, tb, a.lens, 0.1, err_word=err)
        chunk = pkv.paged_decode_attention_q8(t(many), *kv, tb, a.lens, 0.1, err_word=err, **cut)
        k, v = pkv.paged_kv_gather_q8(*kv, tb, t(starts(lens)), sum(lens), err_word=err)
        src = tb[0, :2].contiguous()
        pkv.paged_kv_copy_blocks_q8(*kv, src, tb[0, 2:4].contiguous(), err_word=err)
        kk, _ = pkv.paged_kv_gather_q8(*kv, tb, t(starts([64, 0])), 64, err_word=err)
        assert pkv.get_error(err) == 0
        assert torch.equal(kk[:32].view(torch.uint8), kk[32:].view(torch.uint8))
        results.append([z.view(torch.uint8).cpu().numpy() for z in (one, chunk, k, v, kk)])
    for got, want in zip(*results):
        assert np.array_equal(got, want)
    assert np.isfinite(results[0][0].view(np.float16)).all()
