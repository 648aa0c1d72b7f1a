"""The 8-bit attention where a KV head has more than 32 query rows (chunks of prompts,
long drafts, large groups), against its definition in 64 bits."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv

from q8_util import LIMIT, Paged
from test_q8_gpu import KINDS, OnGpu, marshalled, queries, starts, t  # noqa: F401

pytestmark = pytest.mark.gpu


def workspace(p, T, most, H, fill=0):
    _, Hk, bs, d = p.codes[0].shape
    size = pkv.q8_plan(len(p.lens), T, most, H, Hk, d, bs, p.MB, int(p.lens.max()))
    return torch.full((size,), fill, dtype=torch.uint8, device="cuda")


def counters(ws):
    return ws[:pkv.PKV_WORKSPACE_COUNTER_BYTES]


CHUNKS = [  # kv heads, group, d, block size, lengths, new tokens
    (2, 4, 128, 16, [1500, 300, 64], [500, 300, 64]),
    (1, 1, 64, 16, [700, 33], [300, 33]),
    (2, 8, 128, 32, [900, 257], [130, 256]),
    (1, 3, 64, 64, [500], [170]),
    (1, 5, 128, 128, [400, 90], [80, 7]),
    (1, 16, 128, 16, [700, 20, 1], [33, 3, 1]),
    (1, 71, 64, 16, [300, 40], [5, 1]),
    (1, 128, 128, 256, [600, 3], [4, 3]),
    (3, 6, 128, 16, [65, 64, 63, 129, 128], [65, 1, 63, 64, 0]),
    (1, 2, 128, 16, [17] * 20, [17] * 20),
    (4, 4, 128, 32, [5000], [9]),
    (1, 4, 64, 16, [6000, 0, 5], [200, 0, 5]),
    (8, 4, 128, 16, [1025, 2047], [256, 255]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,bs,lens,news", CHUNKS)
def test_chunks(kind, Hk, g, d, bs, lens, news, marshalled):
    p = Paged(lens, Hk, d, bs, kind, seed=5 * Hk + g)
    OnGpu(p).check(queries(p, sum(news), Hk * g), 1.1 / d ** 0.5, news)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,lens", [(1, 40, 128, [700, 0, 1, 64, 65, 0]), (2, 128, 64, [33, 400]),
                                         (1, 33, 64, [0, 0, 3000])])
def test_one_token_of_a_large_group(kind, Hk, g, d, lens, marshalled):
    """The form without query_start, in which a sequence may be empty."""
    p = Paged(lens, Hk, d, 16, kind, seed=g)
    OnGpu(p).check(queries(p, len(lens), Hk * g), 0.1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,lens,news", [
    (2, 4, 128, [4000, 70, 1000], [40, 70, 300]),
    (1, 8, 128, [20001], [6]),
    (8, 1, 64, [333] * 9, [100] * 9),
])
def test_the_same_again(kind, Hk, g, d, lens, news):
    """Bit for bit, whatever the order in which CTAs end, from a workspace that both this
    kernel and the one for few rows have used; its counters are zero after each call."""
    p = Paged(lens, Hk, d, 16, kind, seed=len(lens))
    gpu = OnGpu(p)
    q, one = queries(p, sum(news), Hk * g), queries(p, len(lens), Hk * g)
    ws = max(workspace(p, sum(news), max(news), Hk * g), workspace(p, len(lens), 1, Hk * g), key=len)
    first = gpu.check(q, 0.1, news, workspace=ws)
    decode = gpu.check(one, 0.1, workspace=ws)
    for i in range(20):
        again = gpu.attend(t(q), 0.1, news, workspace=ws, flags=pkv.PKV_TABLES_READY * (i % 2))
        assert all(np.array_equal(x, y) for x, y in zip(first, again))
        assert not counters(ws).any()
        again = gpu.attend(t(one), 0.1, workspace=ws)
        assert all(np.array_equal(x, y) for x, y in zip(decode, again))
        assert not counters(ws).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", [3, 12])
@pytest.mark.parametrize("gain", [0.0, 1.0, 30.0])
def test_block_scales_that_differ(kind, spread, gain):
    lens, news = [500, 37, 2000], [90, 37, 260]
    p = Paged(lens, 2, 128, 16, kind, seed=spread, spread=spread)
    p.scales[0][p.tables[0, 0]] *= 2.0 ** 4
    OnGpu(p).check(queries(p, sum(news), 8, gain), 0.05, news)


@pytest.mark.parametrize("kind", KINDS)
def test_logits_that_climb(kind):
    """Keys that grow along the sequence: every step moves the references."""
    Hk, d, L = 2, 128, 1600
    p = Paged([L], Hk, d, 16, kind, seed=2)
    for j in range(L // 16):
        p.scales[0][p.tables[0, j]] = 0.002 * (j + 1) / LIMIT[kind] * 4
        p.codes[0][p.tables[0, j], :, :, :] = np.abs(p.codes[0][p.tables[0, j]].astype(np.int16) % 100)
    OnGpu(p).check(np.abs(queries(p, 150, Hk * 4)), 0.3, [150])


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-20])
def test_scales_of_the_softmax(scale):
    p = Paged([130, 9, 60], 2, 64, 16, "int8", seed=1)
    OnGpu(p).check(queries(p, 130, 4), scale, [70, 9, 51])


def test_blocks_of_zeros():
    p = Paged([200, 40], 2, 128, 16, "e4m3", seed=4)
    for b, js in ((0, (0, 1, 2, 3, 4, 9)), (1, (0, 1, 2))):
        for j in js:
            for side in range(2):
                p.codes[side][p.tables[b, j]] = 0
                p.scales[side][p.tables[b, j]] = 0
    OnGpu(p).check(queries(p, 110, 8), 0.2, [70, 40])


def test_a_cached_nan_reaches_its_sequence_alone():
    p = Paged([100, 100, 150], 2, 128, 16, "e4m3", seed=4)
    p.codes[1][p.tables[1, 2], 0, 3, 5] = 127
    news = [50, 40, 50]
    out, _ = OnGpu(p).attend(t(queries(p, sum(news), 4)), 0.1, news)
    want = np.zeros(out.shape, bool)
    want[50:90, :2, 5] = True
    assert np.array_equal(np.isnan(out), want)


def test_a_nan_query_reaches_its_own_row_alone():
    p = Paged([300, 90], 2, 128, 16, "e4m3", seed=4)
    news = [100, 60]
    q = queries(p, sum(news), 8)
    q[37, 3, 9] = np.nan
    q[120, 5, 0] = np.inf
    out, _ = OnGpu(p).attend(t(q), 0.1, news)
    bad = ~np.isfinite(out).all(-1)
    assert bad[37, 3] and set(map(tuple, np.argwhere(bad))) <= {(37, 3), (120, 5)}


def test_queries_with_gaps_and_outputs_given():
    p = Paged([70, 300], 2, 128, 16, "int8", seed=9)
    gpu, news = OnGpu(p), [70, 111]
    q = queries(p, 181, 8)
    want = gpu.check(q, 0.1, news)
    wide = torch.full((181, 8 * 128 + 520), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 1024] = t(q).flatten(1)
    view = wide[:, 8:8 + 1024].unflatten(1, (8, 128))
    out = torch.empty(181, 8, 128, dtype=torch.float16, device="cuda")
    got = gpu.attend(view, 0.1, news, out=out)
    assert np.array_equal(got[0], want[0]) and np.array_equal(out.cpu().numpy(), want[0])


def test_rows_and_sequences_out_of_bounds():
    """Flagged, their rows left as they were, the others computed."""
    lens, news = [140, 150, 160, 170], [20, 30, 1, 140]
    p = Paged(lens, 2, 64, 16, "e4m3", seed=6)
    gpu = OnGpu(p)
    q, at = queries(p, sum(news), 4), starts(news)
    good = gpu.check(q, 0.1, news)[0]

    def run(lens, at, most, rows=len(q)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((rows, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((rows, 4), 7.0, device="cuda")
        pkv.paged_decode_attention_q8(t(np.resize(q, (rows, 4, 64))), *gpu.kv, gpu.tables,
                                      t(np.array(lens, np.int32)), 0.1, query_start=t(np.array(at, np.int32)),
                                      max_q_len=most, max_context_len=170, out=out, lse=lse, err_word=err)
        return pkv.get_error(err), out.cpu().numpy(), lse.cpu().numpy()

    for other in ([140, 10 ** 6, 160, 170], [140, -3, 160, 170], [140, 2, 160, 170]):
        bits, out, lse = run(other, at, 140)
        assert bits == pkv.PKV_ERRBIT_CONTEXT
        assert np.all(out[at[1]:at[2]] == 7) and np.all(lse[at[1]:at[2]] == 7)
        for b in (0, 2, 3):
            gpu.near(b, q, out, lse, 0.1, at)
    bits, out, _ = run(lens, at, 139)  # more new tokens than the host's bound
    assert bits == pkv.PKV_ERRBIT_CONTEXT and np.all(out[at[3]:] == 7)
    for bad in ([0, 20, 50, 51, 2 ** 31 - 1], [0, 20, 50, 2 ** 31 - 1, -2 ** 31], [-5, 20, 50, 51, 191]):
        assert run(lens, bad, 140)[0] == pkv.PKV_ERRBIT_CONTEXT
    # rows behind the last sequence are left as they were
    bits, out, _ = run(lens, at, 140, rows=len(q) + 150)
    assert bits == 0 and np.all(out[len(q):] == 7) and np.array_equal(out[:len(q)], good)


def test_bad_blocks_are_flagged():
    p = Paged([140, 150], 2, 128, 16, "int8", seed=6)
    gpu, news = OnGpu(p), [50, 60]
    q = queries(p, 110, 4)
    good = gpu.check(q, 0.1, news)[0]
    for bad in (-1, p.NB, 2 ** 31 - 1):
        tables = p.tables.copy()
        tables[0, 5] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pkv.paged_decode_attention_q8(t(q), *gpu.kv, t(tables), gpu.lens, 0.1, query_start=t(starts(news)),
                                            max_q_len=60, max_context_len=150, err_word=err)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_BLOCK_ID
        assert np.array_equal(out.cpu().numpy()[50:], good[50:])


def test_a_workspace_that_was_not_cleared_is_reported():
    p = Paged([5000], 1, 128, 16, "int8", seed=8)
    gpu = OnGpu(p)
    q = queries(p, 20, 8)
    ws = workspace(p, 20, 20, 8, fill=255)
    for _ in range(2):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.paged_decode_attention_q8(t(q), *gpu.kv, gpu.tables, gpu.lens, 0.1, workspace=ws, err_word=err,
                                      query_start=t(starts([20])), max_q_len=20, max_context_len=5000)
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_WORKSPACE
    pkv.paged_decode_workspace_clear(ws)
    gpu.check(q, 0.1, [20], workspace=ws)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("most", [1, 9])
def test_as_many_sequences_as_there_may_be(kind, most):
    lens = [1 + 7 * i % 41 for i in range(2048)]
    news = [min(n, most) for n in lens]
    p = Paged(lens, 1, 64, 16, kind, seed=most)
    gpu = OnGpu(p)
    q = queries(p, sum(news), 4)
    if most == 1:
        gpu.check(q, 0.1)
    else:
        gpu.check(q, 0.1, news)


def test_a_replayed_graph_and_two_streams():
    """Two captured calls with a workspace each, replayed on two streams at once with new
    inputs, and an eager call on a third."""
    p = Paged([700, 90, 333], 2, 128, 16, "e4m3", seed=8)
    gpu, news = OnGpu(p), [130, 90, 20]
    at = t(starts(news))
    jobs = []
    for _ in range(2):
        stream = torch.cuda.Stream()
        q = torch.zeros(240, 8, 128, dtype=torch.float16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(240, 8, device="cuda")
        ws = workspace(p, 240, 130, 8)

        def call():
            pkv.paged_decode_attention_q8(q, *gpu.kv, gpu.tables, gpu.lens, 0.1, query_start=at, max_q_len=130,
                                          max_context_len=700, out=out, lse=lse, workspace=ws, err_word=gpu.err)

        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            call()
            with torch.cuda.graph(graph, stream=stream):
                call()
        jobs.append((stream, graph, q, ws, out, lse))  # a graph keeps none of its call's memory
    for i in range(4):
        new = [queries(p, 240, 8) for _ in range(3)]
        for (stream, graph, q, *_), x in zip(jobs, new):
            with torch.cuda.stream(stream):
                q.copy_(torch.from_numpy(x))
                for _ in range(5):
                    graph.replay()
        gpu.check(new[2], 0.1, news)
        torch.cuda.synchronize()
        assert pkv.get_error(gpu.err) == 0
        for (*_, out, lse), x in zip(jobs, new):
            for b in range(3):
                gpu.near(b, x, out.cpu().numpy(), lse.cpu().numpy(), 0.1, starts(news))


def test_two_threads_at_once():
    """Calls of many sizes (each asks for its own shared memory) from two threads, on a
    stream each."""
    problems = []
    for n in (1, 40, 700):
        p = Paged([20 + i % 50 for i in range(n)], 1, 64, 16, "int8", seed=n)
        news = [min(12, int(x)) for x in p.lens]
        problems.append((OnGpu(p), news, queries(p, sum(news), 4), queries(p, n, 4)))
    want = [(gpu.check(q, 0.1, news), gpu.check(one, 0.1)) for gpu, news, q, one in problems]
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(30):
                    j = (i * (k + 1)) % len(problems)
                    gpu, news, q, one = problems[j]
                    for got, ref in zip((gpu.attend(t(q), 0.1, news), gpu.attend(t(one), 0.1)), want[j]):
                        assert all(np.array_equal(x, y) for x, y in zip(got, ref))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed, failed
