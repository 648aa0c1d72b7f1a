"""The give-up paths of the 8-bit attention kernels, run on purpose without a fault.

Every wait of theirs is bounded (about a second).  The test hook PKV_TEST_WAIT_POLLS=0
makes the first wait for a tile give up at once, as a rule while its copies are in
flight: the copies land, and the call returns with PKV_ERRBIT_TIMEOUT.  The next call is
right, with the workspace as it was left."""
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv

from q8_util import Paged
from test_q8_gpu import KINDS, OnGpu, queries, starts, t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hk,g,d,lens,news", [
    (2, 4, 128, [40], None),
    (2, 8, 64, [9000, 1, 70, 6000], None),
    (2, 4, 128, [4000, 30, 500], [3, 5, 8]),
    (1, 4, 128, [40], [40]),
    (2, 4, 64, [700, 90, 64], [300, 90, 64]),
    (1, 8, 128, [9000, 5000], [7, 90]),
])
def test_gives_up_then_recovers(kind, Hk, g, d, lens, news, monkeypatch):
    p = Paged(lens, Hk, d, 16, kind, seed=d)
    gpu, H = OnGpu(p), Hk * g
    many = {} if news is None else dict(query_start=t(starts(news)), max_q_len=max(news))
    T, most = (len(lens), 1) if news is None else (sum(news), max(news))
    q = queries(p, T, H)
    ws = torch.zeros(pkv.q8_plan(len(lens), T, most, H, Hk, d, 16, p.MB, max(lens)), dtype=torch.uint8,
                     device="cuda")
    for _ in range(2):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        monkeypatch.setenv("PKV_TEST_WAIT_POLLS", "0")
        pkv.paged_decode_attention_q8(t(q), *gpu.kv, gpu.tables, gpu.lens, 0.1, workspace=ws,
                                      max_context_len=max(lens), err_word=err, **many)
        torch.cuda.synchronize()  # the kernel returned: no hang, the context is usable
        monkeypatch.delenv("PKV_TEST_WAIT_POLLS")
        assert pkv.get_error(err) == pkv.PKV_ERRBIT_TIMEOUT
        assert not ws[:pkv.PKV_WORKSPACE_COUNTER_BYTES].any()
        gpu.check(q, 0.1, news, workspace=ws)
