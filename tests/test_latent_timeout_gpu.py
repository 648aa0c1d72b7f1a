"""The give-up paths of the latent attention kernels, run on purpose without a fault.

Every wait of theirs is bounded (about a second).  The test hook PKV_TEST_WAIT_POLLS=0
makes the products' first wait for a tile give up at once, as a rule while its copies
are in flight: the other roles stop, the copies land, and the call returns with
PKV_ERRBIT_TIMEOUT.  The next call is right, with the workspace as it was left.  The
batches leave the copies done with their part before the wait gives up (a tile or two
in all) or in the middle of it (many)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from latent_util import Paged, assert_attention, attend64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.library()


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _gives_up_then_recovers(call, monkeypatch):
    """call(err) with the hook, then without; what the second one returns."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    monkeypatch.setenv("PKV_TEST_WAIT_POLLS", "0")
    call(err)
    torch.cuda.synchronize()  # the kernel returned: no hang, the context is usable
    assert pkv.get_error(err) == pkv.PKV_ERRBIT_TIMEOUT
    monkeypatch.delenv("PKV_TEST_WAIT_POLLS")
    err.zero_()
    got = call(err)
    assert pkv.get_error(err) == 0
    return got


@pytest.mark.parametrize("R", [512, 256])
@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[40], [130, 1, 64], [9000, 5000, 70, 6000]])
def test_absorbed(lens, H, R, monkeypatch):
    p = Paged(lens, R, 64, 16, H + R)
    q = np.random.default_rng(H).standard_normal((len(lens), H, R + 64)).astype(np.float16)
    scale = 1.0 / np.sqrt(R + 64)
    most = max(lens)
    size = pkv.latent_plan(len(lens), len(lens), 1, H, R, 64, 16, p.MB, most)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    dev = [_t(x) for x in (q, p.cache, p.tables, p.lens.astype(np.int32))]
    lse = torch.zeros(len(lens), H, device="cuda")
    out = _gives_up_then_recovers(
        lambda err: pkv.paged_latent_attention(*dev, scale, R, max_context_len=most, workspace=ws,
                                               lse=lse, err_word=err), monkeypatch)
    for b, n in enumerate(lens):
        ref = attend64(q[b:b + 1], p.rows[b], p.rows[b][:, :R], [n], scale)
        assert_attention(out[b:b + 1].cpu().numpy(), lse[b:b + 1].cpu().numpy(), *ref, f"{b}")


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n,m,H", [(1, 1, 1), (200, 1000, 5), (200, 1000, 50), (300, 700, 90),
                                   (40, 90, 200)])
def test_expanded(n, m, H, d, monkeypatch):
    """Clusters of four (1 and 5 heads), of two (50) and single CTAs that take over items."""
    rng = np.random.default_rng(n + H + d)
    q = rng.standard_normal((n, H, d + 64)).astype(np.float16)
    kv = rng.standard_normal((m, H, 2 * d)).astype(np.float16)
    kr = rng.standard_normal((m, 64)).astype(np.float16)
    scale = 1.0 / np.sqrt(d + 64)
    dev = [_t(x) for x in (q, kv, kr, np.array([0, n], np.int32), np.array([0, m], np.int32))]
    lse = torch.zeros(n, H, device="cuda")
    out = _gives_up_then_recovers(
        lambda err: pkv.latent_prefill_attention(*dev, scale, n, m, lse=lse, err_word=err),
        monkeypatch)
    h = slice(0, H, max(1, H // 4))
    k = np.concatenate([kv[..., :d], np.repeat(kr[:, None], H, 1)], -1)
    ref = attend64(q[:, h], k[:, h], kv[:, h, d:], m - n + np.arange(n) + 1, scale)
    assert_attention(out[:, h].cpu().numpy(), lse[:, h].cpu().numpy(), *ref, "expanded")
