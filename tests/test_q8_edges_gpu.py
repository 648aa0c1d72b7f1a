"""The 8-bit caches with block scales on the GPU, where a batch's shape, values or tables
are at the edge of what the header allows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv

from q8_util import Paged
from test_q8_gpu import OnGpu, queries, starts, t

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
