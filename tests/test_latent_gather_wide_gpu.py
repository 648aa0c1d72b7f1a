"""paged_latent_gather on rows so wide that a block of threads goes over its rows'
pieces several times, up to the widest."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from latent_util import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,P,bs", [(632, 8, 16), (576, 72, 16), (1024, 64, 32), (1000, 256, 7),
                                    (1984, 64, 16), (8, 2040, 64), (2040, 8, 1)])
def test_gather_of_wide_rows(R, P, bs):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens = [1, 40, 0, 17, 129]
    p = Paged(lens, R, P, bs, R + P)
    # the first two output rows belong to no sequence, nor do the last ones
    start = (2 + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    lat = torch.full((200, R), 5.0, dtype=torch.float16, device="cuda")
    rop = torch.full((200, P), 5.0, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [torch.from_numpy(x).cuda() for x in (p.cache, p.tables, start)]
    pkv.paged_latent_gather(*dev, 200, R, latents=lat, ropes=rop, err_word=err)
    assert pkv.get_error(err) == 0
    rows = np.concatenate(p.rows)
    lat, rop = lat.cpu().numpy(), rop.cpu().numpy()
    assert np.array_equal(lat[2:189], rows[:, :R]) and np.array_equal(rop[2:189], rows[:, R:])
    for x in (lat, rop):
        assert np.all(x[:2] == 5.0) and np.all(x[189:] == 5.0)
