"""Expanded latent attention over no keys at all: a padded batch without a token."""
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from paged_kv_cache_213_gb300 import build as pkv_build
from test_latent_host import INVALID, PF, _call


def test_no_keys_need_no_address():
    """Not refused for its arguments (without a GPU the launch fails instead)."""
    from paged_kv_cache_213_gb300 import latent
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    pkv_build.build()
    fn = latent._lib().latent_prefill_attention
    none = dict(PF, num_seqs=1, total_q=4, total_kv=0, kv=0, kr=0)
    assert _call(fn, none) != INVALID
    assert _call(fn, dict(none, total_kv=1)) == INVALID
    assert _call(fn, dict(none, q=0)) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 60, 200])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 2])
def test_no_keys(n, d, H):
    """Sequences without queries: nothing is written.  One with queries but no key is
    flagged."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    f16 = dict(dtype=torch.float16, device="cuda")
    q, kv, kr = torch.randn(3, H, d + 64).half().cuda(), torch.empty(0, H, 2 * d, **f16), torch.empty(0, 64, **f16)
    start = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, err = torch.full((3, H, d), 7.0, **f16), torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((3, H), 7.0, device="cuda")
    got = pkv.latent_prefill_attention(q, kv, kr, start, none, 0.1, 3, 5, out=out, lse=lse,
                                       err_word=err)
    assert got is out and pkv.get_error(err) == (pkv.PKV_ERRBIT_CONTEXT if n else 0)
    assert torch.all(out == 7.0) and torch.all(lse == 7.0)
