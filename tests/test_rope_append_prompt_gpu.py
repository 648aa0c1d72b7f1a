"""The norm/rotation append at prompt sizes, where a lane takes four heads of a token:
head counts that leave a part of the four, every head size's kernel, both cache types,
padding tokens and queries in place."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from latent_util import assert_once_rounded, e4m3_values
from test_rope_append_gpu import Problem, _check, _run, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.library()


# tokens, heads, KV heads, head size, rotated entries, block size
SIZES = [(1203, 33, 3, 128, 128, 16), (1111, 32, 8, 128, 64, 32), (1999, 40, 5, 64, 64, 16),
         (2501, 1, 17, 64, 0, 64), (1153, 35, 1, 96, 48, 8), (4999, 3, 2, 256, 256, 16),
         (5003, 29, 1, 24, 16, 16)]


def _problem(T, H, Hk, d, rot, bs, **kw):
    lanes = 1
    while 8 * lanes < d:
        lanes *= 2
    assert T * (H + 2 * Hk) * lanes > 600000   # four heads a lane
    p = Problem(T, H, Hk, d, rot, bs, T + d, **kw)
    rng = np.random.default_rng(T)
    slots = p.slots.copy()
    keep = np.ones(T, bool)
    keep[rng.choice(T, 37, replace=False)] = False
    keep[[0, T - 1]] = [True, False]
    slots[~keep] = -1
    return p, slots, keep


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,d,rot,bs", SIZES)
def test_prompt(T, H, Hk, d, rot, bs, interleaved):
    p, slots, keep = _problem(T, H, Hk, d, rot, bs)
    before = torch.full((T, H, d), 9.0, dtype=torch.float16, device="cuda")
    res = _run(p, interleaved, q_out=before, slots=slots)
    assert res[3] == 0
    _check(p, interleaved, res, keep, np.full((T, H, d), 9.0, np.float16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,d,rot,bs", [s for s in SIZES if s[3] % 16 == 0])
def test_prompt_e4m3(T, H, Hk, d, rot, bs, interleaved):
    p, slots, keep = _problem(T, H, Hk, d, rot, bs, fp8=True, spread=20.0)
    ks, vs = 0.01, 0.07
    before = torch.full((T, H, d), 9.0, dtype=torch.float16, device="cuda")
    out, kc, vc, bits = _run(p, interleaved, scales=(ks, vs), q_out=before, slots=slots)
    assert bits == 0
    (q, qm), (k, km) = p.reference(interleaved)
    assert_once_rounded(out[keep], q[keep], qm[keep], "q")
    assert np.all(out[~keep] == 9.0)
    blk, row = p.slots[keep] // bs, p.slots[keep] % bs
    # half a step of E4M3 (2^-4 relative, 2^-10 among the subnormals) and the fp32
    # roundings before it
    x = k[keep] / np.float64(np.float32(ks))
    bound = np.abs(x) * 2.0 ** -4 + 2.0 ** -10 + 34 * 2.0 ** -24 * (km[keep] / ks + np.abs(x))
    assert np.all(np.abs(e4m3_values(kc[blk, :, row]) - np.clip(x, -448, 448)) <= bound)
    # V as the plain append stores it; every other row of both caches as it was
    k2, v2 = _t(p.kc), _t(p.vc)
    pkv.paged_kv_append_fp8(_t(p.k), _t(p.v), _t(slots), k2, v2, ks, vs)
    assert np.array_equal(v2.cpu().numpy(), vc)
    mine = np.zeros((kc.shape[0], bs), bool)
    mine[blk, row] = True
    assert np.array_equal(kc.transpose(0, 2, 1, 3)[~mine], p.kc.transpose(0, 2, 1, 3)[~mine])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,d,rot,bs", SIZES)
def test_prompt_in_place(T, H, Hk, d, rot, bs, interleaved):
    """q_out = q: the queries that another buffer gets, and padding tokens' as they were."""
    p, slots, keep = _problem(T, H, Hk, d, rot, bs)
    want = _run(p, interleaved, q_out=_t(p.q).clone(), slots=slots)[0]
    q, k, v = (x.contiguous() for x in p.device())
    rest = (_t(p.qw), _t(p.kw), 1e-5, _t(p.cs), _t(p.pos) if rot else None, _t(slots), _t(p.kc),
            _t(p.vc))
    got = pkv.paged_qk_norm_rope_append(q, k, v, *rest, interleaved=interleaved, q_out=q)
    assert got is q
    got = got.cpu().numpy()
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    assert np.array_equal(got[~keep].view(np.uint16), p.q[~keep].view(np.uint16))
