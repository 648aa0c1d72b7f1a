"""The norm/rotation append against its 64-bit statement, and with the decode
attention that reads what it wrote."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_213_gb300 as pkv
from gpu_util import assert_close
from latent_util import assert_once_rounded, e4m3_values, norm64, table, turn64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.library()


def _t(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Problem:
    def __init__(self, T, H, Hk, d, rot, bs, seed, norm=True, pad=8, fp8=False, spread=1.0):
        rng = np.random.default_rng(seed)
        # one fused projection's rows, with `pad` unused entries between tokens
        self.fused = (spread * rng.standard_normal((T, (H + 2 * Hk) * d + pad))).astype(np.float16)
        cut = [0, H * d, (H + Hk) * d, (H + 2 * Hk) * d]
        self.q, self.k, self.v = (self.fused[:, a:b].reshape(T, -1, d)
                                  for a, b in zip(cut, cut[1:]))
        self.qw = (1 + 0.2 * rng.standard_normal(d)).astype(np.float16) if norm else None
        self.kw = (1 + 0.2 * rng.standard_normal(d)).astype(np.float16) if norm else None
        self.pos = rng.integers(0, 500, T).astype(np.int32)
        self.cs = table(rot, 500) if rot else None
        NB = -(-T // bs) + 3
        self.slots = rng.permutation(NB * bs)[:T].astype(np.int64)
        kind = np.uint8 if fp8 else np.float16
        self.kc = rng.integers(0, 100, (NB, Hk, bs, d)).astype(kind)
        self.vc = rng.integers(0, 100, (NB, Hk, bs, d)).astype(kind)
        self.T, self.H, self.Hk, self.d, self.bs = T, H, Hk, d, bs

    def device(self):
        f = _t(self.fused)
        H, Hk, d = self.H, self.Hk, self.d
        q, k, v = (x.unflatten(1, (-1, d)) for x in
                   f[:, :(H + 2 * Hk) * d].split([H * d, Hk * d, Hk * d], 1))
        return q, k, v

    def reference(self, interleaved):
        q, k = norm64(self.q, self.qw, EPS), norm64(self.k, self.kw, EPS)
        if self.cs is None:
            return (q, np.abs(q)), (k, np.abs(k))
        c = self.cs[self.pos]
        return turn64(q, c, interleaved), turn64(k, c, interleaved)


def _run(p, interleaved=False, scales=None, q_out=None, slots=None, pos=None):
    q, k, v = p.device()
    kc, vc, err = _t(p.kc), _t(p.vc), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, k, v, _t(p.qw), _t(p.kw), EPS, _t(p.cs),
            _t(p.pos if pos is None else pos) if p.cs is not None else None,
            _t(p.slots if slots is None else slots), kc, vc)
    if scales:
        out = pkv.paged_qk_norm_rope_append_fp8(*args, *scales, interleaved=interleaved,
                                                q_out=q_out, err_word=err)
    else:
        out = pkv.paged_qk_norm_rope_append(*args, interleaved=interleaved, q_out=q_out,
                                            err_word=err)
    return out.cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), pkv.get_error(err)


def _check(p, interleaved, res, keep=None, q_before=None):
    out, kc, vc, _ = res
    keep = np.ones(p.T, bool) if keep is None else keep
    (q, qm), (k, km) = p.reference(interleaved)
    assert_once_rounded(out[keep], q[keep], qm[keep], "q")
    blk, row = p.slots[keep] // p.bs, p.slots[keep] % p.bs
    assert_once_rounded(kc[blk, :, row], k[keep], km[keep], "k")
    assert np.array_equal(vc[blk, :, row].view(np.uint16), p.v[keep].view(np.uint16))
    # every other row of the caches is as it was
    mine = np.zeros((kc.shape[0], p.bs), bool)
    mine[blk, row] = True
    for got, was in ((kc, p.kc), (vc, p.vc)):
        assert np.array_equal(got.transpose(0, 2, 1, 3)[~mine], was.transpose(0, 2, 1, 3)[~mine])
    if q_before is not None:
        assert np.array_equal(out[~keep], q_before[~keep])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,d,rot,bs", [
    (1, 1, 1, 64, 64, 16), (7, 8, 2, 128, 128, 16), (33, 5, 1, 128, 64, 1),
    (5, 4, 4, 96, 48, 32), (3, 6, 3, 80, 16, 8), (2, 2, 1, 256, 256, 64), (9, 3, 1, 8, 0, 16),
    (130, 32, 8, 128, 96, 16)])
def test_append(T, H, Hk, d, rot, bs, interleaved):
    p = Problem(T, H, Hk, d, rot, bs, 10 * T + d)
    res = _run(p, interleaved)
    assert res[3] == 0
    _check(p, interleaved, res)


def test_without_norm_is_exact_where_nothing_turns():
    """No weights and no rotation: the call is the plain append, bit for bit."""
    p = Problem(19, 4, 2, 64, 0, 16, 3, norm=False)
    out, kc, vc, bits = _run(p)
    assert bits == 0 and np.array_equal(out.view(np.uint16), p.q.view(np.uint16))
    k2, v2 = oracle.append(p.k, p.v, p.slots, p.kc, p.vc, p.bs)
    assert np.array_equal(kc.view(np.uint16), k2.view(np.uint16))
    assert np.array_equal(vc.view(np.uint16), v2.view(np.uint16))


def test_one_weight_only():
    p = Problem(6, 4, 2, 128, 128, 16, 4)
    p.kw = None
    _check(p, False, _run(p))


@pytest.mark.parametrize("spread", [1e-4, 200.0])
def test_small_and_large_values(spread):
    """Squares under and over fp16's range; a head of zeros stays zero."""
    p = Problem(8, 4, 2, 128, 128, 16, 5, spread=spread)
    p.fused[3] = 0
    res = _run(p)
    _check(p, False, res)
    assert not np.any(res[0][3])


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (112, 0)])
def test_e4m3(d, rot):
    p = Problem(37, 4, 2, d, rot, 16, 6 + d, fp8=True, spread=20.0)
    ks, vs = 0.01, 0.07   # some K values saturate: |k| / 0.01 above 448
    out, kc, vc, bits = _run(p, scales=(ks, vs))
    assert bits == 0
    (q, qm), (k, km) = p.reference(False)
    assert_once_rounded(out, q, qm, "q")
    blk, row = p.slots // p.bs, p.slots % p.bs
    for got, ref, mag, s in ((kc, k, km, ks), (vc, p.v.astype(np.float64), 0, vs)):
        x = ref / np.float64(np.float32(s))
        # half a step of E4M3 (2^-4 relative, 2^-10 among the subnormals) and the
        # fp32 roundings before it
        near = 34 * 2.0 ** -24 * (mag / s + np.abs(x))
        bound = np.abs(x) * 2.0 ** -4 + 2.0 ** -10 + near
        val = e4m3_values(got[blk, :, row])
        c = np.clip(x, -448, 448)
        assert np.all(np.abs(val - c) <= bound)
    assert np.any(np.abs(e4m3_values(kc[blk, :, row])) == 448)
    # V as the plain append stores it
    k2, v2 = _t(p.kc), _t(p.vc)
    pkv.paged_kv_append_fp8(_t(p.k), _t(p.v), _t(p.slots), k2, v2, ks, vs)
    assert np.array_equal(v2.cpu().numpy(), vc)


@pytest.mark.parametrize("scale", [0.0125, 1.0, 0.3333, 3e-5, 1e-20, 1e30, 5e-39, 117.25])
def test_e4m3_values_are_the_appends_for_every_fp16(scale):
    """V is divided by a corrected reciprocal: the codes of all fp16 patterns
    (infinities and NaN among them) are those of paged_kv_append_fp8."""
    bits = np.arange(65536, dtype=np.uint16).view(np.float16).reshape(64, 8, 128)
    v, slots = _t(bits), torch.arange(64, device="cuda")
    caches = [torch.zeros(4, 8, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    pkv.paged_kv_append_fp8(v, v, slots, caches[0], caches[1], scale, scale)
    pkv.paged_qk_norm_rope_append_fp8(v, v, v, None, None, 0.0, None, None, slots, caches[2],
                                      caches[3], scale, scale)
    assert torch.equal(caches[1], caches[3]) and torch.equal(caches[0], caches[2])


def test_padding_and_bad_tokens():
    """Negative slots are skipped; a slot beyond the pool and a position outside
    the table are flagged; the other tokens land, and skipped rows of q_out stay."""
    p = Problem(12, 4, 2, 64, 64, 16, 8)
    slots, pos = p.slots.copy(), p.pos.copy()
    slots[2], slots[5], pos[7], pos[9] = -1, p.kc.shape[0] * p.bs, 500, -3
    before = torch.full((12, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    res = _run(p, q_out=before, slots=slots, pos=pos)
    assert res[3] == pkv.PKV_ERRBIT_SLOT | pkv.PKV_ERRBIT_POSITION
    keep = np.ones(12, bool)
    keep[[2, 5, 7, 9]] = False
    _check(p, False, res, keep, np.full((12, 4, 64), 9.0, np.float16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 32), (128, 16), (80, 48), (128, 0)])
def test_entries_beyond_the_rotation_stay_bit_for_bit(d, rot, interleaved):
    """Without a norm, the entries that no rotation reaches are the input's bits:
    infinities, negative zeros and subnormals among them."""
    p = Problem(40, 4, 2, d, rot, 16, 31, norm=False)
    odd = np.array([np.inf, -np.inf, -0.0, 0.0, 2.0 ** -24, 65504.0], np.float16)
    for x in (p.q, p.k):
        x[..., rot:] = np.random.default_rng(3).choice(odd, x[..., rot:].shape)
    q, k, v = (_t(x) for x in (p.q, p.k, p.v))
    kc, vc = _t(p.kc), _t(p.vc)
    out = pkv.paged_qk_norm_rope_append(q, k, v, None, None, EPS, _t(p.cs),
                                        _t(p.pos) if rot else None, _t(p.slots), kc, vc,
                                        interleaved=interleaved).cpu().numpy()
    kc = kc.cpu().numpy()[p.slots // 16, :, p.slots % 16]
    assert np.array_equal(out[..., rot:].view(np.uint16), p.q[..., rot:].view(np.uint16))
    assert np.array_equal(kc[..., rot:].view(np.uint16), p.k[..., rot:].view(np.uint16))


def test_no_tokens():
    p = Problem(1, 4, 2, 64, 64, 16, 9)
    e = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    k = e[:, :2]
    out = pkv.paged_qk_norm_rope_append(
        e, k, k, None, None, EPS, _t(p.cs), torch.empty(0, dtype=torch.int32, device="cuda"),
        torch.empty(0, dtype=torch.int64, device="cuda"), _t(p.kc), _t(p.vc))
    assert out.shape == (0, 4, 64)


def test_in_place_and_graph():
    """q_out = q; captured on another stream and replayed on new inputs."""
    p = Problem(16, 8, 2, 128, 128, 16, 11)
    q0, k, v = (x.contiguous() for x in p.device())
    q, kc, vc = q0.clone(), _t(p.kc), _t(p.vc)
    rest = (_t(p.qw), _t(p.kw), EPS, _t(p.cs), _t(p.pos), _t(p.slots), kc, vc)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.paged_qk_norm_rope_append(q, k, v, *rest, q_out=q)
    q.copy_(q0)
    kc.copy_(_t(p.kc))
    vc.copy_(_t(p.vc))
    g.replay()
    torch.cuda.synchronize()
    _check(p, False, (q.cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), 0))


def test_decode_step_reads_what_it_wrote():
    """The layer's run: norm, rotation and append of each sequence's newest token,
    then the decode attention over the cache, against the oracle on the cache."""
    B, H, Hk, d, bs = 6, 8, 2, 128, 16
    rng = np.random.default_rng(21)
    lens = np.array([1, 17, 40, 16, 200, 33], np.int32)
    MB = 13
    NB = B * MB
    bt = rng.permutation(NB).reshape(B, MB).astype(np.int32)
    p = Problem(B, H, Hk, d, d, bs, 22)
    p.kc = rng.standard_normal((NB, Hk, bs, d)).astype(np.float16)
    p.vc = rng.standard_normal((NB, Hk, bs, d)).astype(np.float16)
    last = lens - 1
    p.slots = bt[np.arange(B), last // bs].astype(np.int64) * bs + last % bs
    p.pos = last.astype(np.int32)
    q, k, v = p.device()
    kc, vc = _t(p.kc), _t(p.vc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qr = pkv.paged_qk_norm_rope_append(q, k, v, _t(p.qw), _t(p.kw), EPS, _t(p.cs), _t(p.pos),
                                       _t(p.slots), kc, vc, err_word=err)
    scale = pkv.default_scale(d)
    out = pkv.paged_decode_attention(qr, kc, vc, _t(bt), _t(lens), scale, H, Hk, d, bs,
                                     max_context_len=200, err_word=err,
                                     flags=pkv.PKV_TABLES_READY)
    assert pkv.get_error(err) == 0
    _check(p, False, (qr.cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), 0))
    ref, _, _ = oracle.decode(qr.cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), bt, lens,
                              scale, H, Hk, d, bs)
    assert_close(out.cpu().numpy(), ref, what="step")
