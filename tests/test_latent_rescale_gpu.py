"""Latent attention where the running reference of a row moves while its products are
under way, so that the outputs so far are rescaled: logits that rise steeply along the
sequence for some rows, fall for others and stay level for the rest, over pieces of
many tiles.  Each test first counts, from the inputs, how often the reference moves."""
import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from latent_util import Paged, assert_attention

pytestmark = pytest.mark.gpu

# The kernels' rule: the reference is 6 below a row's first maximum, and moves to 6
# below a new one that lies more than 14 above it (base-2 logits).
HEAD, LAG = 6.0, 8.0
# how strongly a row follows the direction along which the keys grow
SLOPES = np.array([1.0, 0.0, -1.0, 0.5, 1.2])


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.library()


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _moves(tops):
    """How often the reference of each row moves after the first step, for maxima
    tops [steps, rows] (base 2; -inf: the row attends nothing there)."""
    ref = np.where(np.isfinite(tops[0]), tops[0] - HEAD, 0.0)
    moved = np.zeros(tops.shape[1], int)
    for m in tops[1:]:
        up = m - ref > HEAD + LAG
        ref = np.where(up, m - HEAD, ref)
        moved += up
    return moved


def _step_tops(s, size):
    """Maxima of logits s [rows, tokens] over steps of `size` tokens: [steps, rows]."""
    steps = -(-s.shape[1] // size)
    full = np.full((s.shape[0], steps * size), -np.inf)
    full[:, :s.shape[1]] = s
    return full.reshape(s.shape[0], steps, size).max(-1).T


def _attend(q, k, v, end, scale):
    """As latent_util.attend64, by matrix products: q [n, H, E], k [m, E] or [m, H, E];
    also the masked logits in base 2, [n, H, m]."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    qt = q.transpose(1, 0, 2)
    kt = k.T[None] if k.ndim == 2 else k.transpose(1, 2, 0)
    vt = v[None] if v.ndim == 2 else v.transpose(1, 0, 2)
    s = np.matmul(qt, kt) * scale                                  # [H, n, m]
    size = float(np.max(np.matmul(np.abs(qt), np.abs(kt)) * abs(scale)))
    s = np.where(np.arange(k.shape[0]) < np.asarray(end)[None, :, None], s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    p /= l
    out, mag = (np.matmul(p, x).transpose(1, 0, 2) for x in (vt, np.abs(vt)))
    lse = (m + np.log(l))[..., 0].T
    return (out, mag, lse, size), s.transpose(1, 0, 2) / np.log(2.0)


def _pieces(units, workers):
    """The even split of consecutive units: their worker."""
    each, more = divmod(units, workers)
    sizes = np.full(workers, each) + (np.arange(workers) < more)
    return np.repeat(np.arange(workers), sizes)


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("H,new,bs", [(16, 1, 16), (32, 1, 64), (64, 1, 32), (128, 1, 64),
                                      (7, 2, 16), (8, 4, 128), (16, 4, 16), (32, 4, 32)])
def test_absorbed_outputs_follow_the_reference(H, new, bs, R):
    rows = H * new
    tile_rows = 16 if rows <= 16 else 32 if rows <= 32 else 64 if rows <= 64 else 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    workers = sms // 2 if tile_rows == 128 else sms
    B = workers // 2
    rng = np.random.default_rng(R + H + new)
    lens = rng.integers(1100, 1400, B)
    E = R + 64
    p = Paged(lens, R, 64, bs, R + H)
    u = rng.choice([-1.0, 1.0], E)
    scale = 1.0 / np.sqrt(E)
    # base-2 logits of a slope of 1 rise by 11 a tile of 64 tokens
    per_token = 11.0 / 64 * np.log(2.0) / (scale * E)
    for b in range(B):
        t = np.arange(lens[b])
        p.rows[b] = (per_token * t[:, None] * u + p.rows[b].astype(np.float64)).astype(np.float16)
        p.cache[p.tables[b, t // bs], t % bs] = p.rows[b]
    slope = SLOPES[np.arange(B * rows) % len(SLOPES)].reshape(B * new, H)
    q = (slope[..., None] * u + 0.3 * rng.standard_normal((B * new, H, E))).astype(np.float16)
    qs = (new * np.arange(B + 1)).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((B * new, H), 7.0, device="cuda")
    args = (_t(q), _t(p.cache), _t(p.tables), _t(lens.astype(np.int32)), scale, R)
    kw = dict(query_start=_t(qs), max_q_len=new, max_context_len=int(lens.max()), err_word=err)
    out = pkv.paged_latent_attention(*args, lse=lse, **kw)
    assert pkv.get_error(err) == 0
    tiles = -(-lens // 64)
    worker = _pieces(int(tiles.sum()), workers)
    at, moved, longest = 0, 0, 0
    for b in range(B):
        r = slice(new * b, new * (b + 1))
        ref, s = _attend(q[r], p.rows[b], p.rows[b][:, :R], lens[b] - new + np.arange(new) + 1,
                         scale)
        assert_attention(out[r].cpu().numpy(), lse[r].cpu().numpy(), *ref, f"sequence {b}")
        tops = _step_tops(s.reshape(rows, -1), 64)
        mine = worker[at:at + tiles[b]]
        for w in np.unique(mine):
            moved += int(np.any(_moves(tops[mine == w]) > 0))
            longest = max(longest, int((mine == w).sum()))
        at += tiles[b]
    assert longest >= 8 and moved >= B
    again = pkv.paged_latent_attention(*args, **kw)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,ctas", [(80, 1), (40, 2), (9, 4)])
def test_expanded_outputs_follow_the_reference(H, ctas, d):
    """One, two and four CTAs for an item, each with at least three key steps."""
    n, m, step = 256, 1750, 96
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert ctas == (4 if 4 * H <= sms else 2 if 2 * H <= sms else 1)
    rng = np.random.default_rng(H + d)
    E = d + 64
    scale = 1.0 / np.sqrt(E)
    u = rng.choice([-1.0, 1.0], (H, E))
    u[:, d:] = u[0, d:]  # the rotated part is shared
    per_token = 11.0 / step * np.log(2.0) / (scale * E)
    t = np.arange(m)
    kv = rng.standard_normal((m, H, 2 * d))
    kv[..., :d] += per_token * t[:, None, None] * u[:, :d]
    kv = kv.astype(np.float16)
    kr = (per_token * t[:, None] * u[0, d:] + rng.standard_normal((m, 64))).astype(np.float16)
    slope = SLOPES[np.arange(n * H) % len(SLOPES)].reshape(n, H)
    q = (slope[..., None] * u + 0.3 * rng.standard_normal((n, H, E))).astype(np.float16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    args = (_t(q), _t(kv), _t(kr), _t(np.array([0, n], np.int32)), _t(np.array([0, m], np.int32)),
            scale, n, m)
    out = pkv.latent_prefill_attention(*args, lse=lse, err_word=err)
    assert pkv.get_error(err) == 0
    k = np.concatenate([kv[..., :d], np.repeat(kr[:, None], H, 1)], -1)
    ref, s = _attend(q, k, kv[..., d:], m - n + np.arange(n) + 1, scale)
    assert_attention(out.cpu().numpy(), lse.cpu().numpy(), *ref, "expanded")
    tops = _step_tops(s.reshape(n * H, m), step)
    cuts = [len(tops) * c // ctas for c in range(ctas + 1)]
    for a, b in zip(cuts, cuts[1:]):
        assert b - a >= 3 and np.mean(_moves(tops[a:b]) > 0) > 0.3
    again = pkv.latent_prefill_attention(*args)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
