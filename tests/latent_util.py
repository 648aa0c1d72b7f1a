"""Plain 64-bit statements of the norm/rotation append and of latent attention,
seeded paged problems, and error bounds counted from the roundings."""
from __future__ import annotations

import numpy as np

U16 = 2.0 ** -11   # half a step of fp16, relative
U32 = 2.0 ** -24
TINY16 = 2.0 ** -25  # half a step of the fp16 subnormals


def table(rot, positions, seed=0):
    """A rotation table [positions, rot] fp32: cosines, then sines."""
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(positions)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def norm64(x, w, eps):
    x = x.astype(np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)


def turn64(x, cs, interleaved):
    """x [T, H, d] rotated by cs [T, rot]; also |a| + |b| of each entry's pair."""
    half = cs.shape[1] // 2
    cos, sin = cs[:, None, :half].astype(np.float64), cs[:, None, half:].astype(np.float64)
    y, mag = x.copy(), np.abs(x)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def assert_once_rounded(got16, ref, mag, what):
    """fp16 values of an fp32 computation rounded once: half a step of the
    result, and 32 fp32 roundings of the pair it came from (a sum of at most 1024
    squares kept in 8-entry pieces and a shuffle tree, a root, a division, two
    products, one rotation)."""
    err = np.abs(np.asarray(got16, np.float64) - ref)
    bound = U16 * np.abs(ref) + TINY16 + 32 * U32 * mag
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.3f} of the bound"


def e4m3_values(codes):
    c = np.asarray(codes, np.uint8).astype(np.int64)
    sign = np.where(c & 128, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return sign * np.where((c & 127) == 127, np.nan, v)


class Paged:
    """A latent cache in random physical order; every row that no sequence may
    read is NaN and every unused table entry is outside the pool."""

    def __init__(self, lens, R, P, bs, seed, poison=True):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int64)
        self.R, self.P, self.bs = R, P, bs
        need = [-(-int(n) // bs) for n in self.lens]
        self.MB = max(1, max(need))
        self.NB = sum(need) + 3
        perm = rng.permutation(self.NB)
        self.tables = np.full((len(lens), self.MB), self.NB + 7 if poison else 0, np.int32)
        self.cache = np.full((self.NB, bs, R + P), np.nan, np.float16)
        self.rows = []
        at = 0
        for b, n in enumerate(self.lens):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.tables[b, :need[b]] = ids
            x = rng.standard_normal((int(n), R + P)).astype(np.float16)
            t = np.arange(int(n))
            if n:
                self.cache[ids[t // bs], t % bs] = x
            self.rows.append(x)


def attend64(q, k, v, end, scale):
    """One sequence, one head group: q [n, H, E], k [m, E] or [m, H, E], v likewise;
    query i attends the first end[i] keys.  Returns out, sum_t p_t |v_t|, lse and
    the largest scale * sum |q k| (the logits' size, for the bound)."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    sub_k, sub_v = ("tc", "td") if k.ndim == 2 else ("thc", "thd")
    s = np.einsum(f"nhc,{sub_k}->nht", q, k) * scale
    size = float(np.max(np.einsum(f"nhc,{sub_k}->nht", np.abs(q), np.abs(k)) * abs(scale), initial=0.0))
    t = np.arange(k.shape[0])
    s = np.where(t < np.asarray(end)[:, None, None], s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    p /= l
    return (np.einsum(f"nht,{sub_v}->nhd", p, v), np.einsum(f"nht,{sub_v}->nhd", p, np.abs(v)),
            (m + np.log(l))[..., 0], size)


def assert_attention(got, lse, ref, mag, ref_lse, size, what):
    """Bounds of an attention output whose logits, statistics and sums are fp32 and
    whose weights and result are rounded to fp16:
      logits    each off by at most 64 fp32 roundings of scale * sum |q k| (the
                products of fp16 are exact; a tensor-core sum keeps fp32 partial
                sums of 16 products), so a weight by the factor 1 + 2 d,
                d = 64 U32 size
      weights   half an fp16 step each, and half a subnormal step (the largest
                weight is at least 1 before the division by their sum)
      result    half an fp16 step."""
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    d = 64 * U32 * (1 + size)
    bound = (U16 + 4 * d) * mag + U16 * np.abs(ref) + 2 * TINY16
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.3f} of the bound"
    e = np.abs(np.asarray(lse, np.float64) - ref_lse)
    assert np.all(e <= 2 * d + 8 * U32 * (1 + np.abs(ref_lse))), f"{what}: lse off by {e.max():.2e}"
