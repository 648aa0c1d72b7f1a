"""Plain 64-bit statements of the 8-bit caches with block scales, seeded paged
problems, and error bounds counted from the roundings."""
from __future__ import annotations

import numpy as np

U16 = 2.0 ** -11   # half a step of fp16, relative
U32 = 2.0 ** -24
TINY16 = 2.0 ** -25  # half a step of the fp16 subnormals
LIMIT = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c & 128, -1.0, 1.0) * np.where((c & 127) == 127, np.nan, v)


E4M3 = _e4m3_table()
POSITIVE = E4M3[:127]


def values(kind, codes):
    return E4M3[codes] if kind == "e4m3" else codes.astype(np.float64)


def encode(kind, x):
    """Codes of x (doubles): to nearest even, saturated; NaN: the NaN code, or 0."""
    if kind == "int8":
        return np.nan_to_num(np.clip(np.rint(x), -127, 127)).astype(np.int8)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(POSITIVE, a), 1, 126)  # POSITIVE[hi - 1] < a <= POSITIVE[hi]
    low, up = a - POSITIVE[hi - 1], POSITIVE[hi] - a
    code = np.where((low < up) | ((low == up) & (hi % 2 == 1)), hi - 1, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def f32(x):
    with np.errstate(over="ignore"):
        return np.float64(np.float32(x))


def append64(kind, x, starts, lens, tables, codes, scales):
    """The append's definition, block by block and head by head, in place: x
    [T, Hk, d] fp16, codes [NB, Hk, bs, d], scales [NB, Hk] fp32."""
    bs, limit = codes.shape[2], LIMIT[kind]
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        m = L - n
        for j in range(m // bs, -(-L // bs) if n else 0):
            low, high = max(m - j * bs, 0), min(L - j * bs, bs)
            block = tables[b, j]
            for h in range(x.shape[1]):
                y = x[starts[b] + j * bs + low - m:starts[b] + j * bs + high - m, h].astype(np.float64)
                a = np.max(np.abs(y), where=np.isfinite(y), initial=0.0)
                had = float(scales[block, h]) if low else 0.0
                if had > 0:
                    k, r = 0, f32(a / f32(had * limit))
                    while r > 2.0 ** k:
                        k += 1
                    s = had * 2.0 ** k
                    if k:
                        old = values(kind, codes[block, h, :low]) * 2.0 ** -k
                        codes[block, h, :low] = encode(kind, old)
                else:
                    s = f32(a / limit)
                q = np.float64(np.float32(y / (s if s > 0 else 1.0)))
                codes[block, h, low:high] = encode(kind, q)
                scales[block, h] = s


class Paged:
    """8-bit caches in random physical order.  What no sequence may read is NaN (E4M3
    codes, scales) or a far code (int8), and unused table entries are outside the
    pool.  spread: block scales vary by 2^-spread to 2^spread."""

    def __init__(self, lens, Hk, d, bs, kind, seed, spread=0, extra=3):
        rng = np.random.default_rng(seed)
        self.rng, self.kind = rng, kind
        self.lens = np.asarray(lens, np.int64)
        need = [-(-int(n) // bs) for n in self.lens]
        self.MB = max(1, max(need, default=1))
        self.NB = sum(need) + extra
        perm = rng.permutation(self.NB)
        self.tables = np.full((len(need), self.MB), self.NB + 7, np.int32)
        self.tables[:, ::2] = -5
        dt = np.uint8 if kind == "e4m3" else np.int8
        shape = (self.NB, Hk, bs, d)
        self.codes = [np.full(shape, 127, dt) for _ in "kv"]
        self.scales = [np.full((self.NB, Hk), np.nan, np.float32) for _ in "kv"]
        at = 0
        for b, n in enumerate(self.lens):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.tables[b, :need[b]] = ids
            for side in range(2):
                for j, i in enumerate(ids):
                    rows = min(bs, int(n) - j * bs)
                    x = rng.standard_normal((Hk, rows, d))
                    s = np.abs(x).max((1, 2)) / LIMIT[kind]
                    s = s.astype(np.float32).astype(np.float64)
                    self.codes[side][i, :, :rows] = encode(kind, x / s[:, None, None])
                    self.scales[side][i] = s * 2.0 ** rng.integers(-spread, spread + 1, Hk)

    def tokens(self, side, b, n):
        """The first n tokens of sequence b as doubles: [n, Hk, d]."""
        bs = self.codes[0].shape[2]
        t = np.arange(n)
        ids = self.tables[b, t // bs]
        return values(self.kind, self.codes[side][ids, :, t % bs]) * \
            self.scales[side][ids][..., None].astype(np.float64)


    def spread_in_steps(self, b, n, keys):
        """[n, Hk]: the largest V scale in a token's step of `keys` tokens over its own."""
        bs = self.codes[0].shape[2]
        own = self.scales[1][self.tables[b, np.arange(n) // bs]].astype(np.float64)
        most = np.repeat(np.maximum.reduceat(own, np.arange(0, n, keys)), keys, axis=0)[:n]
        return np.where(own > 0, most / np.where(own > 0, own, 1.0), 1.0)


def attend64(q, k, v, scale, spread=None):
    """One sequence: q [n, H, d], k, v [m, Hk, d]; query i attends the first m - n +
    i + 1 keys.  Returns out, sum_t p_t |v_t|, lse, the largest scale * sum |q k|,
    and sum |v_t| / l over the tokens whose weight is below 2^-8 of the largest.  spread
    [m, Hk]: that sum is of spread |v_t|, over weights below 2^-8 spread."""
    n, H, d = q.shape
    m, Hk, _ = k.shape
    g = H // Hk
    q = q.astype(np.float64).reshape(n, Hk, g, d)
    s = np.einsum("nhgc,thc->nhgt", q, k) * scale
    size = float(np.max(np.einsum("nhgc,thc->nhgt", np.abs(q), np.abs(k)) * abs(scale), initial=0.0))
    seen = np.arange(m) <= m - n + np.arange(n)[:, None]
    s = np.where(seen[:, None, None], s, -np.inf)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    l = p.sum(-1, keepdims=True)
    spread = np.ones((m, Hk)) if spread is None else spread
    small = np.einsum("nhgt,thc->nhgc", (p < 2.0 ** -8 * spread.T[:, None]) & seen[:, None, None],
                      spread[..., None] * np.abs(v)) / l
    p /= l
    out, mag = (np.einsum("nhgt,thc->nhgc", p, x) for x in (v, np.abs(v)))
    lse = (top + np.log(l))[..., 0]
    return [x.reshape(n, H, -1) for x in (out, mag)] + [lse.reshape(n, H), size, small.reshape(n, H, -1)]


def assert_attention(got, lse, ref, what):
    """Bounds of an attention output whose logits, statistics and sums are fp32 and
    whose weights (times the block's V scale over a reference) and result are fp16:
      logits    each off by at most 64 fp32 roundings of scale * sum |q k|, so a
                weight by the factor 1 + 2 d, d = 64 U32 (1 + size)
      weights   half an fp16 step each; where the product with the scales' ratio is
                below fp16's normal numbers, half a subnormal step.  The ratio is at
                least 1/64 and a row's largest weight at least 1, so that takes a
                weight below 2^-8 of the largest, and costs it 64 * TINY16 of |v|.  Where
                keys of several blocks share a reference, that of the largest V scale
                in the step, both are larger by what the key's scale is smaller
      result    half an fp16 step."""
    out, mag, ref_lse, size, small = ref
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    d = 64 * U32 * (1 + size)
    bound = (U16 + 4 * d) * mag + U16 * np.abs(out) + 2 * TINY16 + 64 * TINY16 * small
    err = np.abs(got - out)
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.3f} of the bound"
    e = np.abs(np.asarray(lse, np.float64) - ref_lse)
    assert np.all(e <= 2 * d + 8 * U32 * (1 + np.abs(ref_lse))), f"{what}: lse off by {e.max():.2e}"
