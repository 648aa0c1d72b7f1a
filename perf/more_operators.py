"""The cases on which the operators of the 8-bit caches with block scales are measured.

A cache of codes (E4M3 or int8) with one scale for each block of tokens and KV
head.  Three operators, as a serving loop uses them:

  append  the new tokens' K/V are quantised as they are written; a block's scale
          covers what the block holds, and grows by powers of two when a new
          token needs it (``paged_kv_append_q8``)
  attend  attention of each sequence's newest tokens over the codes: decode,
          drafts to verify, chunks of a prompt (``paged_decode_attention_q8``)
  gather  the first tokens of each sequence back in fp16, in token order
          (``paged_kv_gather_q8``)

With ``own`` false ``run`` computes each in its plain form (elementary torch
operations in fp32, rounded once); with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEVICE = "cuda"
F8 = torch.float8_e4m3fn


# --- cases -----------------------------------------------------------------

def listed():
    return [
        # one decode iteration of a 32-sequence batch: latency counts
        dict(name="append decode 32", op="append", seqs=32, low=127, high=2047, new_low=1,
             new_high=1, kv_heads=8, heads=32, dim=128, kind="e4m3", block=16),
        # five draft tokens a sequence, which straddle blocks
        dict(name="append drafts", op="append", seqs=24, low=200, high=2900, new_low=5,
             new_high=5, kv_heads=8, heads=32, dim=128, kind="int8", block=16),
        # prompts of a batch in one go, each behind a cached piece that ends inside a block
        dict(name="append prompts", op="append", seqs=5, low=37, high=37, new_low=411,
             new_high=2903, kv_heads=8, heads=64, dim=128, kind="e4m3", block=32),
        # the smallest decode: one short sequence
        dict(name="attend one", op="attend", seqs=1, low=699, high=699, new_low=1, new_high=1,
             kv_heads=8, heads=32, dim=128, kind="e4m3", block=16),
        # a decode step of a 32-sequence batch
        dict(name="attend batch 32", op="attend", seqs=32, low=127, high=2047, new_low=1,
             new_high=1, kv_heads=8, heads=32, dim=128, kind="e4m3", block=16),
        # many sequences from one token on, eight query heads on a KV head
        dict(name="attend mix 100", op="attend", seqs=100, low=0, high=1499, new_low=1,
             new_high=1, kv_heads=8, heads=64, dim=128, kind="int8", block=32),
        # long contexts: bytes alone
        dict(name="attend long", op="attend", seqs=8, low=32767, high=32767, new_low=1,
             new_high=1, kv_heads=8, heads=32, dim=128, kind="e4m3", block=64),
        # a smaller model: heads of 64, no sharing of KV heads
        dict(name="attend small heads", op="attend", seqs=12, low=300, high=5000, new_low=1,
             new_high=1, kv_heads=12, heads=12, dim=64, kind="int8", block=16),
        # draft tokens verified, five a sequence
        dict(name="attend verify 5", op="attend", seqs=24, low=200, high=2900, new_low=5,
             new_high=5, kv_heads=8, heads=32, dim=128, kind="e4m3", block=16),
        # ragged chunks of prompts behind cached contexts: products, not bytes
        dict(name="attend chunks", op="attend", seqs=3, low=1800, high=2500, new_low=150,
             new_high=700, kv_heads=8, heads=32, dim=128, kind="e4m3", block=16),
        # the cached part of three short prompts
        dict(name="gather short", op="gather", seqs=3, low=17, high=600, kv_heads=8, dim=128,
             kind="int8", block=16),
        # a batch of long cached contexts
        dict(name="gather long", op="gather", seqs=8, low=2000, high=16000, kv_heads=8, dim=128,
             kind="e4m3", block=64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "gather"])
    dim, kind, block = rng.choice([64, 128, 128]), rng.choice(["e4m3", "int8"]), \
        rng.choice([16, 16, 32, 64, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 8, 12])
    case = dict(op=op, kv_heads=kv, dim=dim, kind=kind, block=block)
    if op == "gather":
        seqs = _log(rng, 1, 32)
        high = _log(rng, 1, 8 * 9000 * 8 // (seqs * kv))
        return dict(case, seqs=seqs, low=max(0, high // rng.choice([1, 3, 10]) - 1), high=high)
    heads = kv * rng.choice([1, 2, 4, 4, 8])
    case["heads"] = heads
    if op == "append":
        seqs = _log(rng, 1, 128)
        new = _log(rng, 1, max(1, 8000 * 8 // (seqs * kv)))
        held = _log(rng, 1, 2000) - 1
        return dict(case, seqs=seqs, low=held // rng.choice([1, 2, 5]), high=held,
                    new_low=max(1, new // rng.choice([1, 1, 4])), new_high=new)
    new = rng.choice([1, 1, 1, 1, 2, 3, 4, 7, 8, 16, 33, 150, 500])
    seqs = _log(rng, 1, 128 if new <= 8 else 4)
    # products stay below the listed chunks', bytes below the long contexts'
    most = min(131072, 8 * 32768 * 8 * 128 // (seqs * kv * dim),
               92 * 10 ** 6 // (seqs * new * heads) - new)
    high = _log(rng, 1, max(2, most)) - 1
    return dict(case, seqs=seqs, low=high // rng.choice([1, 2, 8]), high=high,
                new_low=max(1, new // rng.choice([1, 1, 4])), new_high=new)


# --- sizes -----------------------------------------------------------------

def _spread(n, low, high):
    """Evenly spread in [low, high] and shuffled: the same for every seed, so that
    work(case) is fixed."""
    if n == 1:
        return [high]
    v = [low + (high - low) * i // (n - 1) for i in range(n)]
    return [v[(i * 7 + 3) % n] if n % 7 else v[(i * 5 + 3) % n] for i in range(n)]


def _lengths(case):
    """Cached tokens before the call, and new ones, of each sequence."""
    held = _spread(case["seqs"], case["low"], case["high"])
    if case["op"] == "gather":
        return held, [0] * len(held)
    return held, _spread(case["seqs"], case["new_low"], case["new_high"])[::-1]


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


def work(case):
    held, new = _lengths(case)
    k, d, block = case["kv_heads"], case["dim"], case["block"]
    if case["op"] == "append":
        touched = sum(-(-(m + n) // block) - m // block for m, n in zip(held, new))
        return dict(bytes=sum(new) * k * d * 2 * (2 + 1) + touched * (k * 2 * 8 + 4),
                    flops=sum(new) * k * d * 2 * 4)
    blocks = sum(-(-(m + n) // block) for m, n in zip(held, new))
    if case["op"] == "gather":
        return dict(bytes=sum(held) * k * d * 2 * (1 + 2) + blocks * (k * 2 * 4 + 4),
                    flops=sum(held) * k * d * 2)
    h, tokens = case["heads"], sum(held) + sum(new)
    pairs = sum(n * m + n * (n + 1) // 2 for m, n in zip(held, new))
    return dict(bytes=tokens * k * d * 2 + blocks * (k * 2 * 4 + 4)
                + sum(new) * h * (d * 2 * 2 + 4), flops=4 * pairs * h * d)


# --- inputs ----------------------------------------------------------------

def _limit(case):
    return 448.0 if case["kind"] == "e4m3" else 127.0


def _coded(case, x, scale):
    """Codes of x fp32 for scales that broadcast to it, saturated, to nearest even."""
    q = x / torch.where(scale > 0, scale, 1.0)
    q = q.clamp(-_limit(case), _limit(case))
    if case["kind"] == "e4m3":
        return q.to(F8).view(torch.uint8)
    return torch.nan_to_num(q).round().to(torch.int8)


def _valued(case, codes):
    return codes.view(F8).float() if case["kind"] == "e4m3" else codes.float()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=DEVICE, generator=g, dtype=torch.float32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEVICE)

    op, s = case["op"], dict(case)
    k, d, block = case["kv_heads"], case["dim"], case["block"]
    held, new = _lengths(case)
    lens = [m + n for m, n in zip(held, new)]
    need = [-(-m // block) for m in lens]
    pool, most = sum(need) + max(1, sum(need) // 10), max(max(need), 1)
    perm = torch.randperm(pool, device=DEVICE, generator=g).int()
    at = ints(_starts(need)[:-1])[:, None] + torch.arange(most, device=DEVICE)
    inside = torch.arange(most, device=DEVICE) < ints(need)[:, None]
    s["tables"] = torch.where(inside, perm[at.long().clamp(max=pool - 1)], 0).int().contiguous()
    s["lens"] = ints(lens)
    s["max_len"] = max(lens)
    # keys with a few loud channels, values of unit deviation: codes and block scales
    loud = 1 + 3 * (torch.rand(d, device=DEVICE, generator=g) < 0.05).float()
    for name, gain in (("k", loud), ("v", 1.0)):
        codes = torch.empty(pool, k, block, d, device=DEVICE,
                            dtype=torch.uint8 if case["kind"] == "e4m3" else torch.int8)
        scales = torch.empty(pool, k, device=DEVICE)
        step = max(1, (1 << 26) // (k * block * d))
        for i in range(0, pool, step):
            x = randn(*codes[i:i + step].shape) * gain
            scales[i:i + step] = x.abs().amax((2, 3)) / _limit(case)
            codes[i:i + step] = _coded(case, x, scales[i:i + step, :, None, None])
        s[name + "_cache"], s[name + "_scales"] = codes, scales
    if op == "gather":
        s["start"], s["total"] = ints(_starts(held)), sum(held)
        return s
    h, t = case["heads"], sum(new)
    s["max_new"] = max(new)
    s["q_start"] = None if max(new) == 1 else ints(_starts(new))
    # the fused projection's output: q, k and v are views of its rows
    qkv = randn(t, (h + 2 * k) * d)
    qkv[:, h * d:(h + k) * d] *= loud.repeat(k)
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in
                              qkv.half().split([h * d, k * d, k * d], dim=1))
    # logits of deviation about 1.7
    s["scale"] = 1.7 / math.sqrt(d * 1.75)
    if op == "attend" and own:
        import paged_kv_cache_213_gb300 as pkv
        s["workspace"] = torch.zeros(
            pkv.q8_plan(case["seqs"], t, s["max_new"], h, k, d, block, most, s["max_len"]),
            dtype=torch.uint8, device=DEVICE)
    return s


# --- one pass --------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "attend": _plain_attend, "gather": _plain_gather}[s["op"]](s)


def _caches(s):
    """The cache's state as values: codes as what they stand for, and the scales."""
    view = (lambda c: c.view(F8)) if s["kind"] == "e4m3" else (lambda c: c)
    return [view(s["k_cache"]), view(s["v_cache"]), s["k_scales"], s["v_scales"]]


def _own(s):
    import paged_kv_cache_213_gb300 as pkv
    cache = s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if s["op"] == "append":
        pkv.paged_kv_append_q8(s["k"], s["v"], *cache, s["tables"], s["lens"],
                               query_start=s["q_start"], max_q_len=s["max_new"])
        return _caches(s)
    if s["op"] == "gather":
        return pkv.paged_kv_gather_q8(*cache, s["tables"], s["start"], s["total"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    out = pkv.paged_decode_attention_q8(s["q"], *cache, s["tables"], s["lens"], s["scale"],
                                        query_start=s["q_start"], max_q_len=s["max_new"],
                                        max_context_len=s["max_len"],
                                        workspace=s["workspace"], lse=lse)
    return [out, lse]


def _query_starts(s):
    if s["q_start"] is None:
        return torch.arange(s["seqs"] + 1, device=DEVICE)
    return s["q_start"].long()


def _plain_append(s):
    block, limit = s["block"], _limit(s)
    start, lens = _query_starts(s), s["lens"].long()
    n = start[1:] - start[:-1]
    first = lens - n
    # the blocks that each sequence touches, and the position of each of their rows
    touched = first[:, None] // block + torch.arange((s["max_new"] + block - 2) // block + 1,
                                                     device=DEVICE)
    pos = touched[..., None] * block + torch.arange(block, device=DEVICE)
    seq, j = torch.nonzero(touched * block < lens[:, None], as_tuple=True)
    pos = pos[seq, j]                                                  # [m, block]
    old = (pos < first[seq, None])[:, None, :, None]
    fresh = (pos >= first[seq, None]) & (pos < lens[seq, None])
    token = (start[seq] - first[seq])[:, None] + pos
    token = torch.where(fresh, token, 0)
    fresh = fresh[:, None, :, None]
    phys = s["tables"][seq, touched[seq, j]].long()
    for new, name in ((s["k"], "k"), (s["v"], "v")):
        cache, scales = s[name + "_cache"], s[name + "_scales"]
        x = new[token].float().transpose(1, 2)                         # [m, heads, block, d]
        top = torch.where(fresh & x.isfinite(), x.abs(), 0).amax((2, 3))
        had = torch.where(old[:, :, 0, 0], scales[phys], 0)
        frac, power = torch.frexp(top / (had * limit))
        up = torch.where(frac > 0.5, power, power - 1).clamp(min=0)
        up = torch.where(had > 0, up, 0)
        scale = torch.where(had > 0, torch.ldexp(had, up), top / torch.full_like(top, limit))
        codes = cache[phys]
        kept = _valued(s, codes) * torch.ldexp(torch.ones_like(had), -up)[:, :, None, None]
        kept = _coded(s, kept, torch.ones_like(kept))
        kept = torch.where((up > 0)[:, :, None, None], kept, codes)
        fill = _coded(s, x, scale[:, :, None, None])
        cache[phys] = torch.where(fresh, fill, torch.where(old, kept, codes))
        scales[phys] = scale
    return _caches(s)


def _rows(s, name, most):
    """The first `most` tokens' values of every sequence: [seqs, kv heads, most, d] fp32."""
    blocks = s["tables"][:, :-(-most // s["block"])].long()
    x = _valued(s, s[name + "_cache"][blocks])                         # [b, blocks, h, block, d]
    x *= s[name + "_scales"][blocks][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :most]


def _plain_attend(s):
    b, h, k, d, most, mq = s["seqs"], s["heads"], s["kv_heads"], s["dim"], s["max_len"], s["max_new"]
    start = _query_starts(s)
    n = start[1:] - start[:-1]
    i = torch.arange(mq, device=DEVICE)
    at = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(b, mq, k, h // k, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(q, _rows(s, "k", most).transpose(2, 3)).mul_(s["scale"])
    last = s["lens"].long()[:, None] - n[:, None] + i
    hidden = torch.arange(most, device=DEVICE) > last[..., None]       # [b, mq, most]
    x.view(b, k, mq, h // k, most).masked_fill_(hidden[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _rows(s, "v", most)) / total
    lse = m + total.log()
    out, lse = (y.view(b, k, mq, h // k, -1).transpose(1, 2).flatten(2, 3) for y in (out, lse))
    if s["q_start"] is None:
        return [out[:, 0].half(), lse[:, 0, :, 0]]
    inside = i < n[:, None]
    return [out[inside].half(), lse[inside][..., 0]]


def _plain_gather(s):
    r = torch.arange(s["total"], device=DEVICE)
    seq = torch.searchsorted(s["start"], r.int(), right=True) - 1
    t = r - s["start"][seq]
    phys, row = s["tables"][seq, t // s["block"]].long(), t % s["block"]
    outs = []
    for name in ("k", "v"):
        x = _valued(s, s[name + "_cache"][phys, :, row]) * s[name + "_scales"][phys][..., None]
        outs.append(x.clamp(-65504, 65504).half())
    return outs


# --- the definitions in 64 bits ---------------------------------------------

def _e4m3_table():
    """What each of the 256 codes stands for."""
    c = torch.arange(256, device=DEVICE)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 512, (8 + m) * torch.pow(2.0, (e - 10).double()))
    return torch.where(c >= 128, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    held, new = _lengths(case)
    block, kv, d = s["block"], s["kv_heads"], s["dim"]
    table = _e4m3_table()

    def values(codes):
        return table[codes.long()] if s["kind"] == "e4m3" else codes.double()

    def tokens(name, b, m):
        """The first m tokens of sequence b: [m, kv heads, d]."""
        ids = s["tables"][b, :-(-m // block)].long()
        x = values(s[name + "_cache"][ids]) * s[name + "_scales"][ids].double()[..., None, None]
        return x.permute(0, 2, 1, 3).flatten(0, 1)[:m]

    if s["op"] == "gather":
        lists = [[tokens(n, b, m) for b, m in enumerate(held)] for n in "kv"]
        return [torch.cat(x) for x in lists]
    if s["op"] == "append":
        # code values as the definition has them: quotients in fp32, E4M3's last rounding left out
        out = []
        for name in "kv":
            x, scales = s[name], s[name + "_scales"]
            cache = values(s[name + "_cache"])
            at = 0
            for m, n, ids in zip(held, new, s["tables"].tolist()):
                for j in range(m // block, -(-(m + n) // block)):
                    low, high = max(m, j * block), min(m + n, (j + 1) * block)
                    y = x[at + low - m:at + high - m].double().transpose(0, 1)
                    top, top_code = y.abs().amax((1, 2)), _limit(case)
                    scale = (top / top_code).float().double()
                    if j * block < m:
                        old = scales[ids[j]].double()
                        reach = (top / (old * top_code).float().double()).float().double()
                        grow = torch.pow(2.0, torch.log2(reach).ceil().clamp(min=0))
                        scale = old * grow
                        kept = cache[ids[j], :, :m - j * block] / grow[:, None, None]
                        if s["kind"] == "int8":
                            kept = kept.round()
                        cache[ids[j], :, :m - j * block] = kept
                    y = (y / scale[:, None, None]).float().double()
                    if s["kind"] == "int8":
                        y = y.round()
                    cache[ids[j], :, low - j * block:high - j * block] = y.clamp(-top_code, top_code)
                    scales[ids[j]] = scale.float()
                at += n
            out.append((cache if s["kind"] == "e4m3" else cache.to(torch.int8), scales))
        return [out[0][0], out[1][0], out[0][1], out[1][1]]
    g, outs, lses = s["heads"] // kv, [], []
    starts = _starts(new)
    for b, (m, n) in enumerate(zip(held, new)):
        key, value = tokens("k", b, m + n), tokens("v", b, m + n)
        q = s["q"][starts[b]:starts[b + 1]].double()
        seen = torch.ones(n, m + n, dtype=torch.bool, device=DEVICE).tril(m)
        o, e = [], []
        for h in range(s["heads"]):
            x = ((q[:, h] @ key[:, h // g].T) * s["scale"]).where(seen, -math.inf)
            e.append(torch.logsumexp(x, -1))
            o.append(torch.softmax(x, -1) @ value[:, h // g])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
    return [torch.cat(outs), torch.cat(lses)]
