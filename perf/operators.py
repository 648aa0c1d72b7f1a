"""The cases on which the operators around the paged caches are measured.

Five operators, as a serving loop uses them:

  qk_append      per-head RMS norm of queries and keys, rotation by position, and
                 the append of K/V into their cache slots, in one pass
                 (``paged_qk_norm_rope_append`` and its E4M3 form)
  latent_append  the same step for a latent cache: norm of the token's latent,
                 rotation of the shared key part and of the queries' part
                 (``paged_latent_append``)
  latent_attend  attention of new tokens over the paged latent cache, absorbed
                 form: keys are whole rows, values their first ``latent`` entries
                 (``paged_latent_attention``)
  latent_gather  a prompt's cached latents out of their blocks, in token order
                 (``paged_latent_gather``)
  latent_prefill causal attention over keys and values expanded from the
                 latents, for prompts (``latent_prefill_attention``)

With ``own`` false ``run`` computes each in its plain form (elementary torch
operations in fp32, rounded once); with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6


# --- cases -----------------------------------------------------------------

def listed():
    return [
        # one decode iteration of a 32-sequence batch: latency counts
        dict(name="qk append decode", op="qk_append", tokens=32, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, norm=True, fp8=False, block=16),
        # a long prompt into an E4M3 cache, half of each head rotated
        dict(name="qk append prompt e4m3", op="qk_append", tokens=8191, heads=64, kv_heads=8,
             dim=128, rot=64, interleaved=True, norm=True, fp8=True, block=32),
        # one decode iteration over a latent cache
        dict(name="latent append decode", op="latent_append", tokens=64, heads=32, latent=512,
             rope=64, interleaved=False, norm=True, block=16),
        # a long prompt into the latent cache
        dict(name="latent append prompt", op="latent_append", tokens=8003, heads=128, latent=512,
             rope=64, interleaved=True, norm=True, block=64),
        # the smallest decode: one short sequence, the heads one GPU of eight holds
        dict(name="latent decode one", op="latent_attend", seqs=1, low=700, high=700, new=1,
             heads=16, latent=512, rope=64, block=16),
        # a small batch's decode, few heads: bound by reading the cache
        dict(name="latent decode 32", op="latent_attend", seqs=32, low=128, high=2048, new=1,
             heads=16, latent=512, rope=64, block=16),
        # draft tokens verified, 4 a sequence
        dict(name="latent verify 4", op="latent_attend", seqs=16, low=500, high=8000, new=4,
             heads=32, latent=512, rope=64, block=32),
        # a full serving batch with every head on one GPU: bytes and products balance
        dict(name="latent decode 64 x 128 heads", op="latent_attend", seqs=64, low=3000,
             high=5000, new=1, heads=128, latent=512, rope=64, block=64),
        # the cached part of one short prompt
        dict(name="latent gather short", op="latent_gather", seqs=3, low=17, high=600,
             latent=512, rope=64, block=16),
        # a batch of long cached contexts before the next prompt chunk
        dict(name="latent gather long", op="latent_gather", seqs=8, low=2000, high=16000,
             latent=512, rope=64, block=64),
        # prompt chunks behind cached contexts, ragged
        dict(name="latent prefill chunks", op="latent_prefill", seqs=3, low=150, high=600,
             before=1500, heads=32, dim=128, rope=64),
        # one whole prompt, every head
        dict(name="latent prefill prompt", op="latent_prefill", seqs=1, low=4096, high=4096,
             before=0, heads=128, dim=128, rope=64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["qk_append", "latent_append", "latent_attend", "latent_attend",
                     "latent_gather", "latent_prefill"])
    if op == "qk_append":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8191), heads=kv * rng.choice([1, 2, 4, 8]),
                    kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75,
                    fp8=rng.random() < 0.5, block=rng.choice([16, 32, 64]))
    latent = rng.choice([512, 512, 256])
    if op == "latent_append":
        return dict(op=op, tokens=_log(rng, 1, 8003), heads=_log(rng, 1, 128), latent=latent,
                    rope=64, interleaved=rng.random() < 0.5, norm=rng.random() < 0.75,
                    block=rng.choice([16, 32, 64, 128]))
    if op == "latent_attend":
        # rows x tokens x sequences stay below the largest listed case
        seqs, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 96, 128])
        most = min(131072, 64 * 4000 * 128 // (seqs * new * heads), 64 * 4000 // seqs)
        high = _log(rng, 16, max(16, most))
        return dict(op=op, seqs=seqs, low=max(new, high // rng.choice([1, 2, 8])),
                    high=max(new, high), new=new, heads=heads, latent=latent, rope=64,
                    block=rng.choice([16, 32, 64, 128]))
    if op == "latent_gather":
        seqs = _log(rng, 1, 32)
        high = _log(rng, 1, 8 * 9000 // seqs)
        return dict(op=op, seqs=seqs, low=max(1, high // rng.choice([1, 3, 10])), high=high,
                    latent=latent, rope=64, block=rng.choice([16, 32, 64, 128]))
    seqs, heads = rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 6, 8, 32, 40, 128])
    high = _log(rng, 1, int(4096 * math.sqrt(128 / (heads * seqs)) / 1.5) if heads * seqs > 32
                else 4096)
    return dict(op=op, seqs=seqs, low=max(1, high // rng.choice([1, 2, 4])), high=high,
                before=rng.choice([0, 0, 33, high // 2]), heads=heads,
                dim=rng.choice([128, 128, 64]), rope=64)


# --- sizes -----------------------------------------------------------------

def _lengths(case):
    """Sequence lengths of a ragged batch, evenly spread in [low, high] and
    shuffled: the same for every seed, so that work(case) is fixed."""
    n, low, high = case["seqs"], case["low"], case["high"]
    if n == 1:
        return [high]
    lens = [low + (high - low) * i // (n - 1) for i in range(n)]
    return [lens[(i * 7 + 3) % n] if n % 7 else lens[(i * 5 + 3) % n] for i in range(n)]


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


def work(case):
    op = case["op"]
    if op == "qk_append":
        t, h, k, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        cache = 1 if case["fp8"] else 2
        return dict(bytes=t * (2 * h * d * 2 + 2 * k * d * (2 + cache) + case["rot"] * 4 + 12),
                    flops=t * (h + k) * d * 8)
    row = case["latent"] + case["rope"] if "latent" in case else 0
    if op == "latent_append":
        t = case["tokens"]
        return dict(bytes=t * (2 * row * 2 + 2 * case["heads"] * case["rope"] * 2
                               + case["rope"] * 4 + 12),
                    flops=t * (case["latent"] * 4 + (case["heads"] + 1) * case["rope"] * 3))
    lens = _lengths(case)
    if op == "latent_gather":
        n = sum(lens)
        return dict(bytes=n * row * 2 * 2 + 4 * sum(-(-m // case["block"]) for m in lens),
                    flops=0)
    if op == "latent_attend":
        new, h, r = case["new"], case["heads"], case["latent"]
        pairs = sum(new * m - new * (new - 1) // 2 for m in lens)
        return dict(bytes=sum(lens) * row * 2 + case["seqs"] * new * h * ((row + r) * 2 + 4),
                    flops=2 * pairs * h * (row + r))
    h, d, p, before = case["heads"], case["dim"], case["rope"], case["before"]
    pairs = sum(n * before + n * (n + 1) // 2 for n in lens)
    nq, nk = sum(lens), sum(lens) + before * len(lens)
    return dict(bytes=nq * h * ((d + p + d) * 2 + 4) + nk * (h * 2 * d + p) * 2,
                flops=2 * pairs * h * (d + p + d))


# --- inputs ----------------------------------------------------------------

def _rotations(rot, positions):
    """cos and sin of position * 10000^(-2i/rot), a table [positions, rot]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _tables(lens, block, g):
    """Physical blocks of each sequence in random order: [seqs, most] and the pool's size."""
    need = [-(-m // block) for m in lens]
    pool = sum(need) + max(1, sum(need) // 10)
    most = max(need)
    perm = torch.randperm(pool, device=DEVICE, generator=g).int()
    at = torch.tensor(_starts(need)[:-1], device=DEVICE)[:, None] \
        + torch.arange(most, device=DEVICE)
    inside = torch.arange(most, device=DEVICE) < torch.tensor(need, device=DEVICE)[:, None]
    return torch.where(inside, perm[at.clamp(max=pool - 1)], 0).int().contiguous(), pool


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=DEVICE, generator=g, dtype=torch.float32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEVICE)

    op, s = case["op"], dict(case)
    if op in ("qk_append", "latent_append"):
        t, block = case["tokens"], case["block"]
        pool = -(-t // block) + 8
        positions = 16384
        s["slots"] = torch.randperm(pool * block, device=DEVICE, generator=g)[:t].contiguous()
        s["positions"] = torch.randint(0, positions, (t,), device=DEVICE, generator=g).int()
        if op == "qk_append":
            h, k, d = case["heads"], case["kv_heads"], case["dim"]
            # the fused projection's output: q, k and v are views of its rows
            qkv = randn(t, (h + 2 * k) * d).half()
            s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in
                                      qkv.split([h * d, k * d, k * d], dim=1))
            s["q_weight"] = (1 + 0.1 * randn(d)).half() if case["norm"] else None
            s["k_weight"] = (1 + 0.1 * randn(d)).half() if case["norm"] else None
            s["rotations"] = _rotations(case["rot"], positions)
            kind = torch.uint8 if case["fp8"] else torch.float16
            s["k_cache"] = torch.zeros(pool, k, block, d, dtype=kind, device=DEVICE)
            s["v_cache"] = torch.zeros(pool, k, block, d, dtype=kind, device=DEVICE)
            s["k_scale"], s["v_scale"] = 0.0125, 0.01
        else:
            r, p, h = case["latent"], case["rope"], case["heads"]
            s["kv"] = randn(t, r + p).half()  # the down projection's output
            s["weight"] = (1 + 0.1 * randn(r)).half() if case["norm"] else None
            s["rotations"] = _rotations(p, positions)
            s["cache"] = torch.zeros(pool, block, r + p, dtype=torch.float16, device=DEVICE)
            # queries as projected (128 plain and p rotated entries a head), and the
            # absorbed queries whose last p entries the call fills
            s["q"] = randn(t, h, 128 + p).half()
            s["q_absorbed"] = torch.zeros(t, h, r + p, dtype=torch.float16, device=DEVICE)
        return s
    lens = _lengths(case)
    if op == "latent_prefill":
        h, d, p, before = case["heads"], case["dim"], case["rope"], case["before"]
        s["q_start"] = ints(_starts(lens))
        s["kv_start"] = ints(_starts([n + before for n in lens]))
        nq, nk = sum(lens), sum(lens) + before * len(lens)
        s["q"] = randn(nq, h, d + p).half()
        s["kv"] = randn(nk, h, 2 * d).half()
        s["k_rope"] = randn(nk, p).half()
        s["max_q"], s["max_kv"] = max(lens), max(lens) + before
        s["scale"] = 1.0 / math.sqrt(d + p)
        return s
    r, p, block = case["latent"], case["rope"], case["block"]
    s["tables"], pool = _tables(lens, block, g)
    s["cache"] = randn(pool, block, r + p).half()
    s["max_len"] = max(lens)
    if op == "latent_gather":
        s["start"], s["total"] = ints(_starts(lens)), sum(lens)
        return s
    s["lens"] = ints(lens)
    s["q"] = randn(case["seqs"] * case["new"], case["heads"], r + p).half()
    s["q_start"] = ints([i * case["new"] for i in range(case["seqs"] + 1)])
    # queries and latents of unit entries: logits of deviation about 1.7
    s["scale"] = 1.7 / math.sqrt(r + p)
    return s


# --- one pass --------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"qk_append": _plain_qk_append, "latent_append": _plain_latent_append,
            "latent_attend": _plain_attend, "latent_gather": _plain_gather,
            "latent_prefill": _plain_prefill}[s["op"]](s)


def _own(s):
    import paged_kv_cache_213_gb300 as pkv
    op = s["op"]
    if op == "qk_append":
        if s["fp8"]:
            q = pkv.paged_qk_norm_rope_append_fp8(
                s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["rotations"],
                s["positions"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                s["v_scale"], interleaved=s["interleaved"])
            return [q, s["k_cache"].view(torch.float8_e4m3fn),
                    s["v_cache"].view(torch.float8_e4m3fn)]
        q = pkv.paged_qk_norm_rope_append(
            s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["rotations"],
            s["positions"], s["slots"], s["k_cache"], s["v_cache"],
            interleaved=s["interleaved"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "latent_append":
        r = s["latent"]
        pkv.paged_latent_append(s["kv"], s["weight"], EPS, s["rotations"], s["positions"],
                                s["slots"], s["cache"], q_rope=s["q"][..., 128:],
                                q_out=s["q_absorbed"][..., r:], interleaved=s["interleaved"])
        return [s["cache"], s["q_absorbed"]]
    if op == "latent_gather":
        return pkv.paged_latent_gather(s["cache"], s["tables"], s["start"], s["total"],
                                       s["latent"])
    if op == "latent_attend":
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
        out = pkv.paged_latent_attention(s["q"], s["cache"], s["tables"], s["lens"], s["scale"],
                                         s["latent"], query_start=s["q_start"],
                                         max_q_len=s["new"], max_context_len=s["max_len"],
                                         lse=lse)
        return [out, lse]
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    out = pkv.latent_prefill_attention(s["q"], s["kv"], s["k_rope"], s["q_start"], s["kv_start"],
                                       s["scale"], s["max_q"], s["max_kv"], lse=lse)
    return [out, lse]


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotated(x, cs, interleaved):
    """x [tokens, heads, dim] fp32 with its first entries rotated by cs [tokens, rot]."""
    half = cs.shape[1] // 2
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def _codes(x, scale):
    """E4M3 codes of x / scale, saturating."""
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_qk_append(s):
    cs = s["rotations"][s["positions"].long()]
    q = _rotated(_normed(s["q"], s["q_weight"]), cs, s["interleaved"]).half()
    k = _rotated(_normed(s["k"], s["k_weight"]), cs, s["interleaved"])
    block, row = s["slots"] // s["block"], s["slots"] % s["block"]
    if s["fp8"]:
        s["k_cache"][block, :, row] = _codes(k, s["k_scale"])
        s["v_cache"][block, :, row] = _codes(s["v"].float(), s["v_scale"])
        return [q, s["k_cache"].view(torch.float8_e4m3fn),
                s["v_cache"].view(torch.float8_e4m3fn)]
    s["k_cache"][block, :, row] = k.half()
    s["v_cache"][block, :, row] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _plain_latent_append(s):
    r = s["latent"]
    cs = s["rotations"][s["positions"].long()]
    c = _normed(s["kv"][:, :r], s["weight"])
    k = _rotated(s["kv"][:, None, r:].float(), cs, s["interleaved"])[:, 0]
    s["cache"][s["slots"] // s["block"], s["slots"] % s["block"]] = torch.cat([c, k], 1).half()
    s["q_absorbed"][..., r:] = _rotated(s["q"][..., 128:].float(), cs, s["interleaved"]).half()
    return [s["cache"], s["q_absorbed"]]


def _rows_of(s, lens_max):
    """Cache rows of every sequence's tokens, padded to lens_max: [seqs, lens_max]."""
    t = torch.arange(lens_max, device=DEVICE)
    return s["tables"].long()[:, t // s["block"]] * s["block"] + t % s["block"]


def _plain_gather(s):
    n = torch.arange(s["total"], device=DEVICE)
    seq = torch.searchsorted(s["start"], n.int(), right=True) - 1
    t = n - s["start"][seq]
    rows = s["tables"][seq, t // s["block"]].long() * s["block"] + t % s["block"]
    got = s["cache"].flatten(0, 1)[rows]
    return [got[:, :s["latent"]].contiguous(), got[:, s["latent"]:].contiguous()]


def _plain_attend(s):
    b, new, h, r, most = s["seqs"], s["new"], s["heads"], s["latent"], s["max_len"]
    kv = s["cache"].flatten(0, 1)[_rows_of(s, most)].float()           # [b, most, row]
    q = s["q"].float().view(b, new * h, -1)
    x = torch.matmul(q, kv.transpose(1, 2)).mul_(s["scale"]).view(b, new, h, most)
    last = s["lens"].long()[:, None] - new + torch.arange(new, device=DEVICE)
    x.masked_fill_((torch.arange(most, device=DEVICE) > last[..., None])[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, new * h, most), kv[..., :r]).view(b, new, h, r) / total
    lse = (m + total.log())[..., 0]
    return [out.half().view(b * new, h, r), lse.view(b * new, h)]


def _padded(x, start, most):
    """Rows of each sequence, padded with its last: [seqs, most, ...]."""
    at = start[:-1].long()[:, None] + torch.arange(most, device=DEVICE)
    return x[at.clamp(max=x.shape[0] - 1)]


def _plain_prefill(s):
    d, mq, mk = s["dim"], s["max_q"], s["max_kv"]
    nq = (s["q_start"][1:] - s["q_start"][:-1]).long()
    q = _padded(s["q"], s["q_start"], mq).float().transpose(1, 2)      # [b, h, mq, d + p]
    kv = _padded(s["kv"], s["kv_start"], mk).float().transpose(1, 2)   # [b, h, mk, 2 d]
    kr = _padded(s["k_rope"], s["kv_start"], mk).float()[:, None]
    x = torch.matmul(q[..., :d], kv[..., :d].transpose(2, 3))
    x += torch.matmul(q[..., d:], kr.transpose(2, 3))
    x *= s["scale"]
    i, j = torch.arange(mq, device=DEVICE), torch.arange(mk, device=DEVICE)
    x.masked_fill_((j > i[:, None] + s["before"])[None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x -= m
    p = x.exp_()
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, kv[..., d:]) / total).transpose(1, 2)       # [b, mq, h, d]
    lse = (m + total.log())[..., 0].transpose(1, 2)
    inside = i < nq[:, None]
    return [out[inside].half(), lse[inside]]


# --- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("qk_append", "latent_append"):
        ang = s["rotations"].double()[s["positions"].long()]
        z = torch.complex(*ang.chunk(2, dim=1))[:, None]

        def turn(x):
            n = 2 * z.shape[-1]
            if s["interleaved"]:
                w = torch.view_as_real(torch.view_as_complex(
                    x[..., :n].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
            else:
                w = torch.complex(x[..., :n // 2].contiguous(),
                                  x[..., n // 2:n].contiguous()) * z
                w = torch.cat([w.real, w.imag], -1)
            return torch.cat([w, x[..., n:]], -1)

        def norm(x, w):
            x = x.double()
            return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1]
                                            + EPS).sqrt() * w.double()

        at = s["slots"]
        if op == "qk_append":
            caches = []
            for x, scale in ((turn(norm(s["k"], s["k_weight"])), s["k_scale"]),
                             (s["v"].double(), s["v_scale"])):
                n, h, block, d = s["k_cache"].shape
                c = torch.zeros(n * block, h, d, dtype=torch.float64, device=DEVICE)
                c[at] = (x / scale).clamp(-448, 448) if s["fp8"] else x
                caches.append(c.view(n, block, h, d).transpose(1, 2).contiguous())
            return [turn(norm(s["q"], s["q_weight"])), *caches]
        r = s["latent"]
        cache = s["cache"].double()
        flat = cache.view(-1, cache.shape[-1])
        flat[at, :r] = norm(s["kv"][:, :r], s["weight"])
        flat[at, r:] = turn(s["kv"][:, None, r:].double())[:, 0]
        q = s["q_absorbed"].double()
        q[..., r:] = turn(s["q"][..., 128:].double())
        return [cache, q]
    if op == "latent_gather":
        return None  # a copy: the plain form's values are exact
    lens = _lengths(case)
    outs, lses = [], []
    if op == "latent_attend":
        r, h, new = s["latent"], s["heads"], s["new"]
        for b, n in enumerate(lens):
            blocks = s["tables"][b, :-(-n // s["block"])].long()
            kv = s["cache"][blocks].flatten(0, 1)[:n].double()
            q = s["q"][b * new:(b + 1) * new].double()
            x = torch.einsum("ihc,tc->iht", q, kv) * s["scale"]
            seen = torch.ones(new, n, dtype=torch.bool, device=DEVICE).tril(n - new)
            x = x.where(seen[:, None], -math.inf)
            lses.append(torch.logsumexp(x, -1))
            outs.append(torch.einsum("iht,tc->ihc", torch.softmax(x, -1), kv[:, :r]))
        return [torch.cat(outs), torch.cat(lses)]
    d, before = s["dim"], s["before"]
    qs, ks = s["q_start"].tolist(), s["kv_start"].tolist()
    for b, n in enumerate(lens):
        m = n + before
        seen = torch.ones(n, m, dtype=torch.bool, device=DEVICE).tril(before)
        kr = s["k_rope"][ks[b]:ks[b + 1]].double()
        o, e = [], []
        for h in range(s["heads"]):
            q = s["q"][qs[b]:qs[b + 1], h].double()
            kv = s["kv"][ks[b]:ks[b + 1], h].double()
            x = (q @ torch.cat([kv[:, :d], kr], 1).T) * s["scale"]
            x = x.where(seen, -math.inf)
            e.append(torch.logsumexp(x, -1))
            o.append(torch.softmax(x, -1) @ kv[:, d:])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
    return [torch.cat(outs), torch.cat(lses)]
