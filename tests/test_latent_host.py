"""Host refusals of the norm/rotation append and of the latent cache's entry
points: bad arguments return before any CUDA work, so these run without a GPU."""
import os
import re

import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from paged_kv_cache_213_gb300 import build as pkv_build
from paged_kv_cache_213_gb300 import latent, rope

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096  # an aligned address that no refused call follows
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    latent._lib()
    return rope._lib()


def _call(fn, base, **change):
    args = {**base, **change}
    assert set(args) == set(base)
    return fn(*args.values())


QK = dict(q_out=P, q=P, k=P, v=P, q_stride=512, k_stride=128, v_stride=128, q_weight=P, k_weight=P,
          eps=1e-6, cos_sin=P, positions=P, max_positions=64, rot_dim=64, interleaved=0, slots=P,
          k_cache=P, v_cache=P, num_tokens=0, n_q_heads=8, n_kv_heads=2, head_dim=64,
          block_size=16, num_blocks=4, err=0, stream=0)


def test_qk_append_refusals(lib):
    fn = lib.paged_qk_norm_rope_append
    assert _call(fn, QK) == 0                       # no tokens: a no-op
    one = dict(QK, num_tokens=1)
    for change in (dict(num_tokens=-1), dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=60),
                   dict(block_size=0), dict(num_blocks=0), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=-16),
                   dict(interleaved=2), dict(q_stride=504), dict(k_stride=132),
                   dict(v_stride=120), dict(q_stride=-512), dict(q=0), dict(k=0), dict(v=0),
                   dict(q_out=0), dict(slots=0), dict(k_cache=0), dict(v_cache=0),
                   dict(cos_sin=0), dict(positions=0), dict(max_positions=0), dict(q=P + 8),
                   dict(k_weight=P + 2), dict(slots=P + 4), dict(cos_sin=P + 4),
                   dict(err=P + 1), dict(q_stride=1024)):   # in place with gaps
        assert _call(fn, one, **change) == INVALID, change
    assert _call(fn, one, head_dim=264, q_stride=8 * 264, k_stride=528, v_stride=528) == UNSUPPORTED


def test_qk_append_fp8_refusals(lib):
    fn = lib.paged_qk_norm_rope_append_fp8
    base = {}
    for k, x in QK.items():
        if k == "err":
            base |= dict(k_scale=0.1, v_scale=0.1)
        base[k] = x
    assert _call(fn, base) == 0
    for change in (dict(k_scale=0.0), dict(v_scale=float("inf")), dict(k_scale=float("nan")),
                   dict(head_dim=72, q_stride=576, k_stride=144, v_stride=144)):
        assert _call(fn, base, **change) == INVALID, change


LA = dict(kv=P, kv_stride=576, weight=P, eps=1e-6, cos_sin=P, positions=P, max_positions=64,
          interleaved=0, slots=P, cache=P, q_rope=P, q_token_stride=4 * 192, q_head_stride=192,
          q_out=2 * P, out_token_stride=4 * 576, out_head_stride=576, n_q_heads=4, num_tokens=0,
          latent_dim=512, rope_dim=64, block_size=16, num_blocks=4, err=0, stream=0)


def test_latent_append_refusals(lib):
    fn = lib.paged_latent_append
    assert _call(fn, LA) == 0
    assert _call(fn, LA, q_rope=0, q_out=0, n_q_heads=0) == 0
    one = dict(LA, num_tokens=1)
    for change in (dict(num_tokens=-1), dict(latent_dim=0), dict(latent_dim=500), dict(rope_dim=8),
                   dict(rope_dim=0), dict(block_size=0), dict(num_blocks=0), dict(eps=-1e-6),
                   dict(interleaved=-1), dict(max_positions=0), dict(kv_stride=568),
                   dict(kv_stride=580), dict(q_out=0), dict(q_rope=0), dict(n_q_heads=0),
                   dict(q_head_stride=56), dict(q_head_stride=68), dict(out_token_stride=576),
                   dict(q_token_stride=632), dict(q_out=P), dict(kv=0), dict(cache=0),
                   dict(slots=0), dict(positions=0), dict(cos_sin=0), dict(kv=P + 4),
                   dict(q_rope=P + 2), dict(weight=P + 8), dict(positions=P + 2)):
        assert _call(fn, one, **change) == INVALID, change
    assert _call(fn, one, latent_dim=1032, kv_stride=2048) == UNSUPPORTED
    assert _call(fn, one, rope_dim=272, kv_stride=2048) == UNSUPPORTED


AT = dict(out=P, q=P, cache=P, tables=P, lens=P, start=P, num_seqs=0, total_q=0, max_q_len=1,
          MB=8, NB=64, scale=0.1, H=16, R=512, P=64, bs=16, mcl=100, ws=0, ws_bytes=0, lse=0,
          err=0, stream=0)


def test_latent_attention_refusals(lib):
    fn = lib.paged_latent_attention
    for change in (dict(num_seqs=-1), dict(total_q=-1), dict(max_q_len=-1), dict(H=0), dict(MB=0),
                   dict(NB=0), dict(scale=float("inf")), dict(R=0), dict(P=-64),
                   dict(MB=1 << 27, bs=16), dict(start=0, num_seqs=3, total_q=2),
                   dict(start=0, num_seqs=2, total_q=2, max_q_len=2)):
        assert _call(fn, AT, **change) == INVALID, change
    for change in (dict(R=128), dict(R=576), dict(P=32), dict(bs=8), dict(bs=48), dict(bs=512),
                   dict(num_seqs=4097)):
        assert _call(fn, AT, **change) == UNSUPPORTED, change


def test_latent_attention_refuses_pools_beyond_32_bit_rows(lib):
    """Cache rows are numbered in 32 bits: refused before the workspace is looked at."""
    one = dict(AT, num_seqs=1, total_q=1)
    for blocks in (1 << 27, 1 << 60, (1 << 63) - 1):
        assert _call(lib.paged_latent_attention, one, NB=blocks) == UNSUPPORTED


GA = dict(latents=P, ropes=P, cache=P, tables=P, start=P, num_seqs=2, total=0, MB=8, NB=64, R=512,
          P=64, bs=16, err=0, stream=0)


def test_gather_refusals(lib):
    fn = lib.paged_latent_gather
    assert _call(fn, GA) == 0 and _call(fn, GA, num_seqs=0, total=5) == 0
    one = dict(GA, total=5)
    for change in (dict(num_seqs=-1), dict(total=-1), dict(MB=0), dict(NB=0), dict(R=0),
                   dict(R=20), dict(P=4), dict(bs=0), dict(latents=0), dict(ropes=0),
                   dict(cache=0), dict(tables=0), dict(start=0), dict(latents=P + 8),
                   dict(start=P + 2)):
        assert _call(fn, one, **change) == INVALID, change
    assert _call(fn, one, R=2048) == UNSUPPORTED
    assert _call(fn, one, total=1 << 31) == UNSUPPORTED


PF = dict(out=P, q=P, kv=P, kr=P, qs=P, ks=P, num_seqs=0, total_q=0, total_kv=0, max_q=4, max_kv=4,
          scale=0.1, H=2, d=128, P=64, lse=0, err=0, stream=0)


def test_prefill_refusals(lib):
    fn = lib.latent_prefill_attention
    assert _call(fn, PF) == 0 and _call(fn, PF, num_seqs=2, total_q=4, max_q=0) == 0
    one = dict(PF, num_seqs=1, total_q=4, total_kv=4)
    for change in (dict(num_seqs=-1), dict(total_q=-1), dict(total_kv=-1), dict(max_q=-1),
                   dict(max_kv=-1), dict(H=0), dict(d=0), dict(scale=float("nan")), dict(out=0),
                   dict(q=0), dict(kv=0), dict(kr=0), dict(qs=0), dict(ks=0), dict(q=P + 8),
                   dict(kr=P + 8), dict(lse=P + 2)):
        assert _call(fn, one, **change) == INVALID, change
    for change in (dict(d=96), dict(P=32), dict(H=70000)):
        assert _call(fn, one, **change) == UNSUPPORTED, change


def test_position_bit_is_its_own():
    bits = {}
    for name in ("pagedkv.h", "pagedkv_rope.h"):
        text = open(os.path.join(ROOT, "include", name)).read()
        for n, x in re.findall(r"^#define (PKV_ERRBIT_\w+) (0x[0-9a-f]+)", text, flags=re.M):
            bits[n] = int(x, 16)
    assert bits["PKV_ERRBIT_POSITION"] == pkv.PKV_ERRBIT_POSITION
    assert len(set(bits.values())) == len(bits) and all(b & (b - 1) == 0 for b in bits.values())


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(1, 2, 64, dtype=torch.float16)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_qk_norm_rope_append(x, x, x, None, None, 1e-6, None, None,
                                      torch.zeros(1, dtype=torch.int64), c, c)
    lc = torch.zeros(2, 16, 576, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_latent_attention(torch.zeros(1, 2, 576, dtype=torch.float16), lc, i[None], i,
                                   0.1, 512)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_latent_append(torch.zeros(1, 576, dtype=torch.float16), None, 1e-6,
                                torch.zeros(4, 64), i, i.long(), lc)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_latent_gather(lc, i[None], torch.zeros(2, dtype=torch.int32), 1, 512)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.latent_prefill_attention(torch.zeros(1, 2, 192, dtype=torch.float16),
                                     torch.zeros(1, 2, 256, dtype=torch.float16),
                                     torch.zeros(1, 64, dtype=torch.float16),
                                     torch.zeros(2, dtype=torch.int32),
                                     torch.zeros(2, dtype=torch.int32), 0.1, 1, 1)
