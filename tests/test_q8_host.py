"""The 8-bit caches with block scales without a GPU: host refusals, and the plain
statements of tests/q8_util.py against torch's E4M3 and against themselves."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_213_gb300 as pkv
from paged_kv_cache_213_gb300 import build as pkv_build
from paged_kv_cache_213_gb300 import q8

from q8_util import E4M3, LIMIT, Paged, append64, encode, values

P = 4096  # an aligned address that no refused call follows
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return q8._lib()


def _call(fn, base, **change):
    args = {**base, **change}
    assert set(args) == set(base)
    return fn(*args.values())


# what every call refuses about its cache
CACHE = [(dict(Hk=0), INVALID), (dict(d=0), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID),
         (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
         (dict(bs=48), UNSUPPORTED), (dict(bs=512), UNSUPPORTED), (dict(NB=1 << 60), UNSUPPORTED),
         (dict(NB=(1 << 31) // 2), UNSUPPORTED)]
POINTERS = [dict(k=0), dict(v=0), dict(ks=0), dict(vs=0), dict(k=P + 8), dict(v=P + 4), dict(ks=P + 2)]

AP = dict(k_new=P, v_new=P, k_stride=128, v_stride=128, start=P, tables=P, lens=P, num_seqs=1, total=2,
          max_q_len=2, MB=8, k=P, v=P, ks=P, vs=P, kind=0, Hk=2, d=64, bs=16, NB=64, err=0, stream=0)


def test_append_refusals(lib):
    fn = lib.paged_kv_append_q8
    for change in (dict(total=0), dict(num_seqs=0), dict(max_q_len=0)):
        assert _call(fn, AP, **change) == 0, change
    for change in POINTERS + [dict(kind=2), dict(kind=-1), dict(num_seqs=-1), dict(total=-1), dict(max_q_len=-1),
                              dict(MB=0), dict(start=0), dict(start=0, num_seqs=2), dict(k_stride=120),
                              dict(v_stride=132), dict(k_stride=-128), dict(k_new=0), dict(v_new=0),
                              dict(tables=0), dict(lens=0), dict(k_new=P + 8), dict(tables=P + 2),
                              dict(err=P + 1), dict(start=P + 2)]:
        assert _call(fn, AP, **change) == INVALID, change
    for change, status in CACHE:
        assert _call(fn, AP, **{**change, "k_stride": 1024, "v_stride": 1024}) == status, change
    assert _call(fn, AP, num_seqs=2049) == UNSUPPORTED


AT = dict(out=P, q=P, q_stride=256, k=P, v=P, ks=P, vs=P, kind=1, tables=P, lens=P, start=P, num_seqs=0, total_q=0,
          max_q_len=1, MB=8, NB=64, scale=0.1, H=4, Hk=2, d=64, bs=16, mcl=100, ws=0, ws_bytes=0, lse=0, err=0,
          stream=0, flags=0)


def test_attention_refusals(lib):
    fn = lib.paged_decode_attention_q8
    assert _call(fn, AT) == 0 and _call(fn, AT, num_seqs=2, total_q=4, max_q_len=0) == 0
    for change in (dict(kind=2), dict(num_seqs=-1), dict(total_q=-1), dict(max_q_len=-1), dict(H=0), dict(H=3),
                   dict(MB=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=1e38),
                   dict(MB=1 << 27), dict(start=0, num_seqs=3, total_q=2), dict(start=0, num_seqs=2, total_q=2,
                                                                               max_q_len=2),
                   dict(q_stride=248), dict(q_stride=260), dict(flags=2), dict(flags=1 << 31)):
        assert _call(fn, AT, **change) == INVALID, change
    for change, status in CACHE:
        assert _call(fn, AT, **{**change, "q_stride": 4096}) == status, change
    for change in (dict(num_seqs=2049), dict(total_q=1 << 29), dict(max_q_len=1 << 29), dict(H=258)):
        assert _call(fn, AT, **change) == UNSUPPORTED, change


PL = dict(num_seqs=0, total_q=0, max_q_len=1, H=4, Hk=2, d=64, bs=16, MB=8, mcl=100)


def test_plan_refusals(lib):
    size = ctypes.c_size_t(7)

    def plan(**change):
        return lib.paged_decode_q8_plan(*{**PL, **change}.values(), ctypes.byref(size))

    assert plan() == 0 and size.value == 0 and plan(H=256) == 0
    for change in (dict(num_seqs=-1), dict(total_q=-1), dict(max_q_len=-1), dict(H=0), dict(H=3), dict(Hk=0),
                   dict(MB=0), dict(MB=1 << 27), dict(d=0), dict(bs=0)):
        assert plan(**change) == INVALID, change
    for change in (dict(num_seqs=2049), dict(H=258), dict(d=96), dict(bs=8), dict(max_q_len=1 << 29)):
        assert plan(**change) == UNSUPPORTED, change
    assert lib.paged_decode_q8_plan(*PL.values(), None) == 0  # the size is not asked for
    with pytest.raises(pkv.PagedKVError):
        pkv.q8_plan(2, 2, 1, 258, 2, 64, 16, 8)


GA = dict(ko=P, vo=P, k=P, v=P, ks=P, vs=P, kind=0, tables=P, start=P, num_seqs=2, total=5, MB=8, NB=64, Hk=2, d=64,
          bs=16, err=0, stream=0)


def test_gather_refusals(lib):
    fn = lib.paged_kv_gather_q8
    assert _call(fn, GA, total=0) == 0 and _call(fn, GA, num_seqs=0) == 0
    for change in POINTERS + [dict(kind=5), dict(num_seqs=-1), dict(total=-1), dict(MB=0), dict(ko=0), dict(vo=0),
                              dict(ko=P + 8), dict(tables=0), dict(start=0), dict(start=P + 2), dict(err=P + 2)]:
        assert _call(fn, GA, **change) == INVALID, change
    for change, status in CACHE:
        assert _call(fn, GA, **change) == status, change
    assert _call(fn, GA, total=1 << 31) == UNSUPPORTED and _call(fn, GA, num_seqs=2049) == UNSUPPORTED


CO = dict(k=P, v=P, ks=P, vs=P, src=P, dst=P, tokens=P, n=1, Hk=2, d=64, bs=16, NB=64, err=0, stream=0)


def test_copy_refusals(lib):
    fn = lib.paged_kv_copy_blocks_q8
    assert _call(fn, CO, n=0) == 0
    for change in POINTERS + [dict(n=-1), dict(src=0), dict(dst=0), dict(src=P + 1), dict(tokens=P + 2),
                              dict(err=P + 1)]:
        assert _call(fn, CO, **change) == INVALID, change
    for change, status in CACHE:
        assert _call(fn, CO, **change) == status, change


def test_constants():
    text = open(os.path.join(os.path.dirname(pkv_build.INCLUDE), "include", "pagedkv_q8.h")).read()
    assert f"PKV_Q8_E4M3 {q8._KINDS[torch.uint8]}" in text and f"PKV_Q8_INT8 {q8._KINDS[torch.int8]}" in text


def test_python_calls_refuse():
    c = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    s, i = torch.zeros(2, 1), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_append_q8(x, x, c, c, s, s, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_decode_attention_q8(x, c, c, s, s, i[None], i, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_gather_q8(c, c, s, s, i[None], torch.zeros(2, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_copy_blocks_q8(c, c, s, s, i, i)
    with pytest.raises(TypeError, match="int8"):
        pkv.paged_kv_append_q8(x, x, c.half(), c.half(), s, s, i[None], i)


# --- the plain statements ---------------------------------------------------

def test_codes_against_torch():
    assert np.array_equal(np.nan_to_num(E4M3), np.nan_to_num(
        torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()))
    x = np.random.default_rng(0).standard_normal(20000) * 2.0 ** np.random.default_rng(1).integers(-12, 9, 20000)
    mid = (E4M3[:126] + E4M3[1:127]) / 2  # ties
    x = np.concatenate([x, mid, -mid, [0.0, -0.0, 448, -448, 1e9, -np.inf, np.inf]])
    x = np.float64(np.float32(x))
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(encode("e4m3", x), want)
    assert encode("e4m3", np.array([np.nan]))[0] == 127 and encode("int8", np.array([np.nan]))[0] == 0
    assert list(encode("int8", np.array([0.5, 1.5, -2.5, 126.5, 127.5, -1e9, np.inf]))) == [0, 2, -2, 126, 127, -127, 127]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_statement(kind):
    """A prompt at once: every value off by half a step of its code; the same tokens in
    pieces: by the bound for pieces; what is not the call's stays."""
    rng = np.random.default_rng(5)
    n, Hk, d, bs = 50, 2, 64, 16
    x = rng.standard_normal((n, Hk, d)).astype(np.float16)
    p = Paged([n], Hk, d, bs, kind, seed=1)
    once = [p.codes[0].copy(), p.scales[0].copy()]
    append64(kind, x, [0, n], [n], p.tables, *once)
    parts = [p.codes[0].copy(), p.scales[0].copy()]
    for a, b in ((0, 7), (7, 8), (8, 37), (37, 50)):
        append64(kind, x[a:b], [0, b - a], [b], p.tables, *parts)
    t = np.arange(n)
    for (codes, scales), steps in ((once, 0.5), (parts, 1.0)):
        ids = p.tables[0, t // bs]
        s = scales[ids][..., None].astype(np.float64)
        got = values(kind, codes[ids, :, t % bs]) * s
        x64 = x.astype(np.float64)
        bound = steps * s if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(x64), steps * 2.0 ** -9 * s)
        assert np.all(np.abs(got - x64) <= bound * (1 + 1e-6))
        spare = [i for i in range(p.NB) if i not in ids]
        assert np.all(codes[spare] == 127) and np.all(np.isnan(scales[spare]))
        assert np.all(codes[p.tables[0, 3], :, 2:] == 127)
        top = np.abs(values(kind, codes[ids[:48], :, t[:48] % bs])).reshape(3, 16, Hk, d).max((1, 3))
        assert np.all(top > LIMIT[kind] / 2.3)
