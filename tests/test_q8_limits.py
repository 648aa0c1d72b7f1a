"""Sizes that the 8-bit attention refuses before it asks for a device (host only)."""
import ctypes

import pytest

from paged_kv_cache_213_gb300 import build as pkv_build
from paged_kv_cache_213_gb300 import q8

UNSUPPORTED = -2


@pytest.fixture(scope="module")
def plan():
    pkv_build.build()
    lib = q8._lib()

    def status(num_seqs, new, H, Hk, length, d=128, bs=256):
        return lib.paged_decode_q8_plan(num_seqs, num_seqs * new, new, H, Hk, d, bs, -(-length // bs), length,
                                        ctypes.byref(ctypes.c_size_t()))
    return status


def test_units_stay_within_their_counters(plan):
    """A warp looks 63 units ahead of its own, and a grid's share is rounded up: counts next
    to 2^31 (127 heads of 16909320 tiles are 2^31 - 8) would not fit an int."""
    assert plan(1, 1, 127, 127, 16909320 * 16) == UNSUPPORTED
    assert plan(2047, 1, 1, 1, 1049088 * 16) == UNSUPPORTED  # 2^31 - 512
    assert plan(1, 1, 127, 127, 16908800 * 16) != UNSUPPORTED  # 2^31 - 66048
