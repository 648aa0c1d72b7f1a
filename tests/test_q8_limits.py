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


def test_no_wait_of_the_kernel_for_many_rows_lasts_a_second(plan):
    """Some of its waits last a piece, all keys of a pair of tiles."""
    assert plan(1, 33, 1, 1, (1 << 25) + 1) == UNSUPPORTED
    assert plan(1, 5, 8, 1, 1 << 26) == UNSUPPORTED
    assert plan(1, 33, 1, 1, 1 << 25) != UNSUPPORTED
    assert plan(1, 32, 1, 1, 1 << 26) != UNSUPPORTED
