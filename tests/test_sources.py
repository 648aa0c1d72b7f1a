"""Statements about the sources that hold for every build of the library."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _native_sources():
    pkg = os.path.join(ROOT, "paged_kv_cache_213_gb300")
    found = [f for ext in ("cu", "cuh", "h", "cpp", "c")
             for f in glob.glob(os.path.join(pkg, "**", f"*.{ext}"), recursive=True)]
    assert len(found) > 20
    return found + glob.glob(os.path.join(ROOT, "include", "*.h"))


def test_no_copy_goes_to_several_ctas_at_once():
    """The library runs as replicas on several GPUs, on pools that it is only given an
    address of: every CTA copies for itself."""
    word = "multi" + "cast"
    for path in _native_sources():
        assert not re.search(word, open(path).read(), flags=re.I), path
