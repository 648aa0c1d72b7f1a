"""What the kernels' memory accesses rely on, as far as the sources show it (host only)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_213_gb300", "csrc")


def _code(path):
    """The file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_no_load_takes_the_path_for_memory_that_never_changes():
    """A kernel that is launched while the one before it in the stream still writes
    reads nothing that is read-only as long as it runs (the compiler takes that path by
    itself where pointers are __restrict__)."""
    found = [f for ext in ("cu", "cuh") for f in glob.glob(os.path.join(CSRC, f"*.{ext}"))]
    early = [f for f in found if "grid_dependency_wait" in _code(f)]
    assert len(found) > 20 and len(early) > 8
    for path in found:
        assert not re.search(r"__ldg\b|ld\.global\.nc", _code(path)), path
    for path in early:
        assert "__restrict__" not in _code(path), path
