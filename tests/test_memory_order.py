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


def test_an_acquire_by_one_lane_comes_before_the_other_lanes_loads():
    """One lane counts an arrival with acquire order; the warp reads the records of those who
    came before.  A shuffle hands the count over but orders no memory: a __syncwarp() has
    to stand between (in the few-row kernel before the loop that reads starts again, in the
    many-row kernel at the head of the loop of joins)."""
    few = _code(os.path.join(CSRC, "q8_attention.cu"))
    after = few[few.index("atomic_add_acq_rel_gpu("):]
    until_break = after[:after.index("if (!whole) break;")]
    assert until_break.index("__shfl_sync(") < until_break.index("__syncwarp();")
    many = _code(os.path.join(CSRC, "q8_prefill.cu"))
    after = many[many.index("atomic_add_acq_rel_gpu("):]
    assert after.index("__syncwarp();") < after.index("__ldcg(")
    pipeline = _code(os.path.join(CSRC, "decode_pipeline.cu"))
    after = pipeline[pipeline.index("atomic_add_relaxed_gpu("):]
    assert after.index("__shfl_sync(") < after.index("__syncwarp();") < after.index("__threadfence();")


def test_a_scale_is_read_by_all_before_one_lane_writes_it():
    """All lanes of a team quantise by the old scale that they read; one of them writes the
    new one.  A barrier has to stand between, in both append kernels."""
    text = _code(os.path.join(CSRC, "q8_append.cu"))
    for kernel in ("q8_append_one_kernel", "q8_append_many_kernel"):
        body = text[text.index(kernel + "(const Q8AppendArgs a)"):]
        read, write = body.index("scales[cell] : 0.f"), body.index("scales[cell] = scale;")
        assert read < body.index("__syncwarp();", read) < write, kernel
