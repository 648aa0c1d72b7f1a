"""The package imports, and its host parts work, on a torch that was built without
CUDA (which lacks the functions that ask for the current device and stream)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
import paged_kv_cache_213_gb300 as pkv
x = torch.zeros(1, 2, 64, dtype=torch.float16)
for call in (lambda: pkv.paged_latent_gather(x, x, x, 1, 32),
             lambda: pkv.paged_qk_norm_rope_append(x, x, x, None, None, 0.0, None, None, x, x, x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("not refused")
from paged_kv_cache_213_gb300.blocks import BlockManager
m = BlockManager(8, 16)
print("fine")
"""


def test_import_without_cuda():
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", CODE], capture_output=True, text=True,
                       cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
