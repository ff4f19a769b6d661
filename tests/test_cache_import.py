"""The package imports, and its helpers work, on a torch that lacks the private
CUDA shortcuts of the cache's host path (as one built without CUDA does)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_cudaCachingAllocator_raw_alloc",
             "_cuda_cudaCachingAllocator_raw_delete"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import exact_attention_fattn_gb300 as F
assert F.fattn_fwd and F.fattn_cache_fwd
c = F.fattn_cache_alloc(2, 1, 64, page=32, device="cpu", bounds=True)
assert c.k.shape == (2, 1, 32, 64) and F.fattn_rope_table(4, 16, device="cpu").shape == (4, 16)
try:
    F.fattn_cache_fwd(torch.zeros((1, 1, 64), dtype=torch.bfloat16), c, *[torch.zeros(1, dtype=torch.int32)] * 3)
except ValueError as e:
    assert "GPU" in str(e)
else:
    raise AssertionError("a cache on the CPU was accepted")
"""


def test_import_without_torchs_private_names():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_alloc_refuses_what_no_call_takes():
    import pytest

    import exact_attention_fattn_gb300 as F

    assert F.fattn_cache_alloc(1, 1024, 64, page=32, device="cpu").k.shape[1] == 1024
    with pytest.raises(ValueError):
        F.fattn_cache_alloc(1, 1025, 64, page=32, device="cpu")
