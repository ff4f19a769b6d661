"""The checked debug variant covers the kernels of the latent cache, the pages and
the rotations: each of their sources has range checks, named once.  Its GPU run
is in test_latent_debug_gpu.py."""

import os
import re

from exact_attention_fattn_gb300 import build


def test_every_kernel_has_range_checks():
    sites = []
    sources = [s for s in build.SOURCES if s.startswith(("fattn_latent_", "fattn_pages", "fattn_rope"))]
    texts = {s: open(os.path.join(build.CSRC, s)).read() for s in sources}
    with_kernels = [s for s in sources if "__global__" in texts[s]]
    assert len(with_kernels) == 5
    for s in with_kernels:
        calls = re.findall(r"dcheck\(.*?, (?:a|args|t)\.status,\s*(\d+)\)", texts[s], flags=re.S)
        assert calls, s
        sites += calls
    assert len(sites) == len(set(sites))


def test_ring_flag_is_taken():
    assert "-DFATTN_LATENT_MIN_RING" in build.DEBUG_FLAGS
