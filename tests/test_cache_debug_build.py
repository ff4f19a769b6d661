"""The checked debug variant covers the paged cache's kernels: each of their
sources has range checks, and the ring depth that its build asks for is one that
a source takes.  Its GPU run is in test_cache_debug_gpu.py."""

import os
import re

from exact_attention_fattn_gb300 import build


def _source(name):
    return open(os.path.join(build.CSRC, name)).read()


def test_every_cache_kernel_has_range_checks():
    with_kernels = [s for s in build.SOURCES if s.startswith("fattn_cache_") and "__global__" in _source(s)]
    assert len(with_kernels) == 5
    sites = []
    for s in with_kernels:
        calls = re.findall(r"dcheck\(.*?, (?:a|args)\.status,\s*(\d+)\)", _source(s), flags=re.S)
        assert calls, s
        sites += calls
    assert len(sites) == len(set(sites))          # a site names one check


def test_debug_flags_are_taken():
    every = "".join(_source(s) for s in build.SOURCES)
    for flag in build.DEBUG_FLAGS:
        name = flag[2:].split("=")[0]
        assert name in every or name == "FATTN_DEBUG", flag   # that one is read in a header
    assert any(f.startswith("-DFATTN_CACHE_") for f in build.DEBUG_FLAGS)
