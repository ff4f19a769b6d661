"""Kernels whose output may be their input read it by plain loads: the read-only path
(ld.global.nc) is for data that nothing writes while a kernel runs."""

import os
import re

import pytest

from exact_attention_fattn_gb300 import build


def source(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name,block", [
    ("fattn_rope.cu", r"const uint16_t\* x = a\.x.*?\n\}"),
    ("fattn_latent_append.cu", r"const uint16_t\* src = a\.q_rope.*?return;\n  \}"),
    ("fattn_cache_append.cu", r"uint4 w\[kQHeads\];.*?const Angles")])
def test_what_may_be_written_in_place_is_read_plainly(name, block):
    text = re.search(block, source(name), flags=re.S).group(0)
    base = {"fattn_rope.cu": "x", "fattn_latent_append.cu": "src", "fattn_cache_append.cu": r"a\.q"}[name]
    assert re.search(r"\*reinterpret_cast<const uint4\*>\(" + base, text)
    assert not re.search(r"(__ldg|ld\.global\.nc|__restrict__)[^;]*\b" + base + r"\b", text)
    assert "__restrict__" not in source(name)
