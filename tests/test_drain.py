"""A kernel whose wait budget is short still waits for the copies and products
that it has in flight before it ends.  The drains' loop runs on the CPU, on a
barrier that completes late and a clock that the loop itself moves on."""

import os
import re
import subprocess

import pytest

from exact_attention_fattn_gb300 import build

PROGRAM = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
using std::max;
static long long now = 0;
static long long done_at = 0;
static long long clock64() { return now += 100; }
static bool mbar_try_wait(uint32_t, uint32_t) { return now >= done_at; }
static bool mbar_try_wait_cl(uint32_t, uint32_t) { return now >= done_at; }
%s
int main() {
  now = 0;
  done_at = 1000000;              // half a millisecond: a copy's time many times over
  bool ok = %s;
  now = 0;
  done_at = 1ll << 62;            // never: the wait ends all the same
  ok = ok && !%s;
  std::printf("%%d\n", ok);
  return !ok;
}
"""


@pytest.mark.parametrize("name", ["mbar_wait_drain", "mbar_drain_cl"])
def test_drains_outlast_a_short_budget(name, tmp_path):
    text = open(os.path.join(build.CSRC, "fattn_ptx.cuh")).read()
    body = re.search(r"__device__ __forceinline__ bool " + name + r"\(.*?\n}\n", text, flags=re.S).group(0)
    floor = re.search(r"constexpr long long kDrainCycles.*?;\n", text)
    src, exe = tmp_path / "drain.cpp", tmp_path / "drain"
    # a budget that a user can set, where the loop takes one
    call = f"{name}(0, 0, 1000)" if "budget" in body.split("{")[0] else f"{name}(0, 0)"
    src.write_text(PROGRAM % ((floor.group(0) if floor else "")
                              + body.replace("__device__ __forceinline__", "static"), call, call))
    subprocess.run([build._nvcc(), "-O2", "-std=c++17", "-cudart", "none", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
