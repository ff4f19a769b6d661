"""How the roles of the latent attention's kernels wait for one another, on the CPU:
the counts of their barriers are taken from the sources and checked against every
order in which the warps that arrive may be."""

import itertools
import os
import re
import subprocess

from exact_attention_fattn_gb300 import build

WARPS = 8
PAIR = r"""
#include <cstdio>
constexpr int kSoftmaxWarps = %d, kRing = 8, kValid = 2, kSegs = 2, kSegReaders = 11;
struct C {
%s
};
int main() {
  for (int cta = 0; cta < 2; ++cta)
    for (int h = 0; h < 2; ++h) {
      std::printf("%%d", C::arrivals(C::kProb + h, cta));
      for (int w = 0; w < kSoftmaxWarps; ++w) std::printf(" %%d", C::counts_on(h, cta, w) ? 1 : 0);
      std::printf("\n");
    }
}
"""


def source(name):
    return open(os.path.join(build.CSRC, name)).read()


def function(text, name):
    found = re.search(r"  (?:__device__ )?static constexpr \w+ " + name + r"\(.*?\) \{(?: [^\n]*\}\n|\n.*?\n  \}\n)", text, flags=re.S)
    assert found, f"no {name} in the source"
    return found.group(0).replace("__device__ ", "")


def run(program, tmp_path):
    src, exe = tmp_path / "counts.cpp", tmp_path / "counts"
    src.write_text(program)
    subprocess.run([build._nvcc(), "-std=c++17", "-cudart", "none", str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True).stdout


def test_every_warp_of_a_pair_has_rescaled_before_the_first_product(tmp_path):
    """O of both CTAs is rescaled by eight warps each, and the product with the leader's
    keys (h = 0) adds to all of it.  Whatever warps are late, that product's barriers are
    complete only when every one of both CTAs has arrived; the second product (h = 1)
    comes after the first, and no barrier counts more or fewer arrivals than it gets."""
    text = source("fattn_latent_pair.cu")
    bars = re.search(r"  enum : int \{.*?\};\n", text, flags=re.S).group(0)
    out = run(PAIR % (WARPS, bars + function(text, "counts_on") + function(text, "arrivals")), tmp_path)
    rows = [[int(x) for x in line.split()] for line in out.splitlines()]
    count = {(cta, h): rows[2 * cta + h] for cta, h in itertools.product(range(2), range(2))}
    for (cta, h), (n, *on) in count.items():
        assert n == sum(on), (cta, h)
        for there in itertools.product((0, 1), repeat=WARPS):       # the warps that have arrived
            if h == 0 and sum(a and b for a, b in zip(there, on)) >= n:
                assert all(there), (cta, there)


def test_a_pairs_barrier_is_armed_only_when_its_last_phase_is_over():
    """Warp 0 of the leader arms the barrier of what the other CTA stores of P once a tile. An
    arrival beyond a phase's count is undefined, so it looks first whether the last tile's
    stores are all there (nothing else that it has waited for by then says so)."""
    text = source("fattn_latent_pair.cu")
    arm = text.index("mbar_arrive_expect_tx(bar(C::kProb + peer)")
    wait = re.search(r"if \(leader && tiles > 0 && "
                     r"!\(ok = wait_warp\(bar\(C::kProb \+ peer\), \(tiles - 1\) & 1, wc, \w+\)\)\)\s*break;", text)
    assert wait and wait.end() < arm
