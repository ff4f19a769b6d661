"""How the roles of the latent attention's kernels wait for one another, on the CPU:
the counts of their barriers are taken from the sources and checked against every
order in which the warps that arrive may be."""

import itertools
import os
import random
import re
import subprocess

import pytest

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


SINGLE = r"""
#include <cstdio>
struct C {
  static constexpr int kRing = %d, kRopes = %d, kSegs = %d, kSoftmax = 128, kSegReaders = 6;
%s
};
int main() {
  for (int two = 0; two < 2; ++two)
    std::printf("%%d %%d %%d\n", C::arrivals(0, two), C::arrivals(2 * C::kRing, two),
                C::arrivals(2 * (C::kRing + C::kRopes) + 7 + C::kSegs, two));
}
"""
SEGS = 4


class Bar:
    """A barrier as a wait by parity sees it."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        assert self.left > 0, "an arrival beyond the phase's count"
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return self.phase & 1 != parity


def simulate(tiles, ring, counts, late):
    """Sequences of one tile each, tiles[i]: whether tile i has a second page; a ring of slots, two
    warps that load and one that uses the tiles.  late(turn): the second one's turn is
    left out.  Returns the tiles used without their second page, or None if all wait."""
    full_count, seg_count = counts
    full, empty = [Bar(full_count) for _ in range(ring)], [Bar(1) for _ in range(ring)]
    published, seg_empty = [0], [Bar(seg_count) for _ in range(SEGS)]
    second, wrong, used = [False] * len(tiles), [], [0]

    def walk():
        for i in range(len(tiles)):
            while i >= SEGS and not seg_empty[i % SEGS].done((i // SEGS - 1) & 1):
                yield
            published[0] = i + 1

    def load(which):
        for i in range(len(tiles)):
            while published[0] <= i:
                yield
            seg_empty[i % SEGS].arrive()
            while i >= ring and not empty[i % ring].done((i // ring - 1) & 1):
                yield
            if which == 1:
                second[i] = True
            if which == 0 or full_count == 2:
                full[i % ring].arrive()
            yield

    def use():
        for i in range(len(tiles)):
            # with one arrival the copy's bytes hold the phase up where there is a second page
            while not full[i % ring].done((i // ring) & 1) or (full_count == 1 and tiles[i] and not second[i]):
                yield
            if tiles[i] and not second[i]:
                wrong.append(i)
            empty[i % ring].arrive()
            used[0] = i + 1
            yield

    def others():                       # the segments' other readers
        for i in range(len(tiles)):
            while used[0] <= i:
                yield
            for _ in range(seg_count - 2):
                seg_empty[i % SEGS].arrive()

    roles = [walk(), load(0), use(), others(), load(1)]
    alive = [True] * 5
    for turn in range(2000):
        for k, r in enumerate(roles):
            if alive[k] and not (k == 4 and late(turn)):
                try:
                    next(r)
                except StopIteration:
                    alive[k] = False
    return wrong if not any(alive) else None


@pytest.mark.parametrize("ring", [2, 3, 6])
def test_neither_warp_that_loads_falls_a_turn_of_the_ring_behind(ring, tmp_path):
    """Sequences of 1 to 32 tokens have no second page, so nothing but the barriers' counts holds
    the first warp back.  However late the second one is, every tile is used, with its pages."""
    text = source("fattn_latent_attn.cu")
    out = run(SINGLE % (8, ring, SEGS, function(text, "arrivals")), tmp_path)
    (pair1, rope1, seg1), (pair2, rope2, seg2) = [[int(x) for x in line.split()] for line in out.splitlines()]
    assert (pair1, rope1) == (1, 1) and seg2 == seg1 + 1 and pair2 == rope2
    r = random.Random(ring)
    for n in range(60):
        tiles = [i % 9 == 8 if n % 3 == 0 else r.random() < 0.2 for i in range(40)]
        k = n % 20 + 1
        for late in (lambda turn: turn % k != 0, lambda turn: turn < 5 * k, lambda turn: r.random() < 1 - 1 / k):
            assert simulate(tiles, ring, (pair2, seg2), late) == []


def test_the_simulation_tells_a_warp_that_is_left_behind():
    """With one arrival a tile, of the first warp, the second one misses a phase."""
    tiles = [i % 9 == 8 for i in range(40)]
    assert simulate(tiles, 2, (1, 7), lambda turn: turn < 50) is None
