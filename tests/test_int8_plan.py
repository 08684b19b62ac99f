"""Which tiles and parts of K the tested sizes of the 8-bit integer product reach (no GPU): csrc/int8_plan.h compiled for the host."""
import os
import subprocess

import pytest

import int8_bits as ref
from test_abi import ROOT
from test_gpu_int8 import SIZES

PROGRAM = r"""
#include <cstdio>
#include "int8_plan.h"
int main() {
  int t, k, n;
  while (scanf("%d %d %d", &t, &k, &n) == 3) {
    if (cl::streamed(t, n, k)) {
      puts("stream 1 0 0 0 0");
      continue;
    }
    const cl::Plan p = cl::plan_product(t, n, k);
    const cl::Shape& s = cl::kShapes[p.shape];
    const long tiles = cl::tiles_of(s, t, n) * p.parts, steps = cl::padded(k) / 128;
    printf("%dx%d %d %ld %ld %ld %d\n", s.tw, s.tt, p.parts, steps, tiles, p.shape == 0 && cl::halved(tiles) ? tiles % cl::kCus : 0L, t % s.tt);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-Wall", "-Werror", "-std=c++17", "-I", os.path.join(ROOT, "compressed_linear_amd", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan")], check=True)

    def of(sizes):
        out = subprocess.run([str(d / "plan")], input="\n".join("%d %d %d" % s for s in sizes), capture_output=True, text=True, check=True)
        return [(line.split()[0],) + tuple(int(v) for v in line.split()[1:]) for line in out.stdout.splitlines()]
    return of


def test_the_sizes_reach_what_they_stand_for(plans):
    for size, (tile, parts, halves), got in zip(ref.PLANS, ref.PLANS.values(), plans(ref.PLANS)):
        name, n, steps, tiles, cut, last = got
        assert (name, n > 1) == (tile, parts), (size, got)
        assert ("none" if cut == 0 else "all" if cut == tiles else "some") == halves, (size, got)
        assert steps // n > 2 * (ref.BUFFERS[tile] + (cut > 0)), (size, got)
        assert last and size[1] % 2 and (cut == 0 or last <= 128), (size, got)


def test_every_tile_is_reached(plans):
    reached = {(got[0], got[1] > 1) for got in plans(ref.PLANS)}
    assert reached == {(tile, parts) for tile in ref.BUFFERS for parts in (False, True)}
    small = {got[0] for got in plans(SIZES)}
    assert "stream" in small and {"64x32", "64x64", "128x64"} <= small


def test_rows_are_computed_by_many_tiles(plans):
    got = [p[:2] for (K, N), tokens in ref.ROWS.items() for p in plans([(T, K, N) for T in tokens])]
    assert {name for name, _ in got} == set(ref.BUFFERS) | {"stream"}
    assert sum(parts > 1 for _, parts in got) >= 3
