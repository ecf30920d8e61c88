"""Which clusters the grouped products are launched in, by what the occupancy query answers (CPU: the rule is plain C++,
compiled here with the host compiler)."""
import os
import shutil
import subprocess

import pytest

import mixture_experts_layer_10_gb300 as moe

SOURCE = r"""
#include <cstdio>
#include "clusters.cuh"
int main() {
  int ok, n4, n2, sms;
  long long tiles;
  while (std::scanf("%d %d %d %d %lld", &ok, &n4, &n2, &sms, &tiles) == 5) {
    const int four = moe::clusters_that_fit(ok, n4, sms, 8), two = moe::clusters_that_fit(ok, n2, sms, 4);
    const int pairs = moe::pairs_per_tile(tiles, [&](int p) { return p == 4 ? four : two; });
    std::printf("%d %d %d %d\n", four, two, moe::clusters_that_fit(ok, 0, sms, 2), pairs);
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("clusters")
    (d / "main.cc").write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(moe.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(d / "main.cc"), "-o", str(d / "main")], check=True)

    def answer(*args):
        r = subprocess.run([str(d / "main")], input=" ".join(map(str, args)), capture_output=True, text=True, check=True)
        return tuple(map(int, r.stdout.split()))
    return answer


# the query's answers for clusters of eight and of four CTAs, SMs, tiles -> clusters of eight, of four, pairs at once, pairs a tile
@pytest.mark.parametrize("ok,n8,n4,sms,tiles,want", [
    (1, 16, 36, 152, 16, (16, 36, 76, 4)), (1, 16, 36, 152, 17, (16, 36, 76, 2)), (1, 16, 36, 152, 37, (16, 36, 76, 1)),
    (1, 100, 100, 152, 1, (19, 38, 76, 4)),                                       # more than the SMs hold
    (1, 0, 36, 152, 1, (-1, 36, 76, 2)), (1, 0, 0, 152, 1, (-1, -1, 76, 1)),      # none of them fits
    (0, 0, 0, 152, 1, (-1, -1, 76, 1)), (0, 7, 7, 152, 1, (-1, -1, 76, 1)),       # no answer
    (1, 1, 1, 6, 1, (-1, 1, 3, 2)),                                               # part of a device
])
def test_split_of_few_tiles(ask, ok, n8, n4, sms, tiles, want):
    assert ask(ok, n8, n4, sms, tiles) == want
