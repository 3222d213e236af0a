"""The rule by which a cluster's CTAs join their sums, compiled for the host."""
import subprocess

import pytest

from paged_kv_cache_bsr_gb300 import build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "pkv_join.h"
// share, the rank that gave up (-1: none) -> whole, total of parts 1.5, 2.5, ...
int main(int, char** argv) {
  const int share = std::atoi(argv[1]), late = std::atoi(argv[2]);
  float total = 77.f;
  const bool whole = pkv::join_ranks(share, [](int k) { return k + 1.5f; }, [&](int k) { return k == late; }, total);
  std::printf("%d %.1f\n", whole ? 1 : 0, total);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("join")
    (at / "join.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(at / "join.cpp"), "-o", str(at / "join")], check=True)
    return str(at / "join")


@pytest.mark.parametrize("share", [1, 2, 4, 8])
def test_a_total_counts_only_where_every_rank_is_done(program, share):
    total = sum(k + 1.5 for k in range(share))
    for late in range(-1, share):
        out = subprocess.run([program, str(share), str(late)], check=True, capture_output=True, text=True).stdout.split()
        assert out[0] == ("1" if late < 0 else "0"), (share, late)
        assert float(out[1]) == total
