"""The FP8 products' plan, compiled for the host: the kernel, tile and split that each case of the
products' tests takes, so that a new fit of the plan cannot leave one of them without a test."""
import shutil
import subprocess

import pytest

from fp8_tile_cases import CASES, TILES
from tenant_serving_amd import build

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")

MAIN = """
#include <cstdio>
#include <cstdlib>
#include "bd_fp8_plan.h"
int main(int argc, char** argv) {  // split_ok T d_in rows...
    int64_t d[4];
    for (int i = 4; i < argc; ++i) d[i - 4] = atoll(argv[i]);
    const bd::Fp8Plan p = bd::plan_fp8(atoll(argv[2]), atoll(argv[3]), d, argc - 4, atoi(argv[1]));
    printf("%d %d %lld", p.tile, p.S, (long long)p.kps);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def f(T, d_outs, d_in, split=True):
        r = subprocess.run([str(d / "plan"), str(int(split)), str(T), str(d_in)] + [str(n) for n in d_outs],
                           check=True, capture_output=True, text=True)
        tile, S, kps = map(int, r.stdout.split())
        return TILES[tile], S, kps
    return f


@pytest.mark.parametrize("tile,S,T,d_outs,d_in", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_cases_take_the_tile_they_name(plan, tile, S, T, d_outs, d_in):
    got, parts, kps = plan(T, d_outs, d_in)
    assert (got, parts) == (tile, S)
    assert parts == 1 or (kps % 512 == 0 and (parts - 1) * kps < d_in <= parts * kps)


def test_cases_cover_the_plan():
    assert {t for t, S, *_ in CASES if S == 1} == set(TILES)
    assert {t for t, S, *_ in CASES if S > 1} == set(TILES) - {"rows", "64x128"}
    odd = {(t, S > 1, T * n % 4) for t, S, T, d_outs, _ in CASES for n in d_outs}
    for t in set(TILES) - {"rows", "64x128"}:  # values that a sum of parts takes one by one
        assert any((t, True, r) in odd for r in (1, 2, 3))


def test_no_split_without_a_workspace(plan):
    for _, _, T, d_outs, d_in in CASES:
        assert plan(T, d_outs, d_in, split=False)[1] == 1
