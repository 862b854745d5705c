"""Which kernel a grouped product takes on devices other than this one: plan
queries against contexts made up on the host."""
import os
import subprocess

import pytest

import rank_sum_residual_gb300 as farn
from rank_sum_residual_gb300 import _build

TENSOR, PAIR = 6, 7


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(clusters of 1, 2 and 4, slots, E, N, H) -> (variant, CTAs per tile)"""
    lib = farn.build_library()
    exe = str(tmp_path_factory.mktemp("plan") / "plan_probe")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["nvcc", "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-o", exe,
                    os.path.join(here, "plan_probe.cu"), lib, "-Xlinker",
                    "-rpath=" + os.path.dirname(lib)], check=True)

    def query(clusters, S, E, N, H, split=0):
        args = [152, *clusters, split, S, E, N, H]
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        status, variant, ctas = map(int, out.stdout.split())
        assert status == farn.FARN_OK
        return variant, ctas
    return query


# calls that split their rows by four where clusters of four fit
SPLIT = [(2, 2, 1024, 2048), (1, 1, 1200, 5000), (20, 3, 512, 4096)]


@pytest.mark.parametrize("S,E,N,H", SPLIT)
def test_rows_are_split_over_clusters_that_fit(plan, S, E, N, H):
    """A device that has no room for a cluster of four CTAs (of two) splits a
    row by two (not at all): such calls stay on the tensor cores."""
    assert plan((152, 76, 36), S, E, N, H) == (TENSOR, 4)
    assert plan((152, 76, 0), S, E, N, H) == (TENSOR, 2)
    assert plan((152, 0, 0), S, E, N, H) == (TENSOR, 1)
    assert plan((152, 76, 0), S, E, N, H, split=4) == (TENSOR, 2)


def test_long_calls_without_pairs(plan):
    assert plan((152, 76, 36), 32768, 64, 4096, 7168) == (PAIR, 2)
    assert plan((152, 0, 0), 32768, 64, 4096, 7168) == (TENSOR, 1)
