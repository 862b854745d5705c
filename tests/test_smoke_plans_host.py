"""The smoke run's products reach the kernels that it says it runs."""
import pytest

import __graft_entry__ as entry
import rank_sum_residual_gb300 as farn
from test_fp8_workspace_host import PAIR, TENSOR, probe  # noqa: F401


@pytest.mark.parametrize("name,sizes", [("nvfp4", entry.NVFP4_PRODUCTS),
                                        ("fp8", entry.FP8_PRODUCTS),
                                        ("experts", entry.FP8_EXPERTS)])
def test_a_short_call_and_one_for_pairs(probe, name, sizes):  # noqa: F811
    plans = [probe(name, *s) for s in sizes]
    assert [p[0] for p in plans] == [farn.FARN_OK] * 2
    assert [p[1] for p in plans] == [TENSOR, PAIR]
    if name == "experts":                       # and the copy of the rows in front of it
        assert plans[0][3] == 0 and plans[1][3] > 0
