"""The sizes of tests/gated_cases.py reach every kernel of the gated product that is built.  CPU only."""
import pytest

from tests import gated_cases, gated_plans
from tests.test_gated_host import instances


@pytest.mark.skipif(not gated_plans.available(), reason="g++ builds the rules")
@pytest.mark.parametrize("t", ["F16", "BF16"])
def test_every_kernel_has_a_size(t):
    few, tiles = set(), set()
    for groups, m, n, k in gated_cases.SIZES:
        for tb in (False, True):
            kernel = gated_plans.gated(groups, m, n, k, tb, "silu", True)
            (few if kernel[0] == "few" else tiles).add(("true" if tb else "false", *map(str, kernel[1:])))
    assert instances(["skinny_gated.hip"], rf"gated_skinny_kernel<IN_{t}, (\w+), (\d), (\d), (\d)>") == few
    assert instances([f"ops_gated_{t.lower()}.hip"], rf"op_kernel<IN_{t}, OP_GATED, false, (\w+), (\d+)>") == tiles


def test_shares():
    for groups, m, _, _ in gated_cases.SIZES:
        s = gated_cases.shares(groups, m)
        assert s is None if not groups else len(s) == groups and sum(s) <= m and 0 in s and sum(s) > m // 2
