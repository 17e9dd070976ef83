"""Which kernel takes a product of language models: that the tests of the tiles reach the tiles they are
for, and that every kernel that the rules can choose is built, and no other."""
import itertools
import os
import re

import pytest

from tests import ops_plans, ops_tile_cases as cases

pytestmark = pytest.mark.skipif(not ops_plans.available(), reason="g++ builds the rules")
CSRC = os.path.join(ops_plans.ROOT, "mixed_precision_dense_amd", "csrc")


@pytest.mark.parametrize("c", cases.FORWARD)
def test_forward_cases(c):
    assert ops_plans.forward(c["m"], c["n"], c["k"], c["tb"], c["act"], c["aux"], bool(c["beta"])) == c["kernel"]


@pytest.mark.parametrize("c", cases.SLOPE)
def test_slope_cases(c):
    assert ops_plans.slope(c["m"], c["n"], c["k"], c["tb"], c["act"]) == c["kernel"]


@pytest.mark.parametrize("c", cases.GROUPED)
def test_grouped_cases(c):
    assert ops_plans.grouped(c["rows"], c["groups"], c["n"], c["k"], c["tb"], c["act"], c["aux"]) == c["kernel"]


@pytest.mark.parametrize("c", cases.GROUPED_GRAD)
def test_grouped_grad_cases(c):
    assert ops_plans.grouped_grad(c["rows"], c["groups"], c["n"], c["k"], c["tb"], c["act"]) == c["kernel"]


@pytest.mark.parametrize("c", cases.WGRAD)
def test_wgrad_cases(c):
    assert ops_plans.wgrad(c["groups"], c["rows"], c["m"], c["n"]) == c["kernel"]


@pytest.mark.parametrize("c", cases.CE + cases.PIECES)
def test_cross_entropy_cases(c):
    got = ops_plans.cross_entropy(c["m"], c["n"], c["k"], c["train"])
    assert {name: got[name] for name in c["kernels"]} == c["kernels"]
    if c["train"]:   # the loss before the gradient takes its own plan
        assert ops_plans.cross_entropy(c["m"], c["n"], c["k"], False)["logits"][0] == "tile"


def test_every_edge_is_reached_by_every_kind():
    edges = {64, 128, 256}
    for kind in (cases.FORWARD, cases.SLOPE, cases.GROUPED):
        assert {c["kernel"][1] for c in kind} == edges
    for kind in (cases.GROUPED_GRAD, cases.WGRAD):
        assert {c["kernel"][1] for c in kind} >= {128, 256}
    assert {c["kernels"][p][1] for c in cases.CE for p in ("logits", "dw", "dx") if p in c["kernels"]} >= {128, 256}
