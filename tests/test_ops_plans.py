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


@pytest.mark.parametrize("c", cases.FEW)
def test_few_rows_cases(c):
    assert ops_plans.forward(c["m"], c["n"], c["k"], c["tb"], "gelu", True, True) == c["kernel"]
    assert ops_plans.slope(c["m"], c["n"], c["k"], c["tb"], "silu") == c["kernel"]


@pytest.mark.parametrize("c", cases.FEW_OF_EXPERTS)
def test_few_rows_of_experts_cases(c):
    assert ops_plans.grouped(c["m"], c["groups"], c["n"], c["k"], c["tb"], "silu", True) == c["kernel"]
    assert ops_plans.grouped_grad(c["m"], c["groups"], c["n"], c["k"], c["tb"], "silu") == c["kernel"]


@pytest.mark.parametrize("t", ["F16", "BF16"])
def test_every_few_rows_kernel_has_a_case(t):
    cased = {(word(ta), word(c["tb"]), *map(str, c["kernel"][1:])) for c in cases.FEW for ta in (False, True)}
    cased |= {("false", word(c["tb"]), *map(str, c["kernel"][1:])) for c in cases.FEW_OF_EXPERTS}
    assert cased == instances([f"skinny_{t.lower()}.hip"], rf"skinny_kernel<IN_{t}, (\w+), (\w+), (\d), (\d), (\d)>")


def test_every_edge_is_reached_by_every_kind():
    edges = {64, 128, 256}
    for kind in (cases.FORWARD, cases.SLOPE, cases.GROUPED):
        assert {c["kernel"][1] for c in kind} == edges
    for kind in (cases.GROUPED_GRAD, cases.WGRAD):
        assert {c["kernel"][1] for c in kind} >= {128, 256}
    assert {c["kernels"][p][1] for c in cases.CE for p in ("logits", "dw", "dx") if p in c["kernels"]} >= {128, 256}


def instances(files, pattern):
    """Arguments of the kernel instances that the sources name."""
    found = []
    for f in files:
        with open(os.path.join(CSRC, f)) as src:
            found += re.findall(r"template __global__ void " + pattern, src.read())
    assert len(found) == len(set(found))
    return set(found)


def word(v):
    return "true" if v else "false"


SIZES = [1, 5, 15, 16, 17, 31, 33, 64, 65, 100, 500, 1000, 4000, 10000, 24000, 24600, 30000, 100000, 1000000]
KS = [1, 64, 200, 1000, 4000, 10000]


@pytest.mark.parametrize("t", ["F16", "BF16"])
def test_the_few_rows_kernels_that_are_built_are_those_that_are_chosen(t):
    chosen = set()
    for m, n, k, tb in itertools.product(SIZES, SIZES, KS, (False, True)):
        for ta in (False, True):
            for act in ("none", "gelu"):
                for kernel in (ops_plans.forward(m, n, k, tb, act, True, True), ops_plans.slope(m, n, k, tb, act)):
                    if kernel[0] == "few":
                        chosen.add((word(ta), word(tb), *map(str, kernel[1:])))
        for groups in (1, 2, 7, 32, 300):
            for kernel in (ops_plans.grouped(m, groups, n, k, tb), ops_plans.grouped_grad(m, groups, n, k, tb, "gelu")):
                if kernel[0] == "few":
                    chosen.add(("false", word(tb), *map(str, kernel[1:])))
    built = instances([f"skinny_{t.lower()}.hip"], rf"skinny_kernel<IN_{t}, (\w+), (\w+), (\d), (\d), (\d)>")
    assert chosen == built, (chosen - built, built - chosen)


@pytest.mark.parametrize("t", ["F16", "BF16"])
@pytest.mark.parametrize("mode,file", [("FORWARD", "ops_forward"), ("SLOPE", "ops_slope")])
def test_every_tile_is_built(t, mode, file):
    both = ("true", "false")
    assert instances([f"{file}_{t.lower()}.hip"], rf"op_kernel<IN_{t}, OP_{mode}, (\w+), (\w+), (\d+)>") == set(
        itertools.product(both, both, ("64", "128", "256")))


def test_the_cross_entropy_tiles_that_are_built_are_those_that_are_chosen():
    stats, probs = set(), set()
    for m, n, k in itertools.product(SIZES, SIZES, KS):
        for train, found in ((False, stats), (True, probs)):
            kernel = ops_plans.cross_entropy(m, n, k, train)["logits"]
            if kernel[0] == "tile":
                found.add(str(kernel[1]))
    for mode, found in (("STATS", stats), ("PROBS", probs)):
        for t in ("F16", "BF16"):
            assert instances(["ops_ce.hip"], rf"op_kernel<IN_{t}, OP_CE_{mode}, false, true, (\d+)>") == found == {"64", "128", "256"}
