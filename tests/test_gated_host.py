"""The host-only argument checks of the gated products, and which kernel takes them.  CPU only
(addresses are never dereferenced)."""
import itertools
import os
import re

import pytest

import mixed_precision_dense_amd as mp
from tests import gated_plans
from tests.test_ops_host import BAD, BIG, NOT, OK, P, checker

CSRC = os.path.join(gated_plans.ROOT, "mixed_precision_dense_amd", "csrc")


def gated(**kw):
    return mp.Gated(**kw)


def grad(**kw):
    return mp.GatedGrad(**{**dict(act="silu", kept=P, ld_kept=128, stride_kept=64), **kw})


GATED = dict(transb=True, m=100, n=64, k=72, alpha=1.0, A=P, a_type="bf16", lda=72, B=P, b_type="bf16", ldb=72, stride_up=64 * 72,
             gated=gated(), D=P, d_type="bf16", ldd=64)
GRAD = dict(transb=True, m=100, n=64, k=72, alpha=1.0, A=P, a_type="bf16", lda=72, B=P, b_type="bf16", ldb=72, grad=grad(), D=P,
            d_type="f32", ldd=128, stride_d=64, workspace=P, workspace_bytes=1 << 20)
GROUPED = dict(transb=True, groups=4, rows=100, n=64, k=72, alpha=1.0, A=P, a_type="f16", lda=72, offsets=P, B=P, b_type="f16", ldb=72,
               stride_b=128 * 72, stride_up=64 * 72, gated=gated(), D=P, d_type="f16", ldd=64)
GROUPED_GRAD = dict(transb=True, groups=4, rows=100, n=64, k=72, alpha=1.0, A=P, a_type="f16", lda=72, offsets=P, B=P, b_type="f16",
                    ldb=72, stride_b=64 * 72, grad=grad(), D=P, d_type="f16", ldd=128, stride_d=64, workspace=P,
                    workspace_bytes=1 << 20)
g1 = checker(mp.mpgemm_check_gated, GATED)
g1_grad = checker(mp.mpgemm_check_gated_grad, GRAD)
ge = checker(mp.mpgemm_check_grouped_gated, GROUPED)
ge_grad = checker(mp.mpgemm_check_grouped_gated_grad, GROUPED_GRAD)
ALL, FORWARD, BACKWARD = [g1, g1_grad, ge, ge_grad], [g1, ge], [g1_grad, ge_grad]


@pytest.mark.parametrize("check", ALL)
def test_types(check):
    assert check() == OK
    for t in ("f16", "bf16"):
        assert check(a_type=t, b_type=t, d_type=t) == OK and check(a_type=t, b_type=t, d_type="f32") == OK
    assert check(a_type="f16", b_type="bf16", d_type="f32") == NOT
    assert check(a_type="bf16", b_type="bf16", d_type="f16") == NOT
    for t in ("f32", "i8", "e4m3", 9, -1):
        assert check(a_type=t, b_type=t, d_type="f32") == NOT


@pytest.mark.parametrize("check", ALL)
def test_sizes_and_nulls(check):
    rows = "rows" if "rows" in check.names else "m"
    for name in {"m", "n", "k", "groups", "rows", "stride_b"} & check.names:
        assert check(**{name: -8}) == BAD, name
    for name in {"A", "B", "D", "offsets"} & check.names:
        assert check(**{name: None}) == BAD, name
    for name in ("lda", "ldb", "ldd"):
        assert check(**{name: 63}) == BAD, name
    for name in (rows, "n", "k"):
        assert check(**{name: BIG, "lda": 1 << 22, "ldb": 1 << 22, "ldd": 1 << 22}) in (BAD, NOT), name
    assert check(k=0, A=None, B=None) == OK
    if "groups" in check.names:
        assert check(groups=65536) == NOT and check(groups=65535, workspace_bytes=1 << 40) == OK if "workspace" in check.names \
            else check(groups=65536) == NOT
        assert check(groups=0, A=None, B=None, D=None, offsets=None) == OK
    for name in {"A", "B", "D"}:
        assert check(**{name: P + 8}) == NOT, name
    assert check(lda=76) == NOT and check(ldb=76) == NOT


@pytest.mark.parametrize("check", FORWARD)
def test_forward_refusals(check):
    rows = "rows" if "rows" in check.names else "m"
    assert check(gated=None) == BAD
    for act in (-1, 5):
        assert check(gated=gated(act=act)) == BAD
    t = "bf16" if check is g1 else "f16"
    other = "f16" if check is g1 else "bf16"
    for side in ("bias_gate", "bias_up"):
        assert check(gated=gated(**{side: P, "bias_type": t})) == OK and check(gated=gated(**{side: P})) == OK
        assert check(gated=gated(**{side: P, "bias_type": other})) == NOT
        assert check(gated=gated(**{side: P + 2})) == NOT and check(gated=gated(**{side: P + 2, "bias_type": t})) == OK
    if check is ge:
        assert check(gated=gated(bias_up=P, bias_stride=-1)) == BAD
    # the pair of weights
    assert check(stride_up=-8) == BAD and check(stride_up=4) == NOT and check(stride_up=0) == OK
    assert check(transb=False, ldb=128, stride_up=64) == OK
    assert check(stride_up=(1 << 30) - (1 << 17)) == OK and check(stride_up=1 << 30) == NOT
    assert check(ldb=1 << 21, stride_up=1 << 29) == NOT and check(ldb=1 << 20, stride_up=1 << 29) == OK
    # the pair that is kept
    kept = dict(kept=P, ld_kept=128, stride_kept=64)
    assert check(gated=gated(**kept)) == OK
    assert check(gated=gated(**{**kept, "kept": P + 8})) == NOT
    assert check(gated=gated(**{**kept, "ld_kept": 63})) == BAD and check(gated=gated(**{**kept, "ld_kept": 132})) == NOT
    assert check(gated=gated(**{**kept, "stride_kept": 68})) == NOT
    for stride in (-64, 0, 56, 72, 128 * 98 + 64):
        assert check(gated=gated(**{**kept, "stride_kept": stride})) == BAD, stride
    assert check(gated=gated(**{**kept, "stride_kept": 128 * 99 + 64})) == OK
    assert check(gated=gated(kept=P, ld_kept=64, stride_kept=64)) == BAD
    assert check(**{rows: 1}, gated=gated(kept=P, ld_kept=64, stride_kept=64)) == OK
    assert check(**{rows: 0}, A=None, B=None, D=None) == OK and check(n=0, A=None, B=None, D=None) == OK


@pytest.mark.parametrize("check", BACKWARD)
def test_backward_refusals(check):
    rows = "rows" if "rows" in check.names else "m"
    groups = 4 if check is ge_grad else 1
    assert check(grad=None) == BAD
    for act in (-1, 5):
        assert check(grad=grad(act=act)) == BAD
    assert check(grad=grad(kept=None)) == BAD and check(grad=grad(kept=P + 8)) == NOT
    assert check(grad=grad(ld_kept=63)) == BAD and check(grad=grad(ld_kept=132)) == NOT
    assert check(grad=grad(stride_kept=-64)) == BAD and check(grad=grad(stride_kept=4)) == NOT
    assert check(grad=grad(stride_kept=0)) == OK                          # (read only: both may be the same)
    assert check(grad=grad(H=P, ldh=64)) == OK and check(grad=grad(H=P, ldh=63)) == BAD
    assert check(grad=grad(H=P + 8, ldh=64)) == NOT and check(grad=grad(H=P, ldh=68)) == NOT
    for stride in (-64, 0, 56, 72):
        assert check(stride_d=stride) in (BAD, NOT), stride
    assert check(stride_d=128 * 99 + 64) == OK
    need = mp.mpgemm_gated_grad_workspace_size(groups, 100, 64)
    assert need > 0 and need == 2 * mp.mpgemm_epilogue_grad_workspace_size(groups, 100, 64)
    assert check(workspace=None, workspace_bytes=0) == OK                 # no dbias: none is needed
    assert check(grad=grad(dbias=P), workspace_bytes=need) == OK and check(grad=grad(dbias=P), workspace_bytes=need - 1) == BAD
    assert check(grad=grad(dbias=P), workspace=None) == BAD and check(grad=grad(dbias=P), workspace=P + 16) == NOT
    assert check(grad=grad(dbias=P + 2)) == NOT
    none = dict(A=None, B=None, D=None)
    assert check(**{rows: 0}, grad=grad(dbias=P, kept=None), **none) == OK
    assert check(**{rows: 0}, grad=grad(dbias=P + 2, kept=None), **none) == NOT
    assert check(n=0, grad=grad(kept=None), **none) == OK
    assert mp.mpgemm_gated_grad_workspace_size(0, 5, 5) == 0 and mp.mpgemm_gated_grad_workspace_size(1, BIG, 5) == 0


SIZES = [1, 5, 15, 16, 17, 31, 33, 64, 65, 100, 500, 1000, 4000, 8000, 10000, 24000, 100000, 1000000]
KS = [1, 64, 200, 1000, 4000]


def instances(files, pattern):
    found = []
    for f in files:
        with open(os.path.join(CSRC, f)) as src:
            found += re.findall(r"template __global__ void " + pattern, src.read())
    assert len(found) == len(set(found))
    return set(found)


@pytest.mark.skipif(not gated_plans.available(), reason="g++ builds the rules")
def test_every_kernel_that_is_built_can_be_chosen_and_no_other():
    few, tiles, grads = set(), set(), set()
    for m, n, k in itertools.product(SIZES, SIZES, KS):
        for groups in (0, 1, 2, 7, 32, 300):
            for tb in (False, True):
                kernel = gated_plans.gated(groups, m, n, k, tb)
                (few if kernel[0] == "few" else tiles).add(("true" if tb else "false", *map(str, kernel[1:])))
            grads.add(gated_plans.gated_grad(groups, m, n, k))
    both = ("true", "false")
    for t in ("F16", "BF16"):
        assert instances(["skinny_gated.hip"], rf"gated_skinny_kernel<IN_{t}, (\w+), (\d), (\d), (\d)>") == few
        assert instances([f"ops_gated_{t.lower()}.hip"], rf"op_kernel<IN_{t}, OP_GATED, false, (\w+), (\d+)>") == tiles
        assert instances([f"ops_gated_grad_{t.lower()}.hip"], rf"op_kernel<IN_{t}, OP_GATED_GRAD, false, (\w+), (\d+)>") == set(
            itertools.product(both, ("64", "128", "256")))
    assert grads == {("tile", e) for e in (64, 128, 256)}
