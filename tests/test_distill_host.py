"""The host-only argument checks of the distillation loss.  CPU only (addresses are never dereferenced)."""
import pytest

import mixed_precision_dense_amd as mp
from tests.test_ops_host import BAD, BIG, NOT, OK, P, checker


def teacher(**kw):
    return mp.Teacher(**{**dict(top=20, index=P, logit=P, ld=20, scale=0.5), **kw})


FORWARD = dict(m=100, n=500, k=72, alpha=1.0, X=P, dtype="bf16", ldx=72, W=P, ldw=72, teacher=teacher(), loss=P, lse=P, picked=P,
               workspace=P, workspace_bytes=1 << 24)
GRAD = dict(m=100, n=500, k=72, alpha=1.0, X=P, dtype="bf16", ldx=72, W=P, ldw=72, teacher=teacher(), lse=P, picked=P, grad=P, dX=P,
            lddx=72, dW=P, lddw=72, workspace=P, workspace_bytes=1 << 24)
forward = checker(mp.mpgemm_check_linear_distill, FORWARD)
grad = checker(mp.mpgemm_check_linear_distill_grad, GRAD)


@pytest.mark.parametrize("check", [forward, grad])
def test_refusals(check):
    assert check() == OK and check(dtype="f16") == OK
    assert check(dtype="f32") == NOT and check(dtype=17) == NOT
    for name in ("m", "k"):
        assert check(**{name: -1}) == BAD
    assert check(n=0) == BAD and check(m=BIG, workspace_bytes=1 << 62) == NOT and check(n=BIG, workspace_bytes=1 << 62) == NOT
    assert check(ldx=71) == BAD and check(ldw=71) == BAD and check(ldx=76) == NOT and check(ldw=76) == NOT
    for name in {"X", "W", "loss", "lse", "picked", "grad", "workspace"} & check.names:
        assert check(**{name: None}) == BAD, name
    for name, off in (("X", 8), ("W", 8), ("lse", 2), ("loss", 2), ("picked", 2), ("grad", 2), ("dX", 8), ("dW", 8), ("workspace", 64)):
        if name in check.names:
            assert check(**{name: P + off}) == NOT, name
    # the teacher
    assert check(teacher=None) == BAD and check(teacher=teacher(top=0)) == BAD and check(teacher=teacher(top=-1)) == BAD
    assert check(teacher=teacher(ld=19)) == BAD and check(teacher=teacher(ld=21)) == OK
    assert check(teacher=teacher(top=1024, ld=1024)) == OK and check(teacher=teacher(top=1025, ld=1025)) == NOT
    assert check(teacher=teacher(ld=BIG)) == NOT
    assert check(teacher=teacher(index=None)) == BAD and check(teacher=teacher(logit=None)) == BAD
    assert check(teacher=teacher(index=P + 4)) == NOT and check(teacher=teacher(logit=P + 2)) == NOT
    assert check(teacher=teacher(lse=P)) == OK and check(teacher=teacher(lse=P + 2)) == NOT


def test_empty_calls():
    none = dict(X=None, W=None, lse=None, picked=None, workspace=None, teacher=teacher(index=None, logit=None))
    assert forward(m=0, loss=None, **none) == OK
    assert grad(m=0, grad=None, **none) == OK and grad(dX=None, dW=None, grad=None, **none) == OK
    assert grad(dX=None) == OK and grad(dW=None) == OK
    assert grad(k=0, X=None, W=None) == OK and forward(k=0, X=None, W=None) == OK


def test_workspaces():
    for train in (False, True):
        need = mp.mpgemm_linear_distill_workspace_size(100, 500, 72, 20, "bf16", train)
        assert need >= mp.mpgemm_linear_ce_workspace_size(100, 500, 72, "bf16", train) > 0
        check = grad if train else forward
        assert check(workspace_bytes=need) == OK and check(workspace_bytes=need - 1) == BAD
    size = mp.mpgemm_linear_distill_workspace_size
    assert size(0, 500, 72, 20, "bf16", True) == 0 and size(100, 0, 72, 20, "bf16", True) == 0
    assert size(100, 500, 72, 0, "bf16", True) == 0 and size(100, 500, 72, 1025, "bf16", True) == 0
    assert size(100, 500, 72, 20, "f32", True) == 0
    assert forward(workspace_bytes=size(100, 500, 72, 20, "bf16", True)) == OK   # the gradient's is enough for both
