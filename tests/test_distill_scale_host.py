"""Which scales of a teacher's logits are taken.  CPU only (addresses are never dereferenced)."""
import pytest

from tests.test_distill_host import forward, grad, teacher
from tests.test_ops_host import BAD, OK


@pytest.mark.parametrize("check", [forward, grad])
def test_scales(check):
    for scale in (float("nan"), float("inf"), float("-inf"), 2e30, -2e30):
        assert check(teacher=teacher(scale=scale)) == BAD, scale
    for scale in (1e30, -1e30, 1.0, 0.0, -0.0, -2.5, 1e-30):
        assert check(teacher=teacher(scale=scale)) == OK, scale


def test_scales_of_empty_calls():
    none = dict(X=None, W=None, lse=None, picked=None, workspace=None)
    for scale, status in ((float("nan"), BAD), (0.0, OK)):
        t = teacher(index=None, logit=None, scale=scale)
        assert forward(m=0, loss=None, teacher=t, **none) == status and grad(m=0, grad=None, teacher=t, **none) == status
