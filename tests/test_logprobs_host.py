"""The host-only argument checks of the log probabilities.  CPU only (addresses are never dereferenced)."""
import pytest

import mixed_precision_dense_amd as mp
from tests.test_ops_host import BAD, BIG, NOT, OK, P, checker

LOGPROBS = dict(m=100, n=501, alpha=1.0, Z=P, z_type="bf16", ldz=504, target=P, logprob=P, lse=P, entropy=P, top=20, top_index=P,
                top_logprob=P, ld_top=20, workspace=P, workspace_bytes=1 << 24)
check = checker(mp.mpgemm_check_logprobs, LOGPROBS)


def test_what_is_refused():
    assert check() == OK
    for t, ldz in (("f16", 504), ("f32", 504), ("f32", 508)):
        assert check(z_type=t, ldz=ldz) == OK
    for t in ("i8", "e4m3", "i32", 17):
        assert check(z_type=t) == NOT
    assert check(m=-1) == BAD and check(n=0) == BAD and check(n=-5) == BAD and check(top=-1) == BAD
    for alpha in (0.0, -1.0, float("nan"), float("inf"), 2e30):
        assert check(alpha=alpha) == BAD, alpha
    assert check(alpha=1e30) == OK and check(alpha=1e-30) == OK
    assert check(ldz=500) == BAD and check(ldz=508) == NOT and check(z_type="f32", ldz=506) == NOT
    for name in ("Z", "target", "top_index", "top_logprob"):
        assert check(**{name: None}) == BAD, name
    for name, off in (("Z", 8), ("target", 4), ("logprob", 2), ("lse", 2), ("entropy", 2), ("top_index", 4), ("top_logprob", 2)):
        assert check(**{name: P + off}) == NOT, name
    assert check(ld_top=19) == BAD and check(ld_top=21) == OK and check(top=64, ld_top=64) == OK and check(top=65, ld_top=65) == NOT
    assert check(m=BIG) == NOT and check(n=BIG, ldz=BIG + 1) == NOT and check(ldz=(1 << 31) + 8) == NOT
    assert check(ldz=1 << 31) == OK


def test_what_may_be_missing():
    assert check(logprob=None, target=None) == OK and check(logprob=None, target=P + 4) == OK
    assert check(lse=None, entropy=None) == OK
    assert check(top=0, top_index=None, top_logprob=None, ld_top=0) == OK
    assert check(m=0, Z=None, target=None, logprob=None, top_index=None, top_logprob=None, workspace=None) == OK


@pytest.mark.parametrize("m,n", [(1, 500000), (3, 100000), (100, 128000)])
def test_workspaces(m, n):
    need = mp.mpgemm_logprobs_workspace_size(m, n, "f32", 20)
    assert need > 0
    at = dict(m=m, n=n, z_type="f32", ldz=n)
    assert check(**at, workspace_bytes=need) == OK and check(**at, workspace_bytes=need - 1) == BAD
    assert check(**at, workspace=None) == BAD and check(**at, workspace=P + 64) == NOT
    assert mp.mpgemm_logprobs_workspace_size(m, 100, "f32", 20) == 0                     # a row is one part
    assert check(m=m, n=100, z_type="f32", ldz=100, workspace=None, workspace_bytes=0) == OK
    for bad in ((0, n, "f32", 20), (m, 0, "f32", 20), (m, n, "i8", 20), (m, n, "f32", 65), (m, n, "f32", -1), (BIG, n, "f32", 1)):
        assert mp.mpgemm_logprobs_workspace_size(*bad) == 0


def test_scalars_that_change_their_value():
    """A scalar is taken by its value at the call: a tensor that holds another one the next time is taken anew."""
    import torch
    alpha = torch.tensor(1.0)
    assert check(alpha=alpha) == OK
    alpha.fill_(-1.0)
    assert check(alpha=alpha) == BAD
    for i in range(200):                                     # more values than are kept
        assert check(alpha=0.5 + i) == OK and check(alpha=-0.5 - i) == BAD
