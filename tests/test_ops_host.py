"""The host-only argument checks of the products of language models: every refusal, and what is let
through.  CPU only (addresses are never dereferenced)."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

import mixed_precision_dense_amd as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if not os.path.exists(mp.LIB_PATH):
    from mixed_precision_dense_amd import build as _b
    _b.build()

ST = {v: k for k, v in mp.STATUS.items()}
OK, BAD, NOT = ST["SUCCESS"], ST["INVALID_VALUE"], ST["NOT_SUPPORTED"]
P = 1 << 20        # a 256-byte aligned fake device address
BIG = (1 << 31) - 1


def checker(fn, defaults):
    def check(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a), set(kw) - set(a)
        a.update(kw)
        return fn(*a.values())
    check.names = set(defaults)
    return check


def epi(**kw):
    return mp.Epilogue(**kw)


EPILOGUE = dict(transa=False, transb=True, m=100, n=64, k=72, alpha=1.0, A=P, a_type="bf16", lda=72, B=P, b_type="bf16", ldb=72,
                epilogue=epi(), beta=0.0, C=None, c_type="bf16", ldc=64, D=P, d_type="bf16", ldd=64)
GRAD = dict(transa=False, transb=True, m=100, n=64, k=72, alpha=1.0, A=P, a_type="bf16", lda=72, B=P, b_type="bf16", ldb=72,
            act="silu", Z=P, ldz=64, D=P, d_type="f32", ldd=64, dbias=P, workspace=P, workspace_bytes=1 << 20)
GROUPED = dict(transb=True, groups=4, rows=100, n=64, k=72, alpha=1.0, A=P, a_type="f16", lda=72, offsets=P, B=P, b_type="f16",
               ldb=72, stride_b=64 * 72, epilogue=epi(), D=P, d_type="f16", ldd=64)
GROUPED_GRAD = dict(transb=True, groups=4, rows=100, n=64, k=72, alpha=1.0, A=P, a_type="f16", lda=72, offsets=P, B=P,
                    b_type="f16", ldb=72, stride_b=64 * 72, act="silu", Z=P, ldz=64, D=P, d_type="f16", ldd=64, dbias=P,
                    workspace=P, workspace_bytes=1 << 20)
WGRAD = dict(groups=4, rows=100, m=72, n=64, alpha=1.0, A=P, a_type="f16", lda=72, X=P, x_type="f16", ldx=64, offsets=P,
             beta=0.0, D=P, d_type="f32", ldd=64, stride_d=72 * 64)
CE = dict(m=100, n=500, k=72, alpha=1.0, X=P, dtype="bf16", ldx=72, W=P, ldw=72, target=P, loss=P, lse=P, workspace=P,
          workspace_bytes=1 << 24)
CE_GRAD = dict(m=100, n=500, k=72, alpha=1.0, X=P, dtype="bf16", ldx=72, W=P, ldw=72, target=P, lse=P, grad=P, dX=P, lddx=72,
               dW=P, lddw=72, workspace=P, workspace_bytes=1 << 24)

epilogue = checker(mp.mpgemm_check_epilogue, EPILOGUE)
epilogue_grad = checker(mp.mpgemm_check_epilogue_grad, GRAD)
grouped = checker(mp.mpgemm_check_grouped, GROUPED)
grouped_grad = checker(mp.mpgemm_check_grouped_grad, GROUPED_GRAD)
wgrad = checker(mp.mpgemm_check_grouped_wgrad, WGRAD)
ce = checker(mp.mpgemm_check_linear_ce, CE)
ce_grad = checker(mp.mpgemm_check_linear_ce_grad, CE_GRAD)
ALL = [epilogue, epilogue_grad, grouped, grouped_grad, wgrad, ce, ce_grad]
TYPED = [(epilogue, "a_type", "b_type"), (epilogue_grad, "a_type", "b_type"), (grouped, "a_type", "b_type"),
         (grouped_grad, "a_type", "b_type"), (wgrad, "a_type", "x_type")]


@pytest.mark.parametrize("check", ALL)
def test_the_defaults_pass(check):
    assert check() == OK


@pytest.mark.parametrize("check,a,b", TYPED)
def test_types(check, a, b):
    for t in ("f16", "bf16"):
        assert check(**{a: t, b: t, "d_type": t}) == OK
        assert check(**{a: t, b: t, "d_type": "f32"}) == OK
    assert check(**{a: "f16", b: "bf16", "d_type": "f32"}) == NOT
    assert check(**{a: "bf16", b: "bf16", "d_type": "f16"}) == NOT
    for t in ("f32", "i8", "e4m3", 9, -1):
        assert check(**{a: t, b: t, "d_type": "f32"}) == NOT


def test_other_types():
    assert epilogue(beta=1.0, C=P, c_type="f32") == OK                       # C apart from D
    assert epilogue(beta=1.0, C=P, c_type="f16") == NOT
    assert epilogue(c_type="i32") == OK                                      # not read
    for t, want in (("bf16", OK), ("f32", OK), ("f16", NOT), ("i8", NOT)):
        assert epilogue(epilogue=epi(bias=P, bias_type=t)) == want
    assert grouped(epilogue=epi(bias=P, bias_type="bf16", bias_stride=64)) == NOT
    for c in (ce, ce_grad):
        assert c(dtype="f16") == OK and c(dtype="f32") == NOT and c(dtype=17) == NOT


@pytest.mark.parametrize("check", ALL)
def test_negative_sizes(check):
    for name in {"m", "n", "k", "groups", "rows"} & check.names:
        assert check(**{name: -1}) == BAD, name


def test_empty_products():
    none = dict(A=None, B=None, D=None)
    assert epilogue(m=0, **none) == OK and epilogue(n=0, **none) == OK
    assert epilogue(k=0, A=None, B=None) == OK
    assert epilogue_grad(n=0, Z=None, dbias=None, workspace=None, **none) == OK
    assert epilogue_grad(m=0, Z=None, workspace=None, workspace_bytes=0, **none) == OK     # dbias = 0 is written
    assert epilogue_grad(m=0, dbias=P + 2, **none) == NOT
    assert grouped(groups=0, offsets=None, **none) == OK and grouped(rows=0, offsets=None, **none) == OK
    assert grouped_grad(rows=0, Z=None, **none) == OK and grouped_grad(rows=0, offsets=None, Z=None, **none) == BAD
    assert grouped_grad(rows=0, dbias=None, offsets=None, Z=None, **none) == OK
    assert wgrad(m=0, A=None, X=None, D=None, offsets=None) == OK
    assert wgrad(rows=0, A=None, X=None) == OK and wgrad(rows=0, A=None, X=None, D=None) == BAD
    assert ce(m=0, X=None, W=None, target=None, loss=None, lse=None, workspace=None) == OK
    assert ce(n=0) == BAD and ce_grad(n=0) == BAD                            # no log of an empty sum
    assert ce(k=0, X=None, W=None) == OK
    assert ce_grad(m=0, X=None, W=None, target=None, lse=None, grad=None, workspace=None) == OK
    assert ce_grad(dX=None) == OK and ce_grad(dW=None) == OK and ce_grad(dX=None, dW=None) == OK
    assert ce_grad(k=0, X=None, W=None) == OK


@pytest.mark.parametrize("check,names", [
    (epilogue, ["A", "B", "D"]), (epilogue_grad, ["A", "B", "Z", "D", "workspace"]), (grouped, ["A", "offsets", "B", "D"]),
    (grouped_grad, ["A", "offsets", "B", "Z", "D", "workspace"]), (wgrad, ["A", "X", "offsets", "D"]),
    (ce, ["X", "W", "target", "loss", "lse", "workspace"]), (ce_grad, ["X", "W", "target", "lse", "grad", "workspace"])])
def test_null_pointers(check, names):
    for name in names:
        assert check(**{name: None}) == BAD, name


def test_other_nulls_and_values():
    assert epilogue(beta=1.0, C=None) == BAD and epilogue(beta=float("nan"), C=None) == BAD
    assert epilogue(beta=-0.0, C=None) == OK
    assert epilogue(epilogue=None) == BAD and grouped(epilogue=None) == BAD
    for act in (-1, 5):
        assert epilogue(epilogue=epi(act=act)) == BAD and epilogue_grad(act=act) == BAD and grouped_grad(act=act) == BAD
    assert epilogue_grad(act="none", Z=None, ldz=0) == OK                    # Z is not read
    assert grouped_grad(act="none", Z=None, ldz=0) == OK
    assert epilogue_grad(dbias=None, workspace=None, workspace_bytes=0) == OK
    assert grouped(stride_b=0) == OK and grouped(stride_b=-8) == BAD         # one B for all
    assert grouped(epilogue=epi(bias=P, bias_type="f16", bias_stride=-1)) == BAD
    one = ctypes.c_float(1.0)
    lib = mp.load()
    assert lib.mpgemm_check_linear_ce(1, 8, 8, None, P, 0, 8, P, 8, P, P, P, P, 1 << 20) == BAD
    assert lib.mpgemm_check_epilogue(2, 0, 8, 8, 8, ctypes.byref(one), P, 0, 8, P, 0, 8, ctypes.byref(epi().struct),
                                     ctypes.byref(one), P, 3, 8, P, 3, 8) == BAD
    assert lib.mpgemm_check_epilogue(0, 0, 8, 8, 8, ctypes.byref(one), P, 0, 8, P, 0, 8, ctypes.byref(epi().struct), None, P, 3, 8,
                                     P, 3, 8) == BAD


@pytest.mark.parametrize("check,names", [
    (epilogue, ["lda", "ldb", "ldd"]), (epilogue_grad, ["lda", "ldb", "ldz", "ldd"]), (grouped, ["lda", "ldb", "ldd"]),
    (grouped_grad, ["lda", "ldb", "ldz", "ldd"]), (wgrad, ["lda", "ldx", "ldd"]), (ce, ["ldx", "ldw"]),
    (ce_grad, ["ldx", "ldw", "lddx", "lddw"])])
def test_leading_dimensions(check, names):
    for name in names:
        assert check(**{name: 56}) == BAD, name                              # below the row
        assert check(**{name: 73}) == NOT, name                              # no whole 16-byte blocks
        assert check(**{name: 1 << 22}) == NOT, name                         # past what offsets reach
        assert check(**{name: (1 << 63) - 8}) == NOT, name
    if check is wgrad:
        assert check(ldd=72) == BAD and check(ldd=72, stride_d=72 * 72) == OK


def test_epilogue_leading_dimensions():
    assert epilogue(transa=True, lda=96) == BAD and epilogue(transa=True, lda=104) == OK
    assert epilogue(transb=False, ldb=56) == BAD and epilogue(transb=False, ldb=64) == OK
    assert epilogue(beta=1.0, C=P, ldc=56) == BAD and epilogue(beta=1.0, C=P, ldc=66) == NOT and epilogue(ldc=1) == OK
    assert epilogue(epilogue=epi(aux=P, ld_aux=56)) == BAD and epilogue(epilogue=epi(aux=P, ld_aux=66)) == NOT
    assert epilogue(epilogue=epi(aux=P, ld_aux=72)) == OK
    assert grouped(stride_b=64 * 72 + 4) == NOT and grouped(stride_b=1 << 62) == NOT
    assert wgrad(stride_d=72 * 64 - 8) == BAD and wgrad(stride_d=72 * 64 + 2) == NOT and wgrad(stride_d=1 << 62) == NOT
    assert wgrad(groups=1, stride_d=0) == OK


@pytest.mark.parametrize("check,names", [
    (epilogue, ["A", "B", "D"]), (epilogue_grad, ["A", "B", "Z", "D"]), (grouped, ["A", "B", "D"]),
    (grouped_grad, ["A", "B", "Z", "D"]), (wgrad, ["A", "X", "D"]), (ce, ["X", "W"]), (ce_grad, ["X", "W", "dX", "dW"])])
def test_alignment(check, names):
    for name in names:
        assert check(**{name: P + 8}) == NOT, name


def test_other_alignments():
    assert epilogue(beta=1.0, C=P + 8) == NOT and epilogue(C=P + 8) == OK
    assert epilogue(epilogue=epi(aux=P + 8, ld_aux=64)) == NOT
    assert epilogue(epilogue=epi(bias=P + 2, bias_type="bf16")) == OK        # a bias has its elements' alignment
    assert epilogue(epilogue=epi(bias=P + 2, bias_type="f32")) == NOT
    assert epilogue(epilogue=epi(bias=P + 1, bias_type="bf16")) == NOT
    assert grouped(offsets=P + 2) == NOT and wgrad(offsets=P + 2) == NOT
    assert epilogue_grad(dbias=P + 2) == NOT and epilogue_grad(workspace=P + 128) == NOT
    assert grouped_grad(dbias=P + 2) == NOT and grouped_grad(workspace=P + 16) == NOT
    for name in ("loss", "lse"):
        assert ce(**{name: P + 2}) == NOT
    assert ce(target=P + 4) == NOT and ce(workspace=P + 64) == NOT
    assert ce_grad(target=P + 4) == NOT and ce_grad(grad=P + 2) == NOT and ce_grad(lse=P + 2) == NOT
    assert ce_grad(workspace=P + 64) == NOT


def test_size_limits():
    top = BIG - 255
    tall = dict(transa=True, transb=False, m=8, n=8, lda=8, ldb=8, ldd=8)
    assert epilogue(k=top, **tall) == OK and epilogue(k=top + 1, **tall) == NOT
    assert epilogue(m=top + 1) == NOT and epilogue(m=BIG + 1) == NOT
    assert epilogue(m=top, n=1 << 20, ldd=1 << 20) == NOT                    # more tiles than a launch holds
    assert epilogue(m=1, n=1 << 21, ldd=1 << 21) == OK
    assert grouped(groups=65535, rows=70000) == OK and grouped(groups=65536, rows=70000) == NOT
    assert wgrad(groups=65536) == NOT and grouped_grad(groups=65536, rows=0, A=None, B=None, D=None, Z=None) == NOT
    assert wgrad(groups=60000, m=4096, lda=4096, stride_d=4096 * 64) == OK
    assert wgrad(groups=60000, m=40000, n=4096, lda=40000, ldx=4096, ldd=4096, stride_d=40000 * 4096) == NOT
    assert ce(n=top + 1) == NOT and ce_grad(m=BIG + 1) == NOT


def test_workspaces():
    size = mp.mpgemm_epilogue_grad_workspace_size
    assert size(1, 100, 61) == size(1, 100, 64) > 0                          # rows of whole 8-column blocks
    assert size(0, 8, 8) == size(1, 0, 8) == size(1, 8, 0) == size(1, -1, 8) == size(65536, 8, 8) == 0
    assert size(8, 100, 64) > size(1, 100, 64)
    need = size(1, 100, 64)
    assert epilogue_grad(workspace_bytes=need) == OK and epilogue_grad(workspace_bytes=need - 1) == BAD
    need = size(4, 100, 64)
    assert grouped_grad(workspace_bytes=need) == OK and grouped_grad(workspace_bytes=need - 1) == BAD
    for train, check in ((False, ce), (True, ce_grad)):
        need = mp.mpgemm_linear_ce_workspace_size(100, 500, 72, "bf16", train)
        assert check(workspace_bytes=need) == OK and check(workspace_bytes=need - 1) == BAD
    # enough for both when the gradients follow, and far from the logits' size
    for m, n, k in ((8, 32000, 4096), (4096, 128000, 4096), (1 << 20, 500, 64)):
        both = mp.mpgemm_linear_ce_workspace_size(m, n, k, "bf16", True)
        assert both >= mp.mpgemm_linear_ce_workspace_size(m, n, k, "bf16", False) > 0
    assert mp.mpgemm_linear_ce_workspace_size(4096, 128000, 4096, "bf16", True) < 4096 * 128000 * 2 / 4
    for args in ((-1, 8, 8, "f16"), (8, 0, 8, "f16"), (8, 8, -1, "f16"), (8, 8, 8, "f32"), (0, 8, 8, "f16")):
        assert mp.mpgemm_linear_ce_workspace_size(*args, True) == 0


def test_sizes_past_one_launch():
    """Rows and blocks past the workgroups of one launch are walked by the kernels beside the products."""
    big = dict(workspace_bytes=1 << 61)
    for m in ((1 << 24) - 1, 1 << 24, 20_000_000):
        assert ce(m=m, n=16, k=64, **big) == OK and ce_grad(m=m, n=16, k=64, **big) == OK
    assert ce_grad(m=1 << 22, n=16, k=8192, ldx=8192, ldw=8192, lddx=8192, lddw=8192, **big) == OK
    assert epilogue_grad(m=0, n=(1 << 30) + 64, ldd=1 << 31, ldz=1 << 31, A=None, B=None, D=None, Z=None) == OK


def test_unknown_handles():
    for run, args in ((mp.mpgemm_run_epilogue, EPILOGUE), (mp.mpgemm_run_epilogue_grad, GRAD), (mp.mpgemm_run_grouped, GROUPED),
                      (mp.mpgemm_run_grouped_grad, GROUPED_GRAD), (mp.mpgemm_run_grouped_wgrad, WGRAD),
                      (mp.mpgemm_run_linear_ce, CE), (mp.mpgemm_run_linear_ce_grad, CE_GRAD)):
        assert run(0x1000, *args.values(), stream=0, check=False) == ST["NOT_INITIALIZED"]
        with pytest.raises(mp.MpgemmError, match=run.__name__):
            run(0x1000, *args.values(), stream=0)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ builds the host checks")
def test_host_checks_under_address_and_ub_sanitizers(tmp_path):
    """The tests above (without the handle's) against the host-only sources built with sanitizers."""
    asan = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("no address sanitizer runtime")
    csrc = os.path.join(ROOT, "mixed_precision_dense_amd", "csrc")
    lib = str(tmp_path / "libmpgemm_ops_host_san.so")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-g", "-O1", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o", lib,
                    os.path.join(csrc, "mpgemm_host.cpp"), os.path.join(csrc, "mpgemm_ops_host.cpp")], check=True)
    env = dict(os.environ, MPGEMM_HOST_CHECK_LIB=lib, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", OMP_NUM_THREADS="4")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-s", "-p", "no:cacheprovider", "-m", "not gpu", __file__, "-k",
                        "not unknown_handles and not sanitizers"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout[-3000:] + r.stderr[:3000]
