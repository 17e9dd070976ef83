"""The order in which a grid takes its tiles: every tile once, whatever their number and shape, with rows that
take no part and with last tiles that hold few rows."""
import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import distill_reference as dref
from tests import ops_reference as ref
from tests.gpu_harness import handle, say
from tests.test_gpu_distill import call
from tests.test_gpu_gated import run_forward

pytestmark = pytest.mark.gpu


def rng(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("k", [8, 300])
@pytest.mark.parametrize("m", [5, 70, 300, 517, 700, 1100, 1400, 2300, 4500, 6000])
def test_every_tile_once(m, k):
    """Small whole numbers, whose sums FP32 holds exactly, so that a product has one right result."""
    g = rng(m + k)
    a = torch.randint(-3, 4, (m, 8 * (k // 8 + 1)), generator=g).bfloat16().cuda()[:, :k]
    for n in (20, 130, 800, 2100, 3300, 6000):
        say(f"[gpu order] {m}x{n}x{k}")
        b = torch.randint(-3, 4, (n, a.stride(0)), generator=g).bfloat16().cuda()[:, :k]
        buf, d = ref.output(m, n, "f32")
        mp.mpgemm_run_epilogue(handle().h, False, True, m, n, k, 1.0, a, "bf16", a.stride(0), b, "bf16", b.stride(0), mp.Epilogue(), 0.0,
                               None, "f32", n, d, "f32", d.stride(0))
        torch.cuda.synchronize()
        assert torch.equal(d, a.float() @ b.float().t()), (m, n, k)
        assert ref.untouched(buf, m, n)


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("m,n,k,shares", [(1025, 2300, 90, None), (1088, 2300, 90, None), (1089, 2300, 90, None),     # tiles of 128
                                          (2049, 2200, 1100, None), (2177, 2200, 1100, None),                       # of 256
                                          (1600, 2300, 90, [1025, 64, 0, 65, 1, 128, 192, 100])])
def test_gated_last_tiles_of_few_rows(m, n, k, shares, tb):
    run_forward(m, n, k, "bf16", "f32", tb, "silu", "after", ("f32", None), "beside", seed=m, shares=shares)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k,share", [(300, 2000, 72, 0.5), (700, 5000, 40, 0.1), (700, 5000, 200, 0.9), (1300, 3000, 136, 0.6),
                                         (1300, 700, 520, 0.99)])
def test_gradients_with_rows_that_do_not_count(m, n, k, share, t):
    g = rng(m + n)
    x, w = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, 2.0 * k ** -0.5)
    index, logit = dref.teacher(g, m, n, 6, "plain")
    ignored = (torch.rand(m, generator=g) < share).cuda()
    index[ignored] = -1
    grads = torch.randn(m, generator=g).cuda()
    got = call(x, w, t, index, logit, 0.7, None, 1.0, grads)
    d = dref.distill64(x, w, index, logit, 0.7, None, 1.0, k)
    dx, dx_err, dw, dw_err = dref.distill_grad64(x, w, d, grads, 1.0, k, t)
    ref.assert_within(got[0], d["loss"], d["loss_err"], "loss")
    ref.assert_within(got[3], dx, dx_err, "dX")
    ref.assert_within(got[4], dw, dw_err, "dW")
    assert bool((got[3][ignored] == 0).all())


@pytest.mark.parametrize("m", [2000, 4096, 6144])
def test_rows_of_a_multiple_of_32_kb(m):
    """Where D's rows are that far apart a round of 256-wide tiles is laid out differently."""
    n, k = 8192, 1000
    g = rng(m)
    a, b = (torch.randint(-3, 4, (r, k), generator=g).bfloat16().cuda() for r in (m, n))
    want = a.float() @ b.float().t()
    for out in ("f32", "bf16"):
        ld = n if out == "f32" else 2 * n
        d = torch.full((m + 1, ld), ref.SENTINEL, dtype=ref.TYPES[out], device="cuda")
        mp.mpgemm_run_epilogue(handle().h, False, True, m, n, k, 1.0, a, "bf16", k, b, "bf16", k, mp.Epilogue(), 0.0, None, out, ld, d, out,
                               ld)
        torch.cuda.synchronize()
        assert torch.equal(d[:m, :n], want.to(ref.TYPES[out])), (m, out)
        assert bool((d[m] == ref.SENTINEL).all()) and bool((d[:, n:] == ref.SENTINEL).all())
