"""Gated products and their gradient where every row of the outputs is whole 128-byte lines, as a model's widths are:
whole tiles are then stored past the caches.  And their tiles of 256, among them the order of rounds that rows a
multiple of 32 KB apart get.

Whole numbers without an activation have one right result: products of -1, 0 and 1 over k, times -2 .. 2, and their
sums over the rows are at most 2 k m < 2^24 at the sizes here, so that FP32 holds every one of them in any order, and 16 bits
round once.  With an activation the bounds are those of tests/gated_reference.py."""
import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import gated_plans
from tests import gated_reference as gref
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def whole(n):
    return -(-n // 64) * 64


def pair(rows, n, t, layout, fill):
    """(buffer, first, second, elements between them), both of whole lines; what is not theirs is `fill`."""
    c = whole(n)
    if layout == "beside":
        buf = torch.full((rows + 1, 2 * c), fill, dtype=ref.TYPES[t], device="cuda")
        return buf, buf[:rows, :n], buf[:rows, c:c + n], c
    buf = torch.full((2 * rows + 1, c), fill, dtype=ref.TYPES[t], device="cuda")
    return buf, buf[:rows, :n], buf[rows:2 * rows, :n], rows * c


def single(rows, n, t, fill):
    buf = torch.full((rows + 1, whole(n)), fill, dtype=ref.TYPES[t], device="cuda")
    return buf, buf[:rows, :n]


def numbers(gen, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").float()


def ends_of(shares, m):
    ends = [0]
    for s in [m] if shares is None else shares:
        ends.append(ends[-1] + s)
    return ends


def grad_call(transb, m, n, k, t, A, B, kept, stride_kept, act, D, out, stride_d, H, dbias, shares):
    count = 1 if shares is None else len(shares)
    size = mp.mpgemm_gated_grad_workspace_size(count, m, n)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    grad = mp.GatedGrad(act=act, kept=kept, ld_kept=kept.stride(0), stride_kept=stride_kept, H=H, ldh=H.stride(0), dbias=dbias)
    if shares is None:
        mp.mpgemm_run_gated_grad(handle().h, transb, m, n, k, 1.0, A, t, A.stride(0), B, t, B.stride(1), grad, D, out, D.stride(0), stride_d, ws,
                                 size)
    else:
        offsets = torch.tensor(ends_of(shares, m), dtype=torch.int32, device="cuda")
        mp.mpgemm_run_grouped_gated_grad(handle().h, transb, count, m, n, k, 1.0, A, t, A.stride(0), offsets, B, t, B.stride(1),
                                         B.stride(0), grad, D, out, D.stride(0), stride_d, ws, size)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xFF).all())


# (m, n, k, rows of each expert); tiles of 256 but for the first
GRADS = [(300, 320, 200, None), (2048, 8192, 1000, None), (4096, 8192, 1000, None), (6144, 8192, 520, None), (2048, 16384, 520, None),
         (4050, 4072, 1096, None), (4033, 4090, 1000, None), (6144, 4096, 1100, [2048, 0, 2300, 650])]


@pytest.mark.parametrize("layout", ["beside", "after"])
@pytest.mark.parametrize("out", ["f32", "same"])
@pytest.mark.parametrize("t,tb", [("bf16", False), ("f16", True), ("bf16", True), ("f16", False)])
@pytest.mark.parametrize("m,n,k,shares", GRADS)
def test_gradients_of_whole_numbers(m, n, k, shares, t, tb, out, layout):
    kind, count = out if out == "f32" else t, 1 if shares is None else len(shares)
    if gated_plans.available():
        kernel = gated_plans.gated_grad(0 if shares is None else count, m, n, k, "none", True)
        say(f"[gpu gated] grad {m}x{n}x{k} {t}->{kind} tb={tb} {layout} {shares}: {kernel}")
        assert kernel == ("tile", 64 if m == 300 else 256)
    g, ty = rng(m + n), ref.TYPES[t]
    k8 = -(-k // 8) * 8
    A = numbers(g, 1, m, k8).to(ty)
    A[:, k:] = float("nan")
    B = numbers(g, 1, count, *((n, k8) if tb else (k, whole(n)))).to(ty)
    B[:, :, (k if tb else n):] = float("nan")
    kept, G, U, stride_kept = pair(m, n, t, layout, float("nan"))
    G.copy_(numbers(g, 2, m, n))
    U.copy_(numbers(g, 2, m, n))
    dbuf, dG, dU, stride_d = pair(m, n, kind, layout, ref.SENTINEL)
    hbuf, H = single(m, n, t, ref.SENTINEL)
    dbias = torch.full((2 * n * count + 8,), ref.SENTINEL, device="cuda")
    grad_call(tb, m, n, k, t, A, B, kept, stride_kept, "none", dbuf, kind, stride_d, H, dbias, shares)
    ends = ends_of(shares, m)
    for e in range(count):
        r, b = slice(ends[e], ends[e + 1]), (B[e, :, :k].t() if tb else B[e, :, :n]).float()
        E = A[r, :k].float() @ b
        want_g, want_u = E * U[r].float(), E * G[r].float()
        at = 2 * n * e
        assert torch.equal(dG[r], want_g.to(dG.dtype)) and torch.equal(dU[r], want_u.to(dU.dtype)), f"expert {e}"
        assert torch.equal(H[r], G[r] * U[r])
        assert torch.equal(dbias[at:at + n], want_g.double().sum(0).float())
        assert torch.equal(dbias[at + n:at + 2 * n], want_u.double().sum(0).float())
    done = ends[-1]
    assert gref.pair_untouched(dbuf, dG[:done], dU[:done]) and ref.untouched(hbuf, done, n)
    assert bool((dbias[2 * n * count:] == ref.SENTINEL).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,out,tb", [("bf16", "bf16", False), ("f16", "f32", True)])
@pytest.mark.parametrize("m,n,k", [(600, 512, 200), (1200, 2112, 200), (4033, 4090, 1000)])
def test_gradients_with_an_activation(m, n, k, t, out, tb, act):
    g, ty = rng(m + k), ref.TYPES[t]
    say(f"[gpu gated] grad {m}x{n}x{k} {t}->{out} tb={tb} {act}")
    A = torch.randn(m, k, generator=g, device="cuda").to(ty)
    B = (torch.randn(1, *((n, k) if tb else (k, whole(n))), generator=g, device="cuda") * k ** -0.5).to(ty)
    kept, G, U, stride_kept = pair(m, n, t, "beside", float("nan"))
    for x in (G, U):
        x.copy_(2 * torch.randn(m, n, generator=g, device="cuda"))
    dbuf, dG, dU, stride_d = pair(m, n, out, "after", ref.SENTINEL)
    hbuf, H = single(m, n, t, ref.SENTINEL)
    dbias = torch.empty(2 * n, device="cuda")
    grad_call(tb, m, n, k, t, A, B, kept, stride_kept, act, dbuf, out, stride_d, H, dbias, None)
    # (64 bits would take long over all rows of the largest)
    r = torch.arange(m) if m * n < 3e6 else torch.cat([torch.arange(20), torch.arange(250, 262), torch.arange(1020, 1030), torch.arange(m - 70, m)])
    z, z_err = ref.product64(A[r], B[0].t() if tb else B[0, :, :n], k)
    for (v, err), got, name, kind in zip(gref.grad64(z, z_err, G[r], U[r], act), (dG, dU, H), ("dG", "dU", "H"), (out, out, t)):
        gref.check(got[r], v, err, kind, name)
    assert gref.pair_untouched(dbuf, dG, dU) and ref.untouched(hbuf, m, n)


@pytest.mark.parametrize("layout", ["beside", "after"])
@pytest.mark.parametrize("t,out,tb", [("bf16", "bf16", True), ("f16", "f32", False), ("f16", "f16", True)])
@pytest.mark.parametrize("m,n,k,shares", [(600, 512, 200, None), (1200, 2112, 200, None), (1200, 2100, 200, None), (2100, 2176, 1096, None),
                                          (2600, 1408, 264, [1000, 0, 1, 700, 300, 500])])
def test_products(m, n, k, shares, t, out, tb, layout):
    count = 1 if shares is None else len(shares)
    if gated_plans.available():
        say(f"[gpu gated] {m}x{n}x{k} {t}->{out} tb={tb} {layout}: {gated_plans.gated(0 if shares is None else count, m, n, k, tb, 'silu', True)}")
    g, ty, c = rng(m + n), ref.TYPES[t], whole(n)
    A = torch.randn(m, k, generator=g, device="cuda").to(ty)
    # an expert's pair: the gate's rows or columns, then the up projection's
    B = (torch.randn(count, *((2 * n, k) if tb else (k, 2 * c)), generator=g, device="cuda") * k ** -0.5).to(ty)
    bias = torch.randn(2, count, n, generator=g, device="cuda")
    kept, G, U, stride_kept = pair(m, n, t, layout, ref.SENTINEL)
    dbuf, D = single(m, n, out, ref.SENTINEL)
    gated = mp.Gated(act="silu", bias_gate=bias[0], bias_up=bias[1], bias_stride=n, kept=kept, ld_kept=kept.stride(0), stride_kept=stride_kept)
    up = n * k if tb else c
    if shares is None:
        mp.mpgemm_run_gated(handle().h, tb, m, n, k, 1.0, A, t, k, B, t, B.stride(1), up, gated, D, out, D.stride(0))
    else:
        offsets = torch.tensor(ends_of(shares, m), dtype=torch.int32, device="cuda")
        mp.mpgemm_run_grouped_gated(handle().h, tb, count, m, n, k, 1.0, A, t, k, offsets, B, t, B.stride(1), B.stride(0), up, gated, D, out,
                                    D.stride(0))
    torch.cuda.synchronize()
    ends = ends_of(shares, m)
    for e in range(count):
        r = slice(ends[e], ends[e + 1])
        first, second = (B[e, :n].t(), B[e, n:].t()) if tb else (B[e, :, :n], B[e, :, c:c + n])
        (d, d_err), (gz, g_err), (uz, u_err) = gref.forward64(A[r], first, second, k, "silu", bias[0, e], bias[1, e])
        gref.check(D[r], d, d_err, out, f"D of {e}")
        gref.check(G[r], gz, g_err, t, f"G of {e}")
        gref.check(U[r], uz, u_err, t, f"U of {e}")
    done = ends[-1]
    assert ref.untouched(dbuf, done, n) and gref.pair_untouched(kept, G[:done], U[:done])
