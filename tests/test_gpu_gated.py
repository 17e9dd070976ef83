"""The gated products on the GPU -- forward and gradient, dense and of experts' rows -- against the same
in 64 bits, at the sizes where tiles, blocks and stages end.  What lies past the operands' rows and
between a pair's matrices is NaN; what lies past and between the outputs must stay as it was."""
import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import gated_plans
from tests import gated_reference as gref
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def rng(seed):
    return torch.Generator().manual_seed(seed)


def weights(gen, n, k, t, tb, layout, count, scale=1.0):
    """count pairs of weights in one buffer: (buffer view, ld, stride_b, stride_up, [(Bg, Bu)] as k x n)."""
    rows, cols = (n, k) if tb else (k, n)
    pairs = [gref.pair(gen, rows, cols, t, layout, scale * max(k, 1) ** -0.5) for _ in range(count)]
    size = pairs[0][0].numel()
    whole = torch.full((count * size,), float("nan"), dtype=ref.TYPES[t], device="cuda")
    out = []
    for e, (buf, a, b, _) in enumerate(pairs):
        part = whole[e * size:(e + 1) * size].view(buf.shape)
        part.copy_(buf)
        out.append(((a.t(), b.t()) if tb else (a, b)))
    return whole, pairs[0][0].stride(0), size, pairs[0][3], out


def offsets_of(shares, rows, gen):
    """Cumulative rows of each expert."""
    counts = [int(s) for s in shares]
    assert sum(counts) <= rows
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    return torch.tensor(ends, dtype=torch.int32, device="cuda"), ends


def run_forward(m, n, k, t, out, tb, act, layout="after", biases=(None, None), kept=None, alpha=1.0, seed=0, scale=1.0, shares=None):
    """shares: None (one product) or each expert's rows."""
    say(f"[gpu gated] {m}x{n}x{k} {t}->{out} tb={tb} {act} {layout} bias={biases} kept={kept} shares={shares}")
    g = rng(seed)
    count = 1 if shares is None else len(shares)
    A = ref.matrix(g, m, k, t, scale)
    B, ldb, stride_b, up, ws = weights(g, n, k, t, tb, layout, count)
    bt = biases[0] or biases[1] or "f32"
    bias = [None if b is None else torch.randn(count, n + 3, generator=g).to(ref.TYPES[bt]).cuda() for b in biases]
    dbuf, D = ref.output(m, n, out)
    kbuf, G, U, stride = gref.pair_out(m, n, t, kept) if kept else (None, None, None, 0)
    gated = mp.Gated(act=act, bias_gate=bias[0], bias_up=bias[1], bias_type=bt, bias_stride=n + 3, kept=kbuf,
                     ld_kept=kbuf.stride(0) if kept else 0, stride_kept=stride)
    if shares is None:
        mp.mpgemm_run_gated(handle().h, tb, m, n, k, alpha, A, t, A.stride(0), B, t, ldb, up, gated, D, out, D.stride(0))
        ends = [0, m]
    else:
        offs, ends = offsets_of(shares, m, g)
        mp.mpgemm_run_grouped_gated(handle().h, tb, count, m, n, k, alpha, A, t, A.stride(0), offs, B, t, ldb, stride_b, up, gated, D,
                                    out, D.stride(0))
    torch.cuda.synchronize()
    for e in range(count):
        r = slice(ends[e], ends[e + 1])
        bv = [None if b is None else b[e, :n] for b in bias]
        (d, d_err), (gz, g_err), (uz, u_err) = gref.forward64(A[r], *ws[e], k, act, *bv, alpha)
        gref.check(D[r], d, d_err, out, f"D of {e}")
        if kept:
            gref.check(G[r], gz, g_err, t, f"G of {e}")
            gref.check(U[r], uz, u_err, t, f"U of {e}")
    done = ends[-1]
    assert ref.untouched(dbuf, done, n)
    if kept:
        assert gref.pair_untouched(kbuf, G[:done], U[:done])


# ----------------------------------------------------------------------------- forward
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("layout", ["beside", "after"])
@pytest.mark.parametrize("m,n,k", [(1, 256, 64), (1, 5, 1), (2, 17, 129), (15, 33, 71), (16, 16, 32), (17, 40, 1001), (33, 97, 130),
                                   (64, 64, 1024), (65, 7, 63), (100, 130, 200), (129, 257, 65), (300, 520, 136)])
def test_forward_sizes(m, n, k, tb, layout):
    t, out = ("bf16", "f32") if (m + n) % 2 else ("f16", "f16")
    run_forward(m, n, k, t, out, tb, "gelu", layout, (t, t), "beside" if n % 3 else "after", seed=m * n + k)


# one size for each kernel that the rules can choose; (groups' mean rows, n, k) with both storages
# (of few rows and many columns, and tiles of 256, in tests/gated_cases.py: no size here reaches those)
KERNELS = [(0, 9, 100, 200), (0, 9, 24600, 72), (0, 30, 100, 200), (0, 30, 12000, 72), (0, 60, 100, 200), (0, 200, 100, 70),
           (0, 900, 1100, 130), (0, 2100, 2200, 72), (3, 12, 100, 200), (40, 300, 500, 72), (3, 60, 200, 136), (3, 600, 300, 72)]


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("groups,m,n,k", KERNELS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_forward_kernels(groups, m, n, k, tb, t):
    shares = None
    if groups:
        cut = torch.rand(groups, generator=rng(m)) + 0.1
        shares = [int(v) for v in (cut / cut.sum() * m).floor()]
        shares[1] = 0
    say(f"[gpu gated] kernel {gated_plans.gated(groups, m, n, k, tb) if gated_plans.available() else '?'}")
    run_forward(m, n, k, t, t, tb, "silu", "after", (None, "f32"), "beside", seed=n, shares=shares)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("m", [3, 200])
def test_forward_types(act, t, out, m):
    run_forward(m, 200, 96, t, out, True, act, "after", ("f32", None), "after", seed=m, scale=3.0)
    run_forward(m, 72, 96, t, out, False, act, "beside", (None, None), None, alpha=0.5, seed=m + 1)


@pytest.mark.parametrize("m", [4, 150])
def test_forward_without_a_product(m):
    """k = 0: both factors are their biases; A and B may be missing."""
    n = 41
    bias = torch.randn(2, n, generator=rng(3)).cuda()
    dbuf, D = ref.output(m, n, "f32")
    mp.mpgemm_run_gated(handle().h, False, m, n, 0, 1.0, None, "f16", 8, None, "f16", 48, 0,
                        mp.Gated(act="relu", bias_gate=bias[0], bias_up=bias[1]), D, "f32", D.stride(0))
    torch.cuda.synchronize()
    want = (bias[0].double().clamp(min=0) * bias[1].double()).cpu().expand(m, n)
    ref.assert_within(D, want, 2.0 ** -23 * want.abs(), "D")
    assert ref.untouched(dbuf, m, n)


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("m", [5, 90])
def test_forward_nonfinite(m, tb):
    """NaN and infinities of a row of A, or of one column of one weight, reach exactly the outputs they belong to."""
    g, n, k, t = rng(8), 48, 70, "bf16"
    A = ref.matrix(g, m, k, t)
    B, ldb, _, up, ((bg, bu),) = weights(g, n, k, t, tb, "after", 1)
    A[2, 5] = float("nan")
    whole = B.view(-1, ldb)
    if tb:
        whole[7, 3] = float("nan")                       # the gate's column 7
    else:
        whole[3, 7] = float("nan")
    dbuf, D = ref.output(m, n, "f32")
    mp.mpgemm_run_gated(handle().h, tb, m, n, k, 1.0, A, t, A.stride(0), B, t, ldb, up, mp.Gated(act="silu"), D, "f32", D.stride(0))
    torch.cuda.synchronize()
    (d, err), _, _ = gref.forward64(A, bg, bu, k, "silu")
    rows, cols = [r for r in range(m) if r != 2], [c for c in range(n) if c != 7]
    gref.check(D[rows][:, cols], d[rows][:, cols], err[rows][:, cols], "f32", "D")
    assert bool(D[2].isnan().all()) and bool(D[:, 7].isnan().all())


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("shares", [[0, 0, 5], [1, 0, 0, 1], [70, 0, 129, 1], [300], [0, 0]])
def test_experts_without_rows_and_rows_of_no_expert(shares, tb):
    m = sum(shares) + 3                                  # the last rows belong to nobody
    run_forward(m, 72, 65, "bf16", "bf16", tb, "silu", "after", ("bf16", "bf16"), "beside", seed=1, shares=shares)
    if sum(shares):
        run_grad(m, 72, 65, "f16", "f16", tb, "silu", shares=shares, seed=2)


# ----------------------------------------------------------------------------- gradient
def run_grad(m, n, k, t, out, tb, act, layout="beside", made=True, dbias=True, alpha=1.0, seed=0, spread=2.0, shares=None,
             infinite=False):
    say(f"[gpu gated] grad {m}x{n}x{k} {t}->{out} tb={tb} {act} {layout} H={made} shares={shares}")
    g = rng(seed)
    count = 1 if shares is None else len(shares)
    A = ref.matrix(g, m, k, t)
    rows_b, cols_b = (n, k) if tb else (k, n)
    B = ref.matrix(g, count * rows_b, cols_b, t, max(k, 1) ** -0.5)
    kbuf, G, U, ks = gref.pair(g, m, n, t, layout, spread)
    if infinite:
        G[0, 0], G[1, 1], G[0, 2] = float("-inf"), float("-inf"), 0.0
    dbuf, dG, dU, stride_d = gref.pair_out(m, n, out, layout)
    hbuf, H = ref.output(m, n, t) if made else (None, None)
    groups = max(count, 1)
    bbuf = torch.full((groups * 2 * n + 8,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_gated_grad_workspace_size(groups, m, n) if dbias else 0
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    grad = mp.GatedGrad(act=act, kept=kbuf, ld_kept=kbuf.stride(0), stride_kept=ks, H=H, ldh=H.stride(0) if made else 0,
                        dbias=bbuf if dbias else None)
    if shares is None:
        mp.mpgemm_run_gated_grad(handle().h, tb, m, n, k, alpha, A, t, A.stride(0), B, t, B.stride(0), grad, dbuf, out, dbuf.stride(0),
                                 stride_d, ws if dbias else None, size)
        ends = [0, m]
    else:
        offs, ends = offsets_of(shares, m, g)
        mp.mpgemm_run_grouped_gated_grad(handle().h, tb, count, m, n, k, alpha, A, t, A.stride(0), offs, B, t, B.stride(0),
                                         rows_b * B.stride(0), grad, dbuf, out, dbuf.stride(0), stride_d, ws if dbias else None, size)
    torch.cuda.synchronize()
    for e in range(count):
        r = slice(ends[e], ends[e + 1])
        b = B[e * rows_b:(e + 1) * rows_b]
        z, z_err = ref.product64(A[r], b.t() if tb else b, k, alpha)
        (dg, dg_err), (du, du_err), (h, h_err) = gref.grad64(z, z_err, G[r], U[r], act)
        gref.check(dG[r], dg, dg_err, out, f"dG of {e}")
        gref.check(dU[r], du, du_err, out, f"dU of {e}")
        if made:
            gref.check(H[r], h, h_err, t, f"H of {e}")
        if dbias:
            for half, (d, err) in enumerate(((dg, dg_err), (du, du_err))):
                s, s_err = ref.column_sums64(d, err)
                at = (2 * e + half) * n
                ref.assert_within(bbuf[at:at + n], s, s_err, f"dbias {half} of {e}")
    done = ends[-1]
    assert gref.pair_untouched(dbuf, dG[:done], dU[:done])
    if made:
        assert ref.untouched(hbuf, done, n)
    if dbias:
        assert bool((bbuf[groups * 2 * n:] == ref.SENTINEL).all()) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("layout", ["beside", "after"])
@pytest.mark.parametrize("m,n,k", [(1, 9, 40), (16, 64, 64), (31, 100, 129), (64, 33, 64), (65, 65, 65), (200, 300, 100)])
def test_grad_sizes(m, n, k, tb, layout):
    run_grad(m, n, k, "f16", "f32", tb, "silu", layout, seed=m + n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_grad_types(act, t, out):
    run_grad(130, 72, 64, t, out, False, act, infinite=act not in ("none", "relu"), seed=3)
    run_grad(40, 136, 72, t, out, True, act, made=False, dbias=False, alpha=0.25, seed=4)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("m,n,k", [(900, 1800, 130), (2100, 4400, 72)])
def test_grad_large_tiles(m, n, k, tb, t):
    """128- and 256-wide tiles, whole ones and edges."""
    run_grad(m, n, k, t, t, tb, "silu", seed=5)


@pytest.mark.parametrize("m", [0, 7])
def test_grad_without_rows_or_a_product(m):
    """No rows: dbias = 0.  k = 0: E = 0, so that dG, dU and dbias are 0 and H is formed all the same."""
    n = 24
    dbias = torch.full((2 * n,), ref.SENTINEL, device="cuda")
    G, U, H = (ref.matrix(rng(i), max(m, 1), n, "bf16", extra=0) for i in range(3))
    kept = torch.stack([G, U])
    D = torch.full((2, max(m, 1), n), ref.SENTINEL, device="cuda", dtype=torch.bfloat16)
    size = mp.mpgemm_gated_grad_workspace_size(1, m, n)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    step = kept.stride(0)
    grad = mp.GatedGrad(act="silu", kept=kept, ld_kept=n, stride_kept=step, H=H, ldh=n, dbias=dbias)
    mp.mpgemm_run_gated_grad(handle().h, False, m, n, 0, 1.0, None, "bf16", 8, None, "bf16", n, grad, D, "bf16", n, step, ws, size)
    torch.cuda.synchronize()
    assert bool((dbias == 0).all())
    if m:
        assert bool((D == 0).all())
        gref.check(H, *gref.grad64(torch.zeros(m, n, dtype=torch.float64), torch.zeros(m, n, dtype=torch.float64), G, U, "silu")[2],
                   "bf16", "H")


def test_gradient_of_differences():
    """The gradient against differences of the formula: sum of D * R, moved by one entry of G or U."""
    g, m, n, k = rng(11), 6, 16, 24
    A, W = (torch.randn(m, k, generator=g, dtype=torch.float64), torch.randn(k, n, generator=g, dtype=torch.float64))
    G, U = (torch.randn(m, n, generator=g, dtype=torch.float64) for _ in range(2))
    to = lambda x: x.to(torch.float16)                    # noqa: E731
    A, W, G, U = (to(x) for x in (A, W, G, U))
    E = A.double() @ W.double()

    def total(gv, uv):
        return float((ref.act64("gelu_tanh", gv)[0] * uv * E).sum())
    kept = torch.stack([G, U]).cuda()
    D = torch.empty(2, m, n, device="cuda")
    grad = mp.GatedGrad(act="gelu_tanh", kept=kept, ld_kept=n, stride_kept=m * n)
    mp.mpgemm_run_gated_grad(handle().h, False, m, n, k, 1.0, A.cuda(), "f16", k, W.cuda(), "f16", n, grad, D, "f32", n, m * n, None, 0)
    torch.cuda.synchronize()
    h = 1e-4
    for half, i, j in [(0, 0, 0), (0, 3, 7), (0, 5, 15), (1, 0, 1), (1, 4, 4), (1, 5, 15)]:
        d = torch.zeros(m, n, dtype=torch.float64)
        d[i, j] = h
        up, down = [total(G.double() + s * d * (half == 0), U.double() + s * d * (half == 1)) for s in (1, -1)]
        want = (up - down) / (2 * h)
        # the differences' own error is of order h^2 times the third derivative (below 10) times |E U|
        assert abs(float(D[half, i, j]) - want) <= 1e-5 * (1 + abs(float(E[i, j] * U[i, j].double())) + abs(want))


def test_a_graph_of_forward_and_backward():
    """Captured once, replayed on new inputs between eager work: the same bits as eager calls."""
    g, m, n, k, t = rng(5), 300, 264, 192, "bf16"
    X, W, V = (ref.matrix(g, *s, t, 0.1, extra=0) for s in ((m, k), (2 * n, k), (n, k)))
    keep, d, dd = (torch.zeros(m, c, dtype=torch.bfloat16, device="cuda") for c in (2 * n, n, 2 * n))
    sums = torch.zeros(2 * n, device="cuda")
    size = mp.mpgemm_gated_grad_workspace_size(1, m, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step():
        mp.mpgemm_run_gated(handle().h, True, m, n, k, 1.0, X, t, k, W, t, k, n * k,
                            mp.Gated(act="silu", kept=keep, ld_kept=2 * n, stride_kept=n), d, t, n)
        mp.mpgemm_run_gated_grad(handle().h, True, m, n, k, 1.0, X, t, k, V, t, k,
                                 mp.GatedGrad(act="silu", kept=keep, ld_kept=2 * n, stride_kept=n, dbias=sums), dd, t, 2 * n, n,
                                 ws, size)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        X.copy_(ref.matrix(rng(20 + seed), m, k, t, extra=0))
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (keep, d, dd, sums)]
        for x in (keep, d, dd, sums):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, w in zip((keep, d, dd, sums), want):
            assert torch.equal(x, w)
