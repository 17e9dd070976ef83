"""The products of language models on the GPU -- the epilogue product, the grouped products and the
cross entropy of a linear layer, with their gradients -- against the same in 64 bits, at the sizes
where tiles, blocks and stages end; what lies past the operands' rows is NaN, and what lies past
the outputs' must stay as it was."""
import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def rng(seed):
    return torch.Generator().manual_seed(seed)


def operands(gen, m, n, k, t, ta, tb, scale=1.0):
    A = ref.matrix(gen, k, m, t) if ta else ref.matrix(gen, m, k, t)
    s = scale * max(k, 1) ** -0.5
    B = ref.matrix(gen, n, k, t, s) if tb else ref.matrix(gen, k, n, t, s)
    return A, B, (A.t() if ta else A), (B.t() if tb else B)


# ----------------------------------------------------------------------------- epilogue
def run_epilogue(m, n, k, t, out, ta, tb, act, bias=None, aux=False, beta=0.0, c_type=None, alpha=1.0, seed=0, scale=1.0):
    say(f"[gpu ops] epilogue {m}x{n}x{k} {t}->{out} ta={ta} tb={tb} {act} bias={bias} aux={aux} beta={beta} c={c_type}")
    g = rng(seed)
    A, B, a, b = operands(g, m, n, k, t, ta, tb, scale)
    bv = None if bias is None else torch.randn(n, generator=g).to(ref.TYPES[bias]).cuda()
    C = ref.matrix(g, m, n, c_type or out) if beta else None
    dbuf, D = ref.output(m, n, out)
    zbuf, Z = ref.output(m, n, t, extra=16) if aux else (None, None)
    epi = mp.Epilogue(act=act, bias=bv, bias_type=bias or "f32", aux=Z, ld_aux=Z.stride(0) if aux else 0)
    mp.mpgemm_run_epilogue(handle().h, ta, tb, m, n, k, alpha, A, t, A.stride(0), B, t, B.stride(0), epi, beta, C,
                           c_type or out, C.stride(0) if beta else 8, D, out, D.stride(0))
    torch.cuda.synchronize()
    z, z_err = ref.product64(a, b, k, alpha)
    d, err, z, z_err = ref.forward64(z, z_err, act, bv, beta, C)
    ref.assert_within(D, d, err + ref.rounding(d.abs() + err, out), "D")
    assert ref.untouched(dbuf, m, n)
    if aux:
        ref.assert_within(Z, z, z_err + ref.rounding(z.abs() + z_err, t), "Z")
        assert ref.untouched(zbuf, m, n)


@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", [(1, 256, 64), (1, 5, 1), (2, 17, 129), (15, 33, 71), (16, 16, 32), (17, 40, 1001),
                                   (33, 97, 130), (64, 64, 1024), (65, 7, 63), (100, 130, 200), (129, 257, 65),
                                   (300, 520, 136)])
def test_epilogue_sizes(m, n, k, ta, tb):
    t, out = ("bf16", "f32") if (m + n) % 2 else ("f16", "f16")
    run_epilogue(m, n, k, t, out, ta, tb, "gelu", bias=t, aux=True, beta=0.5, seed=m * n + k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("m", [3, 200])
def test_epilogue_types(act, t, out, m):
    run_epilogue(m, 200, 96, t, out, False, True, act, bias="f32", aux=True, seed=m, scale=3.0)
    run_epilogue(m, 72, 96, t, out, False, False, act, beta=-1.0, c_type="f32", alpha=0.5, seed=m + 1)
    run_epilogue(m, 72, 96, t, out, True, False, act, bias=t, beta=1.0, c_type=t, seed=m + 2)


@pytest.mark.parametrize("m,n,k", [(700, 2100, 64), (2600, 2500, 72)])
def test_epilogue_large_tiles(m, n, k):
    """128- and 256-wide tiles, whole ones and edges."""
    run_epilogue(m, n, k, "bf16", "bf16", False, True, "silu", bias="bf16", aux=True, beta=1.0, seed=5)
    run_epilogue(m, n, k, "f16", "f32", True, False, "gelu_tanh", bias="f16", seed=6)


@pytest.mark.parametrize("m", [4, 150])
def test_epilogue_without_a_product(m):
    """k = 0: Z is the bias; A and B may be missing."""
    n, bias = 41, torch.randn(41, generator=rng(3)).cuda()
    dbuf, D = ref.output(m, n, "f32")
    C = ref.matrix(rng(4), m, n, "f32")
    mp.mpgemm_run_epilogue(handle().h, False, False, m, n, 0, 1.0, None, "f16", 8, None, "f16", 48,
                           mp.Epilogue(act="relu", bias=bias), 2.0, C, "f32", C.stride(0), D, "f32", D.stride(0))
    torch.cuda.synchronize()
    want = bias.double().cpu().clamp(min=0) + 2 * C.double().cpu()
    ref.assert_within(D, want, 2.0 ** -22 * (want.abs() + 4 * C.double().cpu().abs()) + 0 * want, "D")
    assert ref.untouched(dbuf, m, n)


@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("m", [3, 100])
def test_gelu_keeps_its_tail(m, t, out):
    """GELU over -13 .. 13, where |z| Phi(-|z|) falls to 1e-37: relative to the value.  exp(-z^2 / 2) takes an argument
    of up to 124 in units of log 2, off by two roundings (2 * 2^-24 * 124, times log 2: 2^-16.6); the short form for
    16-bit values is within 6.5e-6 (2^-17.2); 2^-16 covers both and the roundings after them."""
    say(f"[gpu ops] gelu's tail {t}->{out} {m} rows")
    z = torch.cat([torch.linspace(-13, -5.5, 700), torch.linspace(-5.5, 13, 300), torch.tensor([-6.0, -6.0000005, -5.9999995])])
    z = z[torch.randperm(z.numel(), generator=rng(7))]
    n = z.numel()
    dbuf, D = ref.output(m, n, out)
    mp.mpgemm_run_epilogue(handle().h, False, False, m, n, 0, 1.0, None, t, 8, None, t, 1008, mp.Epilogue(act="gelu", bias=z.cuda()),
                           0.0, None, out, 1008, D, out, D.stride(0))
    torch.cuda.synchronize()
    x = z.double()
    want = (x * 0.5 * torch.erfc(-x * 2 ** -0.5)).expand(m, n)
    ref.assert_within(D, want, 2.0 ** -16 * want.abs() + ref.rounding(want, out), "D")
    assert ref.untouched(dbuf, m, n)


@pytest.mark.parametrize("m", [5, 90])
def test_epilogue_in_place_and_nonfinite(m):
    """D == C; infinities and NaN reach exactly the outputs they belong to."""
    g, n, k = rng(8), 48, 72
    A, B, a, b = operands(g, m, n, k, "bf16", False, True)
    A[1, 3] = float("inf")
    A[2, 5] = float("nan")
    D = ref.matrix(g, m, n, "f32")
    C = D.clone()
    mp.mpgemm_run_epilogue(handle().h, False, True, m, n, k, 1.0, A, "bf16", A.stride(0), B, "bf16", B.stride(0),
                           mp.Epilogue(act="silu"), 1.0, D, "f32", D.stride(0), D, "f32", D.stride(0))
    torch.cuda.synchronize()
    z, z_err = ref.product64(a, b, k)
    d, err, _, _ = ref.forward64(z, z_err, "silu", None, 1.0, C)
    good = [r for r in range(m) if r not in (1, 2)]
    ref.assert_within(D[good], d[good], (err + ref.rounding(d, "f32"))[good], "D")
    assert bool(D[2].isnan().all())
    row = D[1].cpu()
    plus = z[1] > 0
    assert bool((row[plus] == float("inf")).all()) and bool(row[~plus].isnan().all())


# ----------------------------------------------------------------------------- its gradient
def run_grad(m, n, k, t, out, ta, tb, act, dbias=True, alpha=1.0, seed=0, spread=2.0):
    say(f"[gpu ops] epilogue_grad {m}x{n}x{k} {t}->{out} ta={ta} tb={tb} {act}")
    g = rng(seed)
    A, B, a, b = operands(g, m, n, k, t, ta, tb)
    Z = ref.matrix(g, m, n, t, spread)
    if m > 1 and n > 2:
        Z[0, 0], Z[1, 1], Z[0, 2] = float("inf"), float("-inf"), 0.0
    dbuf, D = ref.output(m, n, out)
    bbuf = torch.full((n + 8,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_epilogue_grad_workspace_size(1, m, n) if dbias else 0
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_epilogue_grad(handle().h, ta, tb, m, n, k, alpha, A, t, A.stride(0), B, t, B.stride(0), act, Z,
                                Z.stride(0), D, out, D.stride(0), bbuf if dbias else None, ws if dbias else None, size)
    torch.cuda.synchronize()
    z, z_err = ref.product64(a, b, k, alpha)
    d, err = ref.slope64(z, z_err, act, Z)
    ref.assert_within(D, d, err + ref.rounding(d.abs() + err, out), "dZ")
    assert ref.untouched(dbuf, m, n)
    if dbias:
        s, s_err = ref.column_sums64(d, err)
        ref.assert_within(bbuf[:n], s, s_err, "dbias")
        assert bool((bbuf[n:] == ref.SENTINEL).all()) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", [(1, 9, 40), (16, 64, 64), (31, 100, 129), (64, 33, 64), (65, 65, 65), (200, 300, 100)])
def test_epilogue_grad_sizes(m, n, k, ta, tb):
    run_grad(m, n, k, "f16", "f32", ta, tb, "silu", seed=m + n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("m", [20, 260])
def test_epilogue_grad_types(act, t, out, m):
    run_grad(m, 136, 80, t, out, False, True, act, alpha=0.25, seed=m)
    run_grad(m, 136, 80, t, out, False, False, act, dbias=False, seed=m)


@pytest.mark.parametrize("m,n", [(700, 2100), (2600, 2500)])
def test_epilogue_grad_large_tiles(m, n):
    run_grad(m, n, 64, "bf16", "bf16", False, False, "gelu", seed=9)


def test_epilogue_grad_of_no_rows():
    b = torch.full((20,), 3.0, device="cuda")
    mp.mpgemm_run_epilogue_grad(handle().h, False, True, 0, 20, 8, 1.0, None, "f16", 8, None, "f16", 8, "silu", None, 24,
                                None, "f32", 24, b, None, 0)
    torch.cuda.synchronize()
    assert bool((b == 0).all())


@pytest.mark.parametrize("act", ACTS[2:])
def test_slopes_are_the_activations_differences(act):
    """The gradient's slope against differences of the forward product's own values: with a 1 x 1 product
    of ones, D of the forward pass is act(bias) and D of the gradient act'(Z)."""
    z = torch.linspace(-4, 4, 161)[:, None].half().float()
    h = 2.0 ** -7
    n, one = z.numel(), ref.matrix(rng(0), 1, 1, "f16")
    one.fill_(1.0)
    zero = torch.zeros_like(one.expand(1, 1)).repeat(n, 8)

    def forward(x):
        D = torch.empty(1, 168, device="cuda")
        mp.mpgemm_run_epilogue(handle().h, False, True, 1, n, 1, 1.0, one, "f16", one.stride(0), zero, "f16", 8,
                               mp.Epilogue(act=act, bias=x[:, 0].cuda().contiguous()), 0.0, None, "f32", 168, D, "f32", 168)
        return D[0, :n].double().cpu()

    ones = torch.ones(n, 8, dtype=torch.float16, device="cuda")
    Z = torch.zeros(1, 168, dtype=torch.float16, device="cuda")
    Z[0, :n] = z[:, 0].half()
    D = torch.empty(1, 168, device="cuda")
    mp.mpgemm_run_epilogue_grad(handle().h, False, True, 1, n, 1, 1.0, one, "f16", one.stride(0), ones, "f16", 8, act, Z, 168,
                                D, "f32", 168, None, None, 0)
    diff = (forward(z + h) - forward(z - h)) / (2 * h)
    # central differences: h^2 / 6 of the third derivative (below 2.5), and the values' 2^-17 over h
    assert float((D[0, :n].double().cpu() - diff).abs().max()) <= 2.5 * h * h / 6 + 2 * 4 * 2.0 ** -17 / (2 * h)


# ----------------------------------------------------------------------------- grouped
DIVISIONS = {
    "even": lambda rows, groups: [rows * e // groups for e in range(groups + 1)],
    "one has all": lambda rows, groups: [0] * (groups // 2 + 1) + [rows] * (groups - groups // 2),
    "single rows": lambda rows, groups: [min(e, rows) for e in range(groups)] + [rows],
    "gaps": lambda rows, groups: [min(rows, 1 + (rows * (e // 2 * 2)) // groups) for e in range(groups + 1)],
    "none": lambda rows, groups: [0] * (groups + 1),
}


def experts_of(rows, off):
    e = torch.full((rows,), -1)
    for i in range(len(off) - 1):
        e[off[i]:off[i + 1]] = i
    return e


def experts(gen, groups, n, k, t, tb):
    r, c = (n, k) if tb else (k, n)
    ld = -(-c // 8) * 8 + 8
    buf = torch.full((groups, r + 1, ld), float("nan"), dtype=ref.TYPES[t], device="cuda")
    buf[:, :r, :c] = (torch.randn(groups, r, c, generator=gen) * max(k, 1) ** -0.5).to(ref.TYPES[t]).cuda()
    return buf, ld, (r + 1) * ld


def run_grouped(rows, groups, n, k, t, out, tb, act, division, bias=True, aux=True, seed=0):
    off = DIVISIONS[division](rows, groups)
    say(f"[gpu ops] grouped rows={rows} groups={groups} n={n} k={k} {t}->{out} tb={tb} {act} {division}")
    g = rng(seed)
    A = ref.matrix(g, rows, k, t)
    B, ldb, stride = experts(g, groups, n, k, t, tb)
    bv = torch.randn(groups, n, generator=g).to(ref.TYPES[t]).cuda() if bias else None
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = ref.output(rows, n, out)
    zbuf, Z = ref.output(rows, n, t) if aux else (None, None)
    epi = mp.Epilogue(act=act, bias=bv, bias_type=t, aux=Z, ld_aux=Z.stride(0) if aux else 0, bias_stride=n)
    mp.mpgemm_run_grouped(handle().h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, epi, D, out,
                          D.stride(0))
    torch.cuda.synchronize()
    e = experts_of(rows, off)
    for i in range(groups):
        r = e == i
        if not bool(r.any()):
            continue
        b = B[i, :n, :k].t() if tb else B[i, :k, :n]
        z, z_err = ref.product64(A[r.cuda()], b, k)
        d, err, z, z_err = ref.forward64(z, z_err, act, bv[i] if bias else None)
        ref.assert_within(D[r.cuda()], d, err + ref.rounding(d.abs() + err, out), f"D of expert {i}")
        if aux:
            ref.assert_within(Z[r.cuda()], z, z_err + ref.rounding(z.abs() + z_err, t), f"Z of expert {i}")
    assert bool((D[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(dbuf, rows, n)
    if aux:
        assert bool((Z[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(zbuf, rows, n)


@pytest.mark.parametrize("division", sorted(DIVISIONS))
@pytest.mark.parametrize("rows,groups,n,k", [(1, 3, 40, 64), (8, 32, 130, 96), (70, 5, 33, 71), (200, 3, 72, 129),
                                             (500, 130, 24, 40), (900, 4, 200, 64), (1200, 2, 300, 40)])
def test_grouped_sizes(division, rows, groups, n, k):
    run_grouped(rows, groups, n, k, "bf16", "f32", True, "silu", division, seed=rows)
    run_grouped(rows, groups, n, k, "f16", "f16", False, "gelu", division, bias=False, aux=False, seed=rows + 1)


def run_grouped_grad(rows, groups, n, k, t, out, tb, act, division, seed=0):
    off = DIVISIONS[division](rows, groups)
    say(f"[gpu ops] grouped_grad rows={rows} groups={groups} n={n} k={k} {t}->{out} tb={tb} {act} {division}")
    g = rng(seed)
    A = ref.matrix(g, rows, k, t)
    B, ldb, stride = experts(g, groups, n, k, t, tb)
    Z = ref.matrix(g, rows, n, t)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = ref.output(rows, n, out)
    db = torch.full((groups, n), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_epilogue_grad_workspace_size(groups, rows, n)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_grouped_grad(handle().h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, act, Z,
                               Z.stride(0), D, out, D.stride(0), db, ws, size)
    torch.cuda.synchronize()
    e = experts_of(rows, off)
    for i in range(groups):
        r = e == i
        b = B[i, :n, :k].t() if tb else B[i, :k, :n]
        z, z_err = ref.product64(A[r.cuda()], b, k)
        d, err = ref.slope64(z, z_err, act, Z[r.cuda()])
        ref.assert_within(D[r.cuda()], d, err + ref.rounding(d.abs() + err, out), f"dZ of expert {i}")
        s, s_err = ref.column_sums64(d, err)
        ref.assert_within(db[i], s, s_err, f"dbias of expert {i}")
    assert bool((D[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(dbuf, rows, n)
    assert bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("division", sorted(DIVISIONS))
@pytest.mark.parametrize("rows,groups,n,k", [(8, 32, 130, 96), (70, 5, 33, 71), (500, 130, 24, 40), (900, 4, 200, 64)])
def test_grouped_grad(division, rows, groups, n, k):
    run_grouped_grad(rows, groups, n, k, "bf16", "bf16", False, "silu", division, seed=rows)
    run_grouped_grad(rows, groups, n, k, "f16", "f32", True, "gelu_tanh", division, seed=rows)


@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("division", sorted(DIVISIONS))
@pytest.mark.parametrize("rows,groups,m,n,t,out", [(1, 2, 8, 8, "f16", "f32"), (70, 5, 33, 71, "bf16", "bf16"),
                                                   (300, 9, 130, 72, "f16", "f16"), (500, 70, 24, 40, "bf16", "f32"),
                                                   (700, 3, 1300, 1200, "bf16", "bf16")])
def test_grouped_wgrad(rows, groups, m, n, t, out, division, beta):
    off = DIVISIONS[division](rows, groups)
    say(f"[gpu ops] grouped_wgrad rows={rows} groups={groups} {m}x{n} {t}->{out} {division} beta={beta}")
    g = rng(rows + m)
    A, X = ref.matrix(g, rows, m, t), ref.matrix(g, rows, n, t)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = ref.output(groups * m, n, out)
    old = torch.randn(groups * m, n, generator=g).to(ref.TYPES[out])
    if beta:
        D.copy_(old)
    mp.mpgemm_run_grouped_wgrad(handle().h, groups, rows, m, n, 2.0, A, t, A.stride(0), X, t, X.stride(0), offsets, beta, D, out,
                                D.stride(0), m * D.stride(0))
    torch.cuda.synchronize()
    for i in range(groups):
        r = slice(off[i], off[i + 1])
        z, z_err = ref.product64(A[r].t(), X[r], off[i + 1] - off[i], 2.0)
        d, err, _, _ = ref.forward64(z, z_err, "none", None, beta, old[i * m:(i + 1) * m])
        ref.assert_within(D[i * m:(i + 1) * m], d, err + ref.rounding(d.abs() + err, out), f"dV of expert {i}")
    assert ref.untouched(dbuf, groups * m, n)


@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("rows,n,k", [(37, 72, 96), (300, 137, 200), (2100, 1503, 2008)])
def test_rows_of_one_expert_do_not_reach_another(rows, n, k, tb, t, out):
    """NaN in one expert's rows, and in rows of no expert: what belongs to the others is as without them."""
    say(f"[gpu ops] NaN rows of one expert, {rows}x{n}x{k} {t} tb={tb}")
    g, groups = rng(rows), 4
    off = [rows // 10, rows // 3, rows // 2 + 1, rows - 7, rows - 3]     # (rows before the first and after the last are no expert's)
    e = experts_of(rows, off)
    bad = ((e == 1) | (e < 0)).cuda()
    A, X, Z = ref.matrix(g, rows, k, t), ref.matrix(g, rows, n, t), ref.matrix(g, rows, n, t)
    A[bad], X[bad], Z[bad] = float("nan"), float("inf"), float("nan")
    B, ldb, stride = experts(g, groups, n, k, t, tb)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    h = handle().h
    dbuf, D = ref.output(rows, n, out)
    mp.mpgemm_run_grouped(h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, mp.Epilogue(act="silu"), D, out,
                          D.stride(0))
    gbuf, G = ref.output(rows, n, out)
    db = torch.full((groups, n), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_epilogue_grad_workspace_size(groups, rows, n)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_grouped_grad(h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, "gelu", Z, Z.stride(0), G,
                               out, G.stride(0), db, ws, size)
    vbuf, V = ref.output(groups * k, n, out)
    mp.mpgemm_run_grouped_wgrad(h, groups, rows, k, n, 1.0, A, t, A.stride(0), X, t, X.stride(0), offsets, 0.0, V, out, V.stride(0),
                                k * V.stride(0))
    torch.cuda.synchronize()
    for i in (0, 2, 3):
        r = (e == i).cuda()
        z, z_err = ref.product64(A[r], B[i, :n, :k].t() if tb else B[i, :k, :n], k)
        d, err, _, _ = ref.forward64(z, z_err, "silu")
        ref.assert_within(D[r], d, err + ref.rounding(d.abs() + err, out), f"D of expert {i}")
        d, err = ref.slope64(z, z_err, "gelu", Z[r])
        ref.assert_within(G[r], d, err + ref.rounding(d.abs() + err, out), f"dZ of expert {i}")
        s, s_err = ref.column_sums64(d, err)
        ref.assert_within(db[i], s, s_err, f"dbias of expert {i}")
        v, err = ref.product64(A[r].t(), X[r], int(r.sum()))
        ref.assert_within(V[i * k:(i + 1) * k], v, err + ref.rounding(v.abs() + err, out), f"dV of expert {i}")
    none = (e < 0).cuda()
    assert bool((D[none] == ref.SENTINEL).all()) and bool((G[none] == ref.SENTINEL).all())
    assert ref.untouched(dbuf, rows, n) and ref.untouched(gbuf, rows, n) and ref.untouched(vbuf, groups * k, n)


# ----------------------------------------------------------------------------- cross entropy
def run_ce(m, n, k, t, alpha=1.0, ignored="some", seed=0, scale=2.0, train=True, weight=1.0):
    say(f"[gpu ops] linear_ce {m}x{n}x{k} {t} alpha={alpha} ignored={ignored}")
    g = rng(seed)
    X, W = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, scale * max(k, 1) ** -0.5)
    target = torch.randint(0, n, (m,), generator=g)
    target[0], target[-1] = 0, n - 1
    if ignored == "some" and m > 2:
        target[1::3] = -100
        target[2::7] = n          # past the vocabulary: does not count either
    if ignored == "all":
        target[:] = -1
    target = target.cuda()
    grad = (torch.randn(m, generator=g) * weight / m).cuda()
    if ignored == "some" and m > 2:
        grad[1::3] = float("nan")  # of rows that do not count: must not matter
    loss, lse = torch.full((m + 4,), ref.SENTINEL, device="cuda"), torch.full((m + 4,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, train)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, k, alpha, X, t, X.stride(0), W, W.stride(0), target, loss, lse, ws, size)
    torch.cuda.synchronize()
    want, want_lse, err, lse_err, _, _ = ref.cross_entropy64(X, W, target, alpha, k)
    ref.assert_within(loss[:m], want, err, "loss")
    ref.assert_within(lse[:m], want_lse, lse_err, "lse")
    assert bool((loss[m:] == ref.SENTINEL).all()) and bool((lse[m:] == ref.SENTINEL).all())
    if not train:
        return
    xbuf, dX = ref.output(m, k, t)
    wbuf, dW = ref.output(n, k, t)
    mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, alpha, X, t, X.stride(0), W, W.stride(0), target, lse, grad, dX,
                                 dX.stride(0), dW, dW.stride(0), ws, size)
    torch.cuda.synchronize()
    dx, dx_err, dw, dw_err = ref.cross_entropy_grad64(X, W, target, grad, alpha, k, t)
    ref.assert_within(dX, dx, dx_err, "dX")
    ref.assert_within(dW, dw, dw_err, "dW")
    assert ref.untouched(xbuf, m, k) and ref.untouched(wbuf, n, k) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 8), (1, 300, 64), (3, 17, 9), (16, 257, 40), (50, 1000, 72), (64, 130, 33),
                                   (65, 70, 64), (130, 515, 100), (300, 700, 136)])
def test_linear_ce_sizes(t, m, n, k):
    run_ce(m, n, k, t, seed=m + n)


@pytest.mark.parametrize("ignored", ["none", "all"])
@pytest.mark.parametrize("m", [7, 140])
def test_linear_ce_counting_rows(m, ignored):
    run_ce(m, 90, 48, "f16", alpha=0.5, ignored=ignored, seed=m)


@pytest.mark.parametrize("ignored", ["none", "some", "all"])
@pytest.mark.parametrize("t,m", [("bf16", 511), ("bf16", 512), ("f16", 1100)])
def test_linear_ce_listed_rows(t, m, ignored):
    """From 512 rows on the gradient lists the rows that count."""
    run_ce(m, 300, 75, t, ignored=ignored, seed=m)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m", [3, 32, 64, 100, 128, 129, 300, 511, 512, 700])
def test_linear_ce_rows_that_do_not_count_may_hold_anything(t, m):
    """NaN and infinities in X and grad of rows that do not count: the gradients are those without them, and 0 there."""
    n, k = 190, 75
    say(f"[gpu ops] linear_ce ignored rows of NaN, {m} rows {t}")
    g = rng(m)
    X, W = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, k ** -0.5)
    target = torch.randint(0, n, (m,), generator=g)
    target[1::3], target[5::9] = -100, n
    out = ((target < 0) | (target >= n)).cuda()
    target = target.cuda()
    grad = torch.randn(m, generator=g).cuda()
    plain = X.clone()
    plain[out] = 0
    X[out, 0::2], X[out, 1::4], X[out, 3::4] = float("nan"), float("inf"), float("-inf")
    loss, lse = torch.full((m,), ref.SENTINEL, device="cuda"), torch.full((m,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, loss, lse, ws, size)
    torch.cuda.synchronize()
    want, want_lse, err, lse_err, _, _ = ref.cross_entropy64(plain, W, target, 1.0, k)
    ref.assert_within(loss, want, err, "loss")
    ref.assert_within(lse[~out], want_lse[~out.cpu()], lse_err[~out.cpu()], "lse")
    xbuf, dX = ref.output(m, k, t)
    wbuf, dW = ref.output(n, k, t)
    grad[out] = float("nan")
    mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, lse, grad, dX, dX.stride(0), dW,
                                 dW.stride(0), ws, size)
    torch.cuda.synchronize()
    dx, dx_err, dw, dw_err = ref.cross_entropy_grad64(plain, W, target, grad, 1.0, k, t)
    ref.assert_within(dX, dx, dx_err, "dX")
    ref.assert_within(dW, dw, dw_err, "dW")
    assert bool((dX[out] == 0).all())
    assert ref.untouched(xbuf, m, k) and ref.untouched(wbuf, n, k) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(2, 5, 3), (31, 700, 263), (32, 130, 520), (33, 65, 64), (64, 127, 257), (65, 1000, 40),
                                   (96, 64, 319), (127, 300, 1030), (128, 193, 72), (129, 193, 72)])
def test_linear_ce_few_rows(t, m, n, k):
    """The weights' gradient of at most 128 rows has a kernel of its own; the rows' gradient is summed in ranges."""
    run_ce(m, n, k, t, alpha=0.75, seed=m + n + k)


def test_linear_ce_few_rows_of_a_large_vocabulary():
    run_ce(40, 60000, 72, "bf16", seed=6)


def test_linear_ce_small_weights_and_large_logits():
    run_ce(100, 2000, 64, "f16", weight=1e-4, seed=1)     # gradients far below FP16's normal range
    run_ce(100, 2000, 64, "f16", weight=6e4, seed=2)
    run_ce(40, 600, 64, "bf16", alpha=10.0, seed=3)       # probabilities near 0 and 1
    run_ce(90, 600, 64, "f16", alpha=-10.0, seed=4)


def test_linear_ce_in_pieces():
    """More columns than a piece of the gradient holds (128 MiB of probabilities)."""
    m, n, k = 3000, 50000, 16
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, "bf16", True)
    assert size < 2 * m * n                                # the logits are not kept
    run_ce(m, n, k, "bf16", seed=5)


def test_linear_ce_gradient_against_differences():
    """The gradient of sum(grad * loss) along a direction against differences of the losses themselves."""
    m, n, k, t = 24, 120, 32, "f16"
    g = rng(11)
    X = torch.randn(m, k, generator=g).half()
    W = (torch.randn(n, k, generator=g) * 0.3).half()
    target = torch.randint(0, n, (m,), generator=g).cuda()
    weight = torch.rand(m, generator=g).cuda()
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")

    def total(x, w):
        mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, x.cuda(), t, k, w.cuda(), k, target, loss, lse, ws, size)
        return float((loss.double() * weight.double()).sum())

    dX, dW = torch.empty(m, k, dtype=torch.float16, device="cuda"), torch.empty(n, k, dtype=torch.float16, device="cuda")
    total(X, W)
    mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X.cuda(), t, k, W.cuda(), k, target, lse, weight, dX, k, dW, k, ws, size)
    for x_side in (True, False):
        at, grad = (X, dX) if x_side else (W, dW)
        step = (torch.randn(at.shape, generator=g) * 2.0 ** -5)
        plus, minus = (at.float() + step).half(), (at.float() - step).half()
        moved = (plus.double() - minus.double())
        diff = total(plus, W) - total(minus, W) if x_side else total(X, plus) - total(X, minus)
        want = float((grad.double().cpu() * moved).sum())
        # the midpoint moves by half an FP16 step and the third derivative is below 1 per unit: both are
        # a few 2^-10 of the gradient's terms; losses are within 2^-16 each
        slack = 2.0 ** -8 * float((grad.double().cpu().abs() * moved.abs()).sum()) + m * 2.0 ** -15
        assert abs(diff - want) <= slack, (diff, want, slack)


def test_linear_ce_gradients_one_at_a_time():
    m, n, k, t = 70, 300, 40, "bf16"
    g = rng(12)
    X, W = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, 0.3)
    target = torch.randint(0, n, (m,), generator=g).cuda()
    grad = torch.ones(m, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, loss, lse, ws, size)
    got = []
    for x, w in ((True, True), (True, False), (False, True)):
        dX, dW = torch.zeros(m, 40, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 40, dtype=torch.bfloat16, device="cuda")
        mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, lse, grad,
                                     dX if x else None, 40, dW if w else None, 40, ws, size)
        got.append((dX, dW))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[2][1])
    assert bool((got[1][1] == 0).all()) and bool((got[2][0] == 0).all())
    dW = torch.full((n, 40), 5.0, dtype=torch.bfloat16, device="cuda")
    mp.mpgemm_run_linear_ce_grad(handle().h, 0, n, k, 1.0, None, t, 40, None, 40, None, None, None, None, 40, dW, 40, None, 0)
    torch.cuda.synchronize()
    assert bool((dW == 0).all())                           # a sum over no rows
