"""The products of language models in every kernel, against the same in 64 bits: sizes that the rules give to
64-, 128- and 256-wide tiles, whole tiles and edges, with outputs whose rows are whole lines and not, and to
each shape of the few rows' kernel.
What lies past the operands' rows is NaN, what lies past the outputs' must stay, and a second call gives
the same bits."""
import math

import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import ops_reference as ref, ops_tile_cases as cases
from tests.gpu_harness import handle, say
from tests.test_gpu_ops import (DIVISIONS, experts, experts_of, operands, rng, run_ce, run_epilogue, run_grad, run_grouped,
                                run_grouped_grad)

pytestmark = pytest.mark.gpu


def name_of(c):
    return "-".join(str(v) for v in c.values())


def output(rows, cols, t, pitch):
    """(buffer, view) with rows of whole 128-byte lines, or of 16-byte blocks that are none."""
    size = torch.empty(0, dtype=ref.TYPES[t]).element_size()
    line, block = 128 // size, 16 // size
    ld = -(-cols // line) * line
    if pitch == "odd":
        ld += block
    buf = torch.full((rows + 2, ld), ref.SENTINEL, dtype=ref.TYPES[t], device="cuda")
    assert (buf.stride(0) * size % 128 == 0) == (pitch == "lines") and buf.data_ptr() % 128 == 0
    return buf, buf[:rows, :cols]


def twice(call, outputs):
    """Queues the call; then again, which must not change a bit."""
    call()
    torch.cuda.synchronize()
    first = [v.clone() for v in outputs]
    call()
    torch.cuda.synchronize()
    for a, b in zip(first, outputs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("c", cases.FORWARD, ids=name_of)
def test_forward(c):
    m, n, k, t, out, ta, tb, act = (c[x] for x in ("m", "n", "k", "t", "out", "ta", "tb", "act"))
    say(f"[gpu ops] tiles {c}")
    g = rng(m + k)
    A, B, a, b = operands(g, m, n, k, t, ta, tb)
    bias = None if c["bias"] is None else torch.randn(n, generator=g).to(ref.TYPES[c["bias"]]).cuda()
    C = ref.matrix(g, m, n, c["c"]) if c["beta"] else None
    dbuf, D = output(m, n, out, c["pitch"])
    zbuf, Z = output(m, n, t, c["pitch"]) if c["aux"] else (None, None)
    epi = mp.Epilogue(act=act, bias=bias, bias_type=c["bias"] or "f32", aux=Z, ld_aux=Z.stride(0) if c["aux"] else 0)

    def call():
        src = C
        if c["in_place"]:
            D.copy_(C)
            src = D
        mp.mpgemm_run_epilogue(handle().h, ta, tb, m, n, k, 1.0, A, t, A.stride(0), B, t, B.stride(0), epi, c["beta"], src,
                               c["c"] or out, src.stride(0) if c["beta"] else 8, D, out, D.stride(0))

    twice(call, [v for v in (dbuf, zbuf) if v is not None])
    z, z_err = ref.product64(a, b, k)
    d, err, z, z_err = ref.forward64(z, z_err, act, bias, c["beta"], C)
    ref.assert_within(D, d, err + ref.rounding(d.abs() + err, out), "D")
    assert ref.untouched(dbuf, m, n)
    if c["aux"]:
        ref.assert_within(Z, z, z_err + ref.rounding(z.abs() + z_err, t), "Z")
        assert ref.untouched(zbuf, m, n)


@pytest.mark.parametrize("c", cases.SLOPE, ids=name_of)
def test_slope(c):
    m, n, k, t, out, ta, tb, act = (c[x] for x in ("m", "n", "k", "t", "out", "ta", "tb", "act"))
    say(f"[gpu ops] tiles {c}")
    g = rng(m + k)
    A, B, a, b = operands(g, m, n, k, t, ta, tb)
    Z = ref.matrix(g, m, n, t, 2.0)
    dbuf, D = output(m, n, out, c["pitch"])
    db = torch.full((n + 8,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_epilogue_grad_workspace_size(1, m, n) if c["dbias"] else 0
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")

    def call():
        mp.mpgemm_run_epilogue_grad(handle().h, ta, tb, m, n, k, 1.0, A, t, A.stride(0), B, t, B.stride(0), act, Z, Z.stride(0), D,
                                    out, D.stride(0), db if c["dbias"] else None, ws if c["dbias"] else None, size)

    twice(call, [dbuf, db])
    z, z_err = ref.product64(a, b, k)
    d, err = ref.slope64(z, z_err, act, Z)
    ref.assert_within(D, d, err + ref.rounding(d.abs() + err, out), "dZ")
    assert ref.untouched(dbuf, m, n) and bool((ws[size:] == 0xFF).all()) and bool((db[n:] == ref.SENTINEL).all())
    if c["dbias"]:
        s, s_err = ref.column_sums64(d, err)
        ref.assert_within(db[:n], s, s_err, "dbias")


@pytest.mark.parametrize("c", cases.GROUPED, ids=name_of)
def test_grouped(c):
    rows, groups, n, k, t, out, tb, act = (c[x] for x in ("rows", "groups", "n", "k", "t", "out", "tb", "act"))
    say(f"[gpu ops] tiles {c}")
    g = rng(rows + k)
    off = DIVISIONS[c["division"]](rows, groups)
    A = ref.matrix(g, rows, k, t)
    B, ldb, stride = experts(g, groups, n, k, t, tb)
    bias = torch.randn(groups, n, generator=g).to(ref.TYPES[t]).cuda() if c["bias"] else None
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = output(rows, n, out, c["pitch"])
    zbuf, Z = output(rows, n, t, c["pitch"]) if c["aux"] else (None, None)
    epi = mp.Epilogue(act=act, bias=bias, bias_type=t, aux=Z, ld_aux=Z.stride(0) if c["aux"] else 0, bias_stride=n)

    def call():
        mp.mpgemm_run_grouped(handle().h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, epi, D, out,
                              D.stride(0))

    twice(call, [v for v in (dbuf, zbuf) if v is not None])
    e = experts_of(rows, off)
    for i in range(groups):
        r = e == i
        if not bool(r.any()):
            continue
        z, z_err = ref.product64(A[r.cuda()], B[i, :n, :k].t() if tb else B[i, :k, :n], k)
        d, err, z, z_err = ref.forward64(z, z_err, act, bias[i] if c["bias"] else None)
        ref.assert_within(D[r.cuda()], d, err + ref.rounding(d.abs() + err, out), f"D of expert {i}")
        if c["aux"]:
            ref.assert_within(Z[r.cuda()], z, z_err + ref.rounding(z.abs() + z_err, t), f"Z of expert {i}")
    assert bool((D[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(dbuf, rows, n)
    if c["aux"]:
        assert bool((Z[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(zbuf, rows, n)


@pytest.mark.parametrize("c", cases.GROUPED_GRAD, ids=name_of)
def test_grouped_grad(c):
    rows, groups, n, k, t, out, tb, act = (c[x] for x in ("rows", "groups", "n", "k", "t", "out", "tb", "act"))
    say(f"[gpu ops] tiles grad {c}")
    g = rng(rows + k)
    off = DIVISIONS[c["division"]](rows, groups)
    A = ref.matrix(g, rows, k, t)
    B, ldb, stride = experts(g, groups, n, k, t, tb)
    Z = ref.matrix(g, rows, n, t, 2.0)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = output(rows, n, out, c["pitch"])
    db = torch.full((groups, n), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_epilogue_grad_workspace_size(groups, rows, n)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")

    def call():
        mp.mpgemm_run_grouped_grad(handle().h, tb, groups, rows, n, k, 1.0, A, t, A.stride(0), offsets, B, t, ldb, stride, act, Z,
                                   Z.stride(0), D, out, D.stride(0), db, ws, size)

    twice(call, [dbuf, db])
    e = experts_of(rows, off)
    for i in range(groups):
        r = e == i
        z, z_err = ref.product64(A[r.cuda()], B[i, :n, :k].t() if tb else B[i, :k, :n], k)
        d, err = ref.slope64(z, z_err, act, Z[r.cuda()])
        ref.assert_within(D[r.cuda()], d, err + ref.rounding(d.abs() + err, out), f"dZ of expert {i}")
        s, s_err = ref.column_sums64(d, err)
        ref.assert_within(db[i], s, s_err, f"dbias of expert {i}")
    assert bool((D[(e < 0).cuda()] == ref.SENTINEL).all()) and ref.untouched(dbuf, rows, n) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("c", cases.WGRAD, ids=name_of)
def test_grouped_wgrad(c):
    groups, rows, m, n, t, out, beta = (c[x] for x in ("groups", "rows", "m", "n", "t", "out", "beta"))
    say(f"[gpu ops] tiles wgrad {c}")
    g = rng(rows + m)
    off = DIVISIONS[c["division"]](rows, groups)
    A, X = ref.matrix(g, rows, m, t), ref.matrix(g, rows, n, t)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    dbuf, D = output(groups * m, n, out, c["pitch"])
    old = torch.randn(groups * m, n, generator=g).to(ref.TYPES[out]).cuda()

    def call():
        if beta:
            D.copy_(old)
        mp.mpgemm_run_grouped_wgrad(handle().h, groups, rows, m, n, 2.0, A, t, A.stride(0), X, t, X.stride(0), offsets, beta, D, out,
                                    D.stride(0), m * D.stride(0))

    twice(call, [dbuf])
    for i in range(groups):
        r = slice(off[i], off[i + 1])
        z, z_err = ref.product64(A[r].t(), X[r], off[i + 1] - off[i], 2.0)
        d, err, _, _ = ref.forward64(z, z_err, "none", None, beta, old[i * m:(i + 1) * m])
        ref.assert_within(D[i * m:(i + 1) * m], d, err + ref.rounding(d.abs() + err, out), f"dV of expert {i}")
    assert ref.untouched(dbuf, groups * m, n)


@pytest.mark.parametrize("c", cases.CE, ids=name_of)
def test_cross_entropy(c):
    m, n, k, t = (c[x] for x in ("m", "n", "k", "t"))
    say(f"[gpu ops] tiles cross entropy {c}")
    g = rng(m + n)
    X, W = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, 2.0 * k ** -0.5)
    target = torch.randint(0, n, (m,), generator=g)
    target[0], target[-1] = 0, n - 1
    grad = torch.randn(m, generator=g) / m
    if c["ignored"] == "some":
        target[1::3], grad[1::3] = -100, float("nan")
    target, grad = target.cuda(), grad.cuda()
    loss, lse = torch.full((m + 4,), ref.SENTINEL, device="cuda"), torch.full((m + 4,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, c["train"])
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    twice(lambda: mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, loss, lse, ws, size),
          [loss, lse])
    want, want_lse, err, lse_err, _, _ = ref.cross_entropy64(X, W, target, 1.0, k)
    ref.assert_within(loss[:m], want, err, "loss")
    ref.assert_within(lse[:m], want_lse, lse_err, "lse")
    assert bool((loss[m:] == ref.SENTINEL).all()) and bool((lse[m:] == ref.SENTINEL).all())
    if not c["train"]:
        return
    xbuf, dX = output(m, k, t, "lines")
    wbuf, dW = output(n, k, t, "lines")
    twice(lambda: mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X, t, X.stride(0), W, W.stride(0), target, lse, grad, dX,
                                               dX.stride(0), dW, dW.stride(0), ws, size), [xbuf, wbuf])
    dx, dx_err, dw, dw_err = ref.cross_entropy_grad64(X, W, target, grad, 1.0, k, t)
    ref.assert_within(dX, dx, dx_err, "dX")
    ref.assert_within(dW, dw, dw_err, "dW")
    assert ref.untouched(xbuf, m, k) and ref.untouched(wbuf, n, k) and bool((ws[size:] == 0xFF).all())


@pytest.mark.parametrize("c", cases.PIECES, ids=name_of)
def test_cross_entropy_in_pieces_without_rounding(c):
    """X and W are small integers in columns of their own, so that every logit is 0 and P is 2^-15, or 2^-15 - 1,
    which 16 bits hold as -1; every sum is exact in FP32 (units of 2^-15, below 2^24 of them), over the pieces too."""
    m, n, k, t = (c[x] for x in ("m", "n", "k", "t"))
    say(f"[gpu ops] tiles pieces {c}")
    dt, g = ref.TYPES[t], torch.Generator("cuda").manual_seed(k)
    X, W = torch.zeros(m, k, dtype=dt, device="cuda"), torch.zeros(n, k, dtype=dt, device="cuda")
    X[:, :k // 2] = torch.randint(-3, 4, (m, k // 2), generator=g, device="cuda").to(dt)
    W[:, k // 2:] = torch.randint(-3, 4, (n, k - k // 2), generator=g, device="cuda").to(dt)
    target = torch.randint(0, n, (m,), generator=g, device="cuda")
    target[1::10] = -100
    counts = target >= 0
    grad = torch.where(counts, torch.full((m,), 0.5, device="cuda"), torch.full((m,), float("nan"), device="cuda"))
    loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, X, t, k, W, k, target, loss, lse, ws, size)
    dX, dW = torch.full_like(X, ref.SENTINEL), torch.full_like(W, ref.SENTINEL)
    twice(lambda: mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X, t, k, W, k, target, lse, grad, dX, k, dW, k, ws, size),
          [dX, dW])
    # exponentials of 0 are exact, their sum is; the logarithm and its product with log 2 are off by a unit each
    assert float((lse.double() - 15 * math.log(2)).abs().max()) <= 2.0 ** -19
    p = torch.full((m, n), 2.0 ** -15, device="cuda")
    p[torch.arange(m, device="cuda")[counts], target[counts]] = -1
    p[~counts] = 0
    p = p.double()
    assert torch.equal(dX, (0.5 * (p @ W.double())).to(dt))
    assert torch.equal(dW, (0.5 * (p.t().contiguous() @ X.double())).to(dt))


@pytest.mark.parametrize("m", [3, 200])
def test_cross_entropy_of_no_features(m):
    """k = 0: every logit is 0; X and W may be missing, and there are no gradients to write."""
    n = 77
    target = torch.randint(0, n, (m,), generator=rng(m)).cuda()
    target[1] = -100
    loss, lse = torch.full((m + 4,), ref.SENTINEL, device="cuda"), torch.full((m + 4,), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_linear_ce_workspace_size(m, n, 0, "f16", True)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, 0, 1.0, None, "f16", 8, None, 8, target, loss, lse, ws, size)
    mp.mpgemm_run_linear_ce_grad(handle().h, m, n, 0, 1.0, None, "f16", 8, None, 8, target, lse, loss, lse, 8, lse, 8, ws, size)
    torch.cuda.synchronize()
    want = torch.full((m,), math.log(n), dtype=torch.float64)
    ref.assert_within(lse[:m], want, 2.0 ** -18 + 0 * want, "lse")
    want[1] = 0
    ref.assert_within(loss[:m], want, torch.where(want == 0, 0 * want, 2.0 ** -18 + 0 * want), "loss")
    assert bool((loss[m:] == ref.SENTINEL).all()) and bool((lse[m:] == ref.SENTINEL).all())


@pytest.mark.parametrize("ta", [False, True])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("c", cases.FEW, ids=name_of)
def test_few_rows(c, t, out, ta):
    m, n, k, tb = (c[x] for x in ("m", "n", "k", "tb"))
    run_epilogue(m, n, k, t, out, ta, tb, "gelu", bias=t, aux=True, beta=0.5, seed=m)
    run_grad(m, n, k, t, out, ta, tb, "silu", seed=n)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("c", [c for c in cases.FEW if c["tb"]], ids=name_of)
def test_cross_entropy_of_few_rows(c, t):
    run_ce(c["m"], c["n"], c["k"], t, seed=c["n"])


@pytest.mark.parametrize("division", ["even", "gaps"])
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("c", cases.FEW_OF_EXPERTS, ids=name_of)
def test_few_rows_of_experts(c, t, out, division):
    rows, groups, n, k, tb = (c[x] for x in ("m", "groups", "n", "k", "tb"))
    run_grouped(rows, groups, n, k, t, out, tb, "silu", division, seed=rows)
    run_grouped_grad(rows, groups, n, k, t, out, tb, "silu", division, seed=rows + 1)
