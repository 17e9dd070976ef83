"""The distillation loss of a linear head on the GPU, and its gradients, against the same in 64 bits."""
import math

import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import distill_reference as dref
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu


def rng(seed):
    return torch.Generator().manual_seed(seed)


def call(x, w, t, index, logit, scale, lse_t, alpha, grads=None, dx=True, dw=True, ws=None):
    """(loss, lse, picked, dX, dW); outputs in buffers whose rest must stay as it was."""
    m, k, n, top = x.shape[0], x.shape[1], w.shape[0], index.shape[1]
    ld = index.stride(0)
    loss, lse = (torch.full((m + 1,), ref.SENTINEL, device="cuda") for _ in range(2))
    picked = torch.full((m + 1, ld), ref.SENTINEL, device="cuda")
    train = grads is not None
    size = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, t, train)
    if ws is None:
        ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    teacher = mp.Teacher(top, index, logit, ld, scale=scale, lse=lse_t)
    h = handle().h
    mp.mpgemm_run_linear_distill(h, m, n, k, alpha, x, t, x.stride(0), w, w.stride(0), teacher, loss, lse, picked, ws, size)
    out = [loss, lse, picked]
    if train:
        xbuf, dX = ref.output(m, k, t)
        wbuf, dW = ref.output(n, k, t)
        mp.mpgemm_run_linear_distill_grad(h, m, n, k, alpha, x, t, x.stride(0), w, w.stride(0), teacher, lse, picked, grads,
                                          dX if dx else None, dX.stride(0), dW if dw else None, dW.stride(0), ws, size)
        out += [dX, dW]
    torch.cuda.synchronize()
    assert float(loss[m]) == ref.SENTINEL and float(lse[m]) == ref.SENTINEL
    assert bool((picked[m] == ref.SENTINEL).all()) and bool((picked[:, top:] == ref.SENTINEL).all())
    assert bool((ws[size:] == 0xFF).all())
    if train:
        assert ref.untouched(xbuf, m if dx else 0, k) and ref.untouched(wbuf, n if dw else 0, k)
    return [loss[:m], lse[:m], picked[:m, :top], *out[3:]]


def run(m, n, k, t, top, kind="mixed", given=False, alpha=1.0, scale=0.7, seed=0, train=True, spread=2.0):
    say(f"[gpu distill] {m}x{n}x{k} {t} top={top} {kind} given={given} alpha={alpha}")
    g = rng(seed)
    x, w = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, spread * max(k, 1) ** -0.5)
    index, logit = dref.teacher(g, m, n, top, kind)
    lse_t = None
    if given:
        lse_t = torch.logsumexp(logit.double().cpu() * scale, 1).clamp(min=-5).float() + torch.rand(m, generator=g)
        lse_t = lse_t.cuda()
    grads = torch.randn(m, generator=g).cuda() if train else None
    got = call(x, w, t, index, logit, scale, lse_t, alpha, grads)
    d = dref.distill64(x, w, index, logit, scale, lse_t, alpha, k)
    for name, v in zip(("lse", "picked", "loss"), (got[1], got[2], got[0])):
        ref.assert_within(v, d[name], d[name + "_err"], name)
    if train:
        dx, dx_err, dw, dw_err = dref.distill_grad64(x, w, d, grads, alpha, k, t)
        ref.assert_within(got[3], dx, dx_err, "dX")
        ref.assert_within(got[4], dw, dw_err, "dW")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k,top", [(1, 1, 1, 1), (1, 100, 64, 5), (3, 257, 33, 4), (7, 1000, 129, 20), (16, 64, 520, 64),
                                       (31, 130, 72, 65), (65, 301, 40, 33), (128, 700, 96, 7), (129, 700, 96, 7),
                                       (200, 1021, 65, 128), (300, 515, 200, 3)])
def test_sizes(m, n, k, top, t):
    run(m, n, k, t, top, seed=m + n)
    run(m, n, k, t, top, given=True, alpha=0.6, seed=m + n + 1)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m", [9, 140])
def test_the_same_column_twice(m, t):
    run(m, 300, 64, t, 9, "twice", seed=3)
    run(m, 40, 64, t, 130, "plain", seed=4)              # more entries than columns


@pytest.mark.parametrize("m", [5, 150])
def test_the_most_entries(m):
    run(m, 2000, 40, "bf16", 1024, "plain", seed=5)
    run(m, 2000, 40, "f16", 1000, "mixed", given=True, seed=6)


def test_many_pieces():
    """More rows than one piece of the vocabulary takes: 65536 x 2 bytes by 1024 columns a piece."""
    m, n, k, t, top = 65600, 1300, 8, "bf16", 2
    g = rng(7)
    x, w = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t)
    index = torch.randint(0, n, (m, top), generator=g).cuda()
    index[::4] = -1
    logit = torch.randn(m, top, generator=g).cuda()
    grads = torch.rand(m, generator=g).cuda()
    got = call(x, w, t, index, logit, 1.0, None, 1.0, grads)
    rows = torch.cat([torch.arange(0, 64), torch.arange(m - 64, m)])   # (all of them against 64 bits would take long)
    d = dref.distill64(x[rows], w, index[rows], logit[rows], 1.0, None, 1.0, k)
    ref.assert_within(got[0][rows], d["loss"], d["loss_err"], "loss")
    dx, dx_err, _, _ = dref.distill_grad64(x[rows], w, d, grads[rows], 1.0, k, t)
    ref.assert_within(got[3][rows], dx, dx_err, "dX")


@pytest.mark.parametrize("m", [6, 200])
def test_one_gradient_at_a_time(m):
    g = rng(8)
    x, w = ref.matrix(g, m, 40, "bf16"), ref.matrix(g, 333, 40, "bf16", 0.3)
    index, logit = dref.teacher(g, m, 333, 6)
    grads = torch.randn(m, generator=g).cuda()
    both = call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads)
    assert torch.equal(both[3], call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads, dw=False)[3])
    assert torch.equal(both[4], call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads, dx=False)[4])


@pytest.mark.parametrize("m", [10, 150])
def test_rows_that_do_not_count(m):
    """NaN in their X and grad reaches nothing; a batch of nothing but such rows gives zeros."""
    g = rng(9)
    x, w = ref.matrix(g, m, 64, "bf16"), ref.matrix(g, 500, 64, "bf16", 0.2)
    index, logit = dref.teacher(g, m, 500, 8, "plain")
    grads = torch.randn(m, generator=g).cuda()
    index[1::2] = -1
    clean = call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads)
    x[1::2], grads[1::2], logit[1::2] = float("nan"), float("nan"), float("nan")
    got = call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads)
    for a, b in zip((clean[0], clean[3], clean[4]), (got[0], got[3], got[4])):
        assert torch.equal(a, b)
    assert bool((got[0][1::2] == 0).all()) and bool((got[3][1::2] == 0).all())
    index[:] = -1
    got = call(x, w, "bf16", index, logit, 1.0, None, 1.0, grads)
    assert bool((got[0] == 0).all()) and bool((got[3] == 0).all()) and bool((got[4] == 0).all())


def test_a_student_that_agrees():
    """Where student and teacher all but agree, P keeps its bits: it is formed before it is rounded.  The teacher's logits
    are the student's own, and its lse the student's: the true gradient at its columns is 0."""
    g, m, n, k, top = rng(10), 40, 256, 64, 64
    x, w = ref.matrix(g, m, k, "bf16", extra=0), ref.matrix(g, n, k, "bf16", 0.4, extra=0)
    z = x.double().cpu() @ w.double().cpu().t()
    index = z.topk(top, 1).indices.cuda()
    logit = z.gather(1, index.cpu()).float().cuda()
    lse = torch.logsumexp(z, 1).float().cuda()
    grads = torch.ones(m, device="cuda")
    got = call(x, w, "bf16", index, logit, 1.0, lse, 1.0, grads)
    d = dref.distill64(x, w, index, logit, 1.0, lse, 1.0, k)
    dx, dx_err, dw, dw_err = dref.distill_grad64(x, w, d, grads, 1.0, k, "bf16")
    ref.assert_within(got[3], dx, dx_err, "dX")
    ref.assert_within(got[4], dw, dw_err, "dW")


def test_nothing_to_sum():
    """k = 0: every logit is 0.  m = 0: dW = 0."""
    m, n, top = 5, 37, 3
    index, logit = dref.teacher(rng(11), m, n, top, "plain", extra=0)
    loss, lse, picked = (torch.full((m, c), ref.SENTINEL, device="cuda") for c in (1, 1, top))
    size = mp.mpgemm_linear_distill_workspace_size(m, n, 0, top, "bf16", False)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_distill(handle().h, m, n, 0, 1.0, None, "bf16", 8, None, 8, mp.Teacher(top, index, logit, top), loss, lse,
                                 picked, ws, size)
    q = torch.softmax(logit.double().cpu(), 1)
    want = (q * (q.log() + math.log(n))).sum(1)
    dW = torch.full((n, 8), ref.SENTINEL, dtype=torch.bfloat16, device="cuda")
    mp.mpgemm_run_linear_distill_grad(handle().h, 0, n, 8, 1.0, None, "bf16", 8, None, 8, mp.Teacher(top, None, None, top), None, None,
                                      None, None, 8, dW, 8, None, 0)
    torch.cuda.synchronize()
    assert bool((picked == 0).all()) and bool((dW == 0).all())
    ref.assert_within(loss[:, 0], want, 2.0 ** -16 + 0 * want, "loss")
    ref.assert_within(lse[:, 0], torch.full_like(want, math.log(n)), 2.0 ** -18 + 0 * want, "lse")


def test_gradient_of_differences():
    """dX and dW against differences of the 64-bit loss."""
    g, m, n, k, top, t = rng(12), 4, 50, 16, 5, "f16"
    x, w = ref.matrix(g, m, k, t, extra=0), ref.matrix(g, n, k, t, 0.5, extra=0)
    index, logit = dref.teacher(g, m, n, top, "plain", extra=0)
    grads = torch.rand(m, generator=g).cuda()
    got = call(x, w, t, index, logit, 0.5, None, 0.8, grads)

    def total(xv, wv):
        z = 0.8 * xv @ wv.t()
        q = torch.softmax(logit.double().cpu() * 0.5, 1)
        loss = (q * (q.log() - z.gather(1, index.cpu()) + torch.logsumexp(z, 1, keepdim=True))).sum(1)
        return float((loss * grads.double().cpu()).sum())
    x0, w0, h = x.double().cpu(), w.double().cpu(), 1e-5
    for which, i, j in [("x", 0, 0), ("x", 3, 15), ("w", int(index[0, 0]), 3), ("w", int(index[2, 4]), 9), ("w", 49, 0)]:
        d = torch.zeros_like(x0 if which == "x" else w0)
        d[i, j] = h
        want = (total(x0 + d, w0) - total(x0 - d, w0)) / (2 * h) if which == "x" else (total(x0, w0 + d) - total(x0, w0 - d)) / (2 * h)
        have = float(got[3 if which == "x" else 4][i, j])
        # P and the result are rounded to FP16 (2^-11 each, of sums of up to n + m terms of order one), the difference by h^2
        assert abs(have - want) <= 2.0 ** -10 * (abs(want) + 1.0) + 1e-6, (which, i, j)


def test_a_graph_between_eager_calls():
    g, m, n, k, top, t = rng(13), 150, 1000, 64, 9, "bf16"
    x, w = ref.matrix(g, m, k, t, extra=0), ref.matrix(g, n, k, t, 0.3, extra=0)
    index, logit = dref.teacher(g, m, n, top, extra=0)
    index, logit = index.contiguous(), logit.contiguous()
    grads = torch.randn(m, generator=g).cuda()
    size = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda"), torch.zeros(m, top, device="cuda"), torch.zeros_like(x),
            torch.zeros_like(w)]
    teacher = mp.Teacher(top, index, logit, top)

    def step():
        loss, lse, picked, dX, dW = outs
        mp.mpgemm_run_linear_distill(handle().h, m, n, k, 1.0, x, t, k, w, k, teacher, loss, lse, picked, ws, size)
        mp.mpgemm_run_linear_distill_grad(handle().h, m, n, k, 1.0, x, t, k, w, k, teacher, lse, picked, grads, dX, k, dW, k, ws, size)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(ref.matrix(rng(30 + seed), m, k, t, extra=0))
        new = dref.teacher(rng(40 + seed), m, n, top, extra=0)
        index.copy_(new[0])
        logit.copy_(new[1])
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        ws.fill_(0xFF)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert torch.equal(o, v)
