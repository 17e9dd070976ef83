"""Gated products, the distillation loss and log probabilities as a program uses them: captured into a
graph together, on streams, in place, with large offsets and shared weights, with offsets outside the
contract, after an error that the caller left pending, past a launch's workgroups, and all together in
the example's training."""
import ctypes
import os
import sys

import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import distill_reference as dref
from tests import gated_reference as gref
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def calls(m, n, k, groups, seed):
    """One of each call on its own buffers: (a function that queues them, the outputs, the input)."""
    g = torch.Generator().manual_seed(seed)
    t, top = "bf16", 6
    ld, ldn = -(-k // 8) * 8, -(-n // 8) * 8
    A, W = ref.matrix(g, m, k, t, extra=0), ref.matrix(g, 2 * n, k, t, k ** -0.5, extra=0)
    E = ref.matrix(g, groups * 2 * n, k, t, k ** -0.5, extra=0)
    V = ref.matrix(g, n, k, t, k ** -0.5, extra=0)
    offsets = torch.tensor([m * e // groups for e in range(groups + 1)], dtype=torch.int32, device="cuda")
    index, logit = dref.teacher(g, m, n, top, extra=0)
    weight = torch.rand(m, generator=g).cuda()
    out = {name: torch.zeros(m, c, dtype=torch.bfloat16, device="cuda")
           for name, c in (("D", ldn), ("kept", 2 * ldn), ("dD", 2 * ldn), ("H", ldn), ("G", ldn), ("ekept", 2 * ldn), ("dG", 2 * ldn))}
    out.update({name: torch.zeros(m, device="cuda") for name in ("loss", "lse", "own", "lse2", "entropy")})
    out["dbias"], out["edbias"] = torch.zeros(2 * n, device="cuda"), torch.zeros(groups * 2 * n, device="cuda")
    out["picked"], out["value"] = torch.zeros(m, top, device="cuda"), torch.zeros(m, top, device="cuda")
    out["at"] = torch.zeros(m, top, dtype=torch.int64, device="cuda")
    out["dX"], out["dW"] = torch.zeros(m, ld, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, ld, dtype=torch.bfloat16, device="cuda")
    s1, s2 = mp.mpgemm_gated_grad_workspace_size(1, m, n), mp.mpgemm_gated_grad_workspace_size(groups, m, n)
    s3 = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, t, True)
    s4 = mp.mpgemm_logprobs_workspace_size(m, n, t, top)
    ws = torch.zeros(max(s1, s2, s3, s4), dtype=torch.uint8, device="cuda")
    teacher = mp.Teacher(top, index, logit, top)
    h = handle().h

    def queue(stream=None):
        keep = dict(act="silu", ld_kept=2 * ldn, stride_kept=ldn)
        mp.mpgemm_run_gated(h, True, m, n, k, 1.0, A, t, ld, W, t, ld, n * ld, mp.Gated(kept=out["kept"], **keep), out["D"], t, ldn,
                            stream=stream)
        mp.mpgemm_run_gated_grad(h, True, m, n, k, 1.0, A, t, ld, V, t, ld,
                                 mp.GatedGrad(kept=out["kept"], H=out["H"], ldh=ldn, dbias=out["dbias"], **keep), out["dD"], t, 2 * ldn,
                                 ldn, ws, s1, stream=stream)
        mp.mpgemm_run_grouped_gated(h, True, groups, m, n, k, 1.0, A, t, ld, offsets, E, t, ld, 2 * n * ld, n * ld,
                                    mp.Gated(kept=out["ekept"], **keep), out["G"], t, ldn, stream=stream)
        mp.mpgemm_run_grouped_gated_grad(h, True, groups, m, n, k, 1.0, A, t, ld, offsets, E, t, ld, n * ld,
                                         mp.GatedGrad(kept=out["ekept"], dbias=out["edbias"], **keep), out["dG"], t, 2 * ldn, ldn, ws,
                                         s2, stream=stream)
        mp.mpgemm_run_linear_distill(h, m, n, k, 1.0, A, t, ld, V, ld, teacher, out["loss"], out["lse"], out["picked"], ws, s3,
                                     stream=stream)
        mp.mpgemm_run_linear_distill_grad(h, m, n, k, 1.0, A, t, ld, V, ld, teacher, out["lse"], out["picked"], weight, out["dX"], ld,
                                          out["dW"], ld, ws, s3, stream=stream)
        mp.mpgemm_run_logprobs(h, m, n, 1.0, out["D"], t, ldn, index[:, 0].contiguous() if stream is None else None,
                               out["own"] if stream is None else None, out["lse2"], out["entropy"], top, out["at"], out["value"], top,
                               ws, s4, stream=stream)

    return queue, out, A


@pytest.mark.parametrize("m,n,k,groups", [(5, 120, 72, 3), (300, 520, 136, 4)])
def test_graph_replays_equal_the_eager_calls(m, n, k, groups):
    """Replayed several times on changing inputs, with eager calls and synchronisations in between."""
    say(f"[gpu student] graph {m}x{n}x{k}")
    queue, out, A = calls(m, n, k, groups, 1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        queue(stream=s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            queue(stream=s)
    for turn in range(4):
        A.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(turn)).bfloat16())
        torch.cuda.synchronize()
        for v in out.values():
            v.zero_()
        queue(stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        want = {name: v.clone() for name, v in out.items()}
        for v in out.values():
            v.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        for name, v in out.items():
            assert torch.equal(v, want[name]), (turn, name)


def test_streams_and_repeats():
    """Calls on two streams at a time equal the ones on the current stream, and the same call gives the same
    bits every time."""
    first, second = calls(200, 264, 128, 5, 2), calls(33, 264, 128, 5, 3)
    want = []
    for queue, out, _ in (first, second):
        queue(stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append({name: v.clone() for name, v in out.items()})
        for v in out.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (queue, _, _), s in zip((first, second), streams):
            queue(stream=s)
    torch.cuda.synchronize()
    for (_, out, _), w in zip((first, second), want):
        for name, v in out.items():
            assert torch.equal(v, w[name]), name


@pytest.mark.parametrize("m", [20, 300])
def test_error_left_pending_by_the_caller_does_not_fail_a_call(m):
    """A HIP error the caller left pending on the thread is not returned as a call's status, stops no call half
    way through and stays pending."""
    say(f"[gpu student] pending error, {m} rows")
    hip = ctypes.CDLL("libamdhip64.so.7", mode=os.RTLD_NOLOAD)   # the runtime already loaded
    queue, out, _ = calls(m, 264, 128, 5, m)
    stream = torch.cuda.current_stream().cuda_stream
    queue(stream=stream)
    torch.cuda.synchronize()
    want = {name: v.clone() for name, v in out.items()}
    for v in out.values():
        v.zero_()
    torch.cuda.synchronize()
    bad = hip.hipSetDevice(ctypes.c_int(1 << 20))
    assert bad != 0
    try:
        queue(stream=stream)                                     # (raises for any other status)
        left = hip.hipGetLastError()
    finally:
        hip.hipGetLastError()                                    # leave nothing pending for torch's own launch checks
    torch.cuda.synchronize()
    for name, v in out.items():
        assert torch.equal(v, want[name]), name
    assert left == bad


@pytest.mark.parametrize("out", ["beside", "after"])
@pytest.mark.parametrize("m,n", [(40, 72), (700, 1500), (2100, 4400)])
def test_gradients_in_the_place_of_the_kept_factors(m, n, out):
    """D == kept, alike in type, leading dimension and stride."""
    g, k, t = torch.Generator().manual_seed(m), 72, "bf16"
    A, B = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, k ** -0.5)
    kbuf, _, _, stride = gref.pair(g, m, n, t, out)
    dbuf = torch.zeros_like(kbuf)
    for D in (dbuf, kbuf):
        grad = mp.GatedGrad(act="gelu", kept=kbuf, ld_kept=kbuf.stride(0), stride_kept=stride)
        mp.mpgemm_run_gated_grad(handle().h, True, m, n, k, 1.0, A, t, A.stride(0), B, t, B.stride(0), grad, D, t, kbuf.stride(0), stride,
                                 None, 0)
    torch.cuda.synchronize()
    first = torch.as_strided(dbuf, (m, n), (dbuf.stride(0), 1)), torch.as_strided(dbuf, (m, n), (dbuf.stride(0), 1), stride)
    second = torch.as_strided(kbuf, (m, n), (kbuf.stride(0), 1)), torch.as_strided(kbuf, (m, n), (kbuf.stride(0), 1), stride)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.parametrize("rows", [20, 600])
def test_one_pair_of_weights_for_all_experts(rows):
    """stride_b = 0 and bias_stride = 0: the experts' product of shared weights is the plain one."""
    g = torch.Generator().manual_seed(rows)
    n, k, groups = 72, 64, 5
    A, W = ref.matrix(g, rows, k, "bf16", extra=0), ref.matrix(g, 2 * n, k, "bf16", k ** -0.5, extra=0)
    bias = torch.randn(2, n, generator=g).cuda()
    offsets = torch.tensor([rows * e // groups for e in range(groups + 1)], dtype=torch.int32, device="cuda")
    D = torch.zeros(rows, n, device="cuda")
    mp.mpgemm_run_grouped_gated(handle().h, True, groups, rows, n, k, 1.0, A, "bf16", k, offsets, W, "bf16", k, 0, n * k,
                                mp.Gated(act="silu", bias_gate=bias[0], bias_up=bias[1]), D, "f32", n)
    torch.cuda.synchronize()
    (d, err), _, _ = gref.forward64(A, W[:n].t(), W[n:].t(), k, "silu", bias[0], bias[1])
    gref.check(D, d, err, "f32", "D")


@pytest.mark.parametrize("values", [[-5, 10, 40, 100], [0, 1000, 20, 60], [60, 40, 20, 0], [7, 7, 7, 7], [2 ** 31 - 1, -2 ** 31, 60, 3]])
@pytest.mark.parametrize("rows", [60, 300])
def test_offsets_outside_the_contract_touch_nothing_else(values, rows):
    """Offsets are clamped to 0 .. rows on the device: whatever they hold, only rows of the outputs and of the
    workspace are written."""
    say(f"[gpu student] offsets {values} rows {rows}")
    g = torch.Generator().manual_seed(9)
    n, k, groups = 40, 64, 3
    A, W = ref.matrix(g, rows, k, "f16"), ref.matrix(g, groups * 2 * n, k, "f16")
    offsets = torch.tensor(values, dtype=torch.int64).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda()
    dbuf, D = ref.output(rows, n, "f16")
    kbuf, G, U, ks = gref.pair_out(rows, n, "f16", "beside")
    pbuf, dG, dU, ps = gref.pair_out(rows, n, "f16", "after")
    size = mp.mpgemm_gated_grad_workspace_size(groups, rows, n)
    ws = torch.full((size + 4096,), 0x55, dtype=torch.uint8, device="cuda")
    db = torch.full((groups * 2 * n + 64,), ref.SENTINEL, device="cuda")
    ld = W.stride(0)
    mp.mpgemm_run_grouped_gated(handle().h, True, groups, rows, n, k, 1.0, A, "f16", A.stride(0), offsets, W, "f16", ld, 2 * n * ld,
                                n * ld, mp.Gated(act="silu", kept=kbuf, ld_kept=kbuf.stride(0), stride_kept=ks), D, "f16", D.stride(0))
    mp.mpgemm_run_grouped_gated_grad(handle().h, True, groups, rows, n, k, 1.0, A, "f16", A.stride(0), offsets, W, "f16", ld, n * ld,
                                     mp.GatedGrad(act="silu", kept=kbuf, ld_kept=kbuf.stride(0), stride_kept=ks, dbias=db), pbuf, "f16",
                                     pbuf.stride(0), ps, ws, size)
    torch.cuda.synchronize()
    assert ref.untouched(dbuf, rows, n) and gref.pair_untouched(kbuf, G, U) and gref.pair_untouched(pbuf, dG, dU)
    assert bool((ws[size:] == 0x55).all()) and bool((db[groups * 2 * n:] == ref.SENTINEL).all())


def test_offsets_past_32_bits():
    """Rows and the second of a pair beyond 2^32 bytes and 2^31 elements from the first, in both kernels' reach."""
    n, k, ld = 40, 64, 32768
    for m, rows in ((70000, [0, 1, 65535, 65536, 69999]), (3, [0, 1, 2])):
        g = torch.Generator().manual_seed(m)
        A, W = ref.matrix(g, m, k, "f16", extra=0), ref.matrix(g, 2 * n, k, "f16", k ** -0.5, extra=0)
        far = 3 * 2 ** 30 if m == 3 else m * ld
        kept = torch.zeros(far + m * ld, dtype=torch.float16, device="cuda")
        D = torch.zeros(m, n, dtype=torch.float16, device="cuda")
        mp.mpgemm_run_gated(handle().h, True, m, n, k, 1.0, A, "f16", k, W, "f16", k, n * k,
                            mp.Gated(act="relu", kept=kept, ld_kept=ld, stride_kept=far), D, "f16", n)
        torch.cuda.synchronize()
        (d, err), (gz, g_err), (uz, u_err) = gref.forward64(A[rows], W[:n].t(), W[n:].t(), k, "relu")
        G, U = torch.as_strided(kept, (m, n), (ld, 1)), torch.as_strided(kept, (m, n), (ld, 1), far)
        gref.check(D[rows], d, err, "f16", "D")
        gref.check(G[rows], gz, g_err, "f16", "G")
        gref.check(U[rows], uz, u_err, "f16", "U")
        # and read back, with the gradients in their place
        V = ref.matrix(g, n, k, "f16", k ** -0.5, extra=0)
        want = G[rows].clone(), U[rows].clone()
        mp.mpgemm_run_gated_grad(handle().h, True, m, n, k, 1.0, A, "f16", k, V, "f16", k,
                                 mp.GatedGrad(act="silu", kept=kept, ld_kept=ld, stride_kept=far), kept, "f16", ld, far, None, 0)
        torch.cuda.synchronize()
        e, e_err = ref.product64(A[rows], V.t(), k)
        (dg, dg_err), (du, du_err), _ = gref.grad64(e, e_err, *want, "silu")
        gref.check(G[rows], dg, dg_err, "f16", "dG")
        gref.check(U[rows], du, du_err, "f16", "dU")
        del kept
    # a pair of weights nearly 2^31 bytes apart
    g, far, m = torch.Generator().manual_seed(4), (1 << 30) - (1 << 17), 30
    A = ref.matrix(g, m, k, "f16", extra=0)
    B = torch.zeros(far + n * k, dtype=torch.float16, device="cuda")
    pair = [(torch.randn(n, k, generator=g) * k ** -0.5).half() for _ in range(2)]
    for e, at in enumerate((0, far)):
        B[at:at + n * k] = pair[e].reshape(-1).cuda()
    for rows in (m, 3):
        D = torch.zeros(rows, n, device="cuda")
        mp.mpgemm_run_gated(handle().h, True, rows, n, k, 1.0, A, "f16", k, B, "f16", k, far, mp.Gated(act="silu"), D, "f32", n)
        torch.cuda.synchronize()
        (d, err), _, _ = gref.forward64(A[:rows], pair[0].t(), pair[1].t(), k, "silu")
        gref.check(D, d, err, "f32", "D")


def test_distillation_past_a_grid():
    """More rows than one launch's workgroups, without rounding: every logit is 0, as X and W have columns of their
    own, and the teacher's entries have equal shares of 1/2, so that P is a multiple of 1/16."""
    m, n, k, top, t = (1 << 18) + 3, 16, 8, 2, "bf16"
    say(f"[gpu student] distill past a grid {m}x{n}x{k}")
    g = torch.Generator("cuda").manual_seed(m)
    X, W = (torch.zeros(r, k, dtype=torch.bfloat16, device="cuda") for r in (m, n))
    X[:, :4] = torch.randint(-3, 4, (m, 4), generator=g, device="cuda").bfloat16()
    W[:, 4:] = torch.randint(-3, 4, (n, 4), generator=g, device="cuda").bfloat16()
    index = torch.randint(0, n, (m, top), generator=g, device="cuda")
    index[3::5] = -1
    logit = torch.ones(m, top, device="cuda")
    counts = index[:, 0] >= 0
    grad = torch.where(counts, torch.ones(m, device="cuda"), torch.full((m,), float("nan"), device="cuda"))
    size = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    loss, lse, picked = torch.empty(m, device="cuda"), torch.empty(m, device="cuda"), torch.empty(m, top, device="cuda")
    dX, dW = torch.full_like(X, ref.SENTINEL), torch.full_like(W, ref.SENTINEL)
    teacher = mp.Teacher(top, index, logit, top)
    mp.mpgemm_run_linear_distill(handle().h, m, n, k, 1.0, X, t, k, W, k, teacher, loss, lse, picked, ws, size)
    mp.mpgemm_run_linear_distill_grad(handle().h, m, n, k, 1.0, X, t, k, W, k, teacher, lse, picked, grad, dX, k, dW, k, ws, size)
    torch.cuda.synchronize()
    assert bool((picked == 0).all())
    # log 16 - log 2, off by the roundings of a handful of FP32 operations on numbers below 4
    assert float((loss[counts] - 2.0794415).abs().max()) <= 2.0 ** -18 and bool((loss[~counts] == 0).all())
    # exp(picked - lse) is 1/16 but for those roundings, P and the BF16 it is rounded to then exact to 2^-18
    p = torch.full((m, n), 1.0 / n, device="cuda")
    p.scatter_add_(1, index.clamp(min=0), torch.where(counts, -0.5, 0.0)[:, None].expand(m, top).contiguous())
    p[~counts] = 0
    want = p.double() @ W.double()
    assert float((dX.double() - want).abs().max()) <= 2.0 ** -8 * 3 * 4 * 1.2
    total = p.double().t().contiguous() @ X.double()
    assert float((dW.double() - total).abs().max()) <= 2.0 ** -8 * float(total.abs().max()) + 2.0 ** -18 * 3 * m


def test_vectors_that_are_columns_are_refused():
    """The library takes the values of a vector one after the other: a column of a matrix has others between them."""
    column = torch.zeros(4, 3, device="cuda")[:, 0]
    target = torch.zeros(4, 3, dtype=torch.int64, device="cuda")[:, 0]
    z, flat = torch.zeros(4, 8, device="cuda"), torch.zeros(4, device="cuda")
    for vectors in ((target, flat, None, None), (None, None, column, None), (None, None, None, column)):
        with pytest.raises(ValueError, match="strides"):
            mp.mpgemm_run_logprobs(handle().h, 4, 8, 1.0, z, "f32", 8, *vectors, 0, None, None, 0, None, 0)
    with pytest.raises(ValueError, match="strides"):
        mp.Teacher(3, target, z, 8, lse=column)


def test_the_example_runs():
    import distill_student
    student, teacher, losses = distill_student.train(steps=8)
    assert len(losses) == 8 and all(0 < v < 20 for v in losses)
    tokens = torch.arange(5, device="cuda")
    best = teacher.answer(tokens)[0][:, 0].contiguous()
    own, entropy, at, value = student.answer(tokens, best)
    assert bool((value[:, 1:] <= value[:, :-1]).all()) and bool((own <= value[:, 0] + 1e-6).all())
    for i in range(5):                                            # the same one at a time
        one = student.answer(tokens[i:i + 1], best[i:i + 1])
        assert abs(float(one[0][0] - own[i])) < 0.1 and abs(float(one[1][0] - entropy[i])) < 0.1


def test_the_example_gradients_are_differences_of_its_loss():
    """The loss along the gradient of every weight, against differences in steps of the masters."""
    import distill_student
    teacher, student = distill_student.Teacher(96, 48, 12, 7), distill_student.Student(vocab=96, width=64, inner=128, experts=3, seed=3)
    tokens = torch.randint(0, 96, (256,), generator=torch.Generator().manual_seed(5)).cuda()
    index, value = teacher.answer(tokens)
    index[::9] = -1
    _, grads = student.loss_and_gradients(tokens, index, value)
    for name, grad in grads.items():
        master = student.master[name].clone()
        step = 0.3 * grad / grad.norm()
        loss = []
        for sign in (1, -1):
            student.master[name] = master + sign * step
            student.w[name] = student.master[name].to(torch.bfloat16)
            moved = student.w[name].float() if name != "bias" else student.master[name]
            loss.append((float(student.loss_and_gradients(tokens, index, value)[0]), moved))
        student.master[name], student.w[name] = master, master.to(torch.bfloat16)
        want = float((grad.double() * (loss[0][1] - loss[1][1]).double()).sum())
        diff = loss[0][0] - loss[1][0]
        # BF16 activations and gradients: 2^-8 each over a dozen roundings on the way; the step's third order
        assert abs(diff - want) <= 0.06 * abs(want) + 2e-3, (name, diff, want)
