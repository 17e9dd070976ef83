"""The products of language models as a program uses them: captured into a graph, on streams, with large
offsets, shared weights, offsets outside the contract, after an error that the caller left pending, with
more rows than a launch has workgroups, and all together in the example's training."""
import ctypes
import math
import os
import sys

import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def calls(m, n, k, groups, seed):
    """One of each product on its own buffers: (a function that queues them, the outputs)."""
    g = torch.Generator().manual_seed(seed)
    t = "bf16"
    A, W = ref.matrix(g, m, k, t, extra=0), ref.matrix(g, n, k, t, k ** -0.5, extra=0)
    E = ref.matrix(g, groups * n, k, t, k ** -0.5, extra=0)
    bias = torch.randn(n, generator=g).cuda()
    offsets = torch.tensor([m * e // groups for e in range(groups + 1)], dtype=torch.int32, device="cuda")
    target = torch.randint(0, n, (m,), generator=g).cuda()
    ld = W.stride(0)
    ldn = -(-n // 8) * 8
    out = {name: torch.zeros(m, ldn, dtype=torch.bfloat16, device="cuda") for name in ("D", "Z", "dZ", "G")}
    out["dbias"] = torch.zeros(n, device="cuda")
    out["dV"] = torch.zeros(groups * k, ldn, device="cuda")
    out["loss"], out["lse"] = torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda")
    out["dX"], out["dW"] = torch.zeros(m, ld, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, ld, dtype=torch.bfloat16, device="cuda")
    weight = torch.full((m,), 1.0 / m, device="cuda")
    s1 = mp.mpgemm_epilogue_grad_workspace_size(1, m, n)
    s2 = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.zeros(max(s1, s2), dtype=torch.uint8, device="cuda")
    h = handle().h

    def queue(stream=None):
        mp.mpgemm_run_epilogue(h, False, True, m, n, k, 1.0, A, t, ld, W, t, ld,
                               mp.Epilogue(act="gelu", bias=bias, aux=out["Z"], ld_aux=ldn), 0.0, None, t, ldn, out["D"], t, ldn,
                               stream=stream)
        mp.mpgemm_run_epilogue_grad(h, False, True, m, n, k, 1.0, A, t, ld, W, t, ld, "gelu", out["Z"], ldn, out["dZ"], t, ldn,
                                    out["dbias"], ws, s1, stream=stream)
        mp.mpgemm_run_grouped(h, True, groups, m, n, k, 1.0, A, t, ld, offsets, E, t, ld, n * ld, mp.Epilogue(act="silu"),
                              out["G"], t, ldn, stream=stream)
        mp.mpgemm_run_grouped_wgrad(h, groups, m, k, n, 1.0, A, t, ld, out["dZ"], t, ldn, offsets, 0.0, out["dV"], "f32", ldn,
                                    k * ldn, stream=stream)
        mp.mpgemm_run_linear_ce(h, m, n, k, 1.0, A, t, ld, W, ld, target, out["loss"], out["lse"], ws, s2, stream=stream)
        mp.mpgemm_run_linear_ce_grad(h, m, n, k, 1.0, A, t, ld, W, ld, target, out["lse"], weight, out["dX"], ld, out["dW"], ld,
                                     ws, s2, stream=stream)

    return queue, out, A


@pytest.mark.parametrize("m,n,k,groups", [(5, 120, 72, 3), (300, 520, 136, 4)])
def test_graph_replays_equal_the_eager_calls(m, n, k, groups):
    """Replayed several times on changing inputs, with eager calls and synchronisations in between."""
    say(f"[gpu ops] graph {m}x{n}x{k}")
    queue, out, A = calls(m, n, k, groups, 1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        queue()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            queue()
    for turn in range(4):
        A.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(turn)).bfloat16())
        torch.cuda.synchronize()
        for v in out.values():
            v.zero_()
        queue()
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
    """Calls on two streams at a time, each given explicitly, equal the ones on the current stream, and the
    same call gives the same bits every time."""
    first, second = calls(200, 264, 128, 5, 2), calls(33, 264, 128, 5, 3)
    want = []
    for queue, out, _ in (first, second):
        queue()
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


@pytest.mark.parametrize("m", [64, 300])
def test_error_left_pending_by_the_caller_does_not_fail_a_call(m):
    """A HIP error the caller left pending on the thread (from hipSetDevice on a device that does not
    exist) is not returned as a call's status, stops no call half way through and stays pending."""
    say(f"[gpu ops] pending error, {m} rows")
    hip = ctypes.CDLL("libamdhip64.so.7", mode=os.RTLD_NOLOAD)   # the runtime already loaded
    queue, out, _ = calls(m, 264, 128, 5, m)
    queue()
    torch.cuda.synchronize()
    want = {name: v.clone() for name, v in out.items()}
    for v in out.values():
        v.zero_()
    stream = torch.cuda.current_stream().cuda_stream
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


def test_offsets_past_32_bits():
    """Rows of D, C and Z beyond 2^32 bytes and 2^31 elements from their start, in both kernels' reach."""
    n, k, ld = 40, 64, 32768
    for m in (70000, 66000):
        g = torch.Generator().manual_seed(m)
        A, W = ref.matrix(g, m, k, "f16", extra=0), ref.matrix(g, n, k, "f16", k ** -0.5, extra=0)
        big = torch.zeros(m, ld, dtype=torch.float16, device="cuda")
        aux = torch.zeros(m, ld, dtype=torch.float16, device="cuda")
        assert m * ld > 2 ** 31
        mp.mpgemm_run_epilogue(handle().h, False, True, m, n, k, 1.0, A, "f16", k, W, "f16", k,
                               mp.Epilogue(act="relu", aux=aux, ld_aux=ld), 0.0, None, "f16", ld, big, "f16", ld)
        torch.cuda.synchronize()
        rows = [0, 1, 65535, 65536, 65599, m - 1]
        z, z_err = ref.product64(A[rows], W.t(), k)
        d, err, _, _ = ref.forward64(z, z_err, "relu")
        ref.assert_within(big[rows, :n], d, err + ref.rounding(d, "f16"), "D")
        ref.assert_within(aux[rows, :n], z, z_err + ref.rounding(z, "f16"), "Z")
        assert bool((big[:, n:n + 8] == 0).all())
        del big, aux
    # experts' weights and gradients far apart
    groups, rows, far = 3, 30, 3 * 2 ** 30
    g = torch.Generator().manual_seed(4)
    A, X = ref.matrix(g, rows, k, "f16", extra=0), ref.matrix(g, rows, n, "f16", extra=0)
    B = torch.zeros(2 * far + n * k, dtype=torch.float16, device="cuda")
    experts = [(torch.randn(n, k, generator=g) * k ** -0.5).half() for _ in range(groups)]
    for e in range(groups):
        B[e * far:e * far + n * k] = experts[e].reshape(-1).cuda()
    offsets = torch.tensor([0, 8, 9, rows], dtype=torch.int32, device="cuda")
    D = torch.zeros(rows, n, device="cuda")
    mp.mpgemm_run_grouped(handle().h, True, groups, rows, n, k, 1.0, A, "f16", k, offsets, B, "f16", k, far, mp.Epilogue(), D,
                          "f32", n)
    mp.mpgemm_run_grouped_wgrad(handle().h, groups, rows, n, k, 1.0, X, "f16", n, A, "f16", k, offsets, 0.0, B, "f16", k, far)
    torch.cuda.synchronize()
    cut = offsets.tolist()
    for e in range(groups):
        r = slice(cut[e], cut[e + 1])
        z, err = ref.product64(A[r], experts[e].t(), k)
        ref.assert_within(D[r], z, err + ref.rounding(z, "f32"), f"D of expert {e}")
        v, err = ref.product64(X[r].t(), A[r], cut[e + 1] - cut[e])
        ref.assert_within(B[e * far:e * far + n * k].view(n, k), v, err + ref.rounding(v, "f16"), f"dV of expert {e}")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,k", [(70000, 24), (9000, 15000), ((1 << 24) + 3, 8)])
def test_cross_entropy_past_a_grid(t, m, k):
    """Rows and row blocks past the workgroups of one launch, without any rounding: X and W are small integers in
    columns of their own, so that every logit is 0, P a multiple of 1/16 and each sum exact in FP32."""
    say(f"[gpu ops] linear_ce past a grid {m}x16x{k} {t}")
    n, dt = 16, ref.TYPES[t]
    g = torch.Generator("cuda").manual_seed(m)
    X = torch.zeros(m, k, dtype=dt, device="cuda")
    W = torch.zeros(n, k, dtype=dt, device="cuda")
    X[:, :k // 2] = torch.randint(-3, 4, (m, k // 2), generator=g, device="cuda").to(dt)
    W[:, k // 2:] = torch.randint(-3, 4, (n, k - k // 2), generator=g, device="cuda").to(dt)
    target = torch.randint(0, n, (m,), generator=g, device="cuda")
    target[3::5] = -100
    counts = target >= 0
    grad = torch.where(counts, torch.ones(m, device="cuda"), torch.full((m,), float("nan"), device="cuda"))
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    loss, lse = torch.full((m,), ref.SENTINEL, device="cuda"), torch.full((m,), ref.SENTINEL, device="cuda")
    mp.mpgemm_run_linear_ce(handle().h, m, n, k, 1.0, X, t, k, W, k, target, loss, lse, ws, size)
    torch.cuda.synchronize()
    # exponentials of 0 are exact; the logarithm and its product with log 2 are off by a unit each
    assert float((lse.double() - math.log(n)).abs().max()) <= 2.0 ** -21
    assert torch.equal(loss, torch.where(counts, lse, torch.zeros_like(lse)))
    dX, dW = torch.full_like(X, ref.SENTINEL), torch.full_like(W, ref.SENTINEL)
    mp.mpgemm_run_linear_ce_grad(handle().h, m, n, k, 1.0, X, t, k, W, k, target, lse, grad, dX, k, dW, k, ws, size)
    torch.cuda.synchronize()
    del ws
    p = torch.full((m, n), 1.0 / n, device="cuda")
    p[torch.arange(m, device="cuda")[counts], target[counts]] -= 1
    p[~counts] = 0
    want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
    for r in range(0, m, 1 << 20):
        x = slice(r, min(m, r + (1 << 20)))
        assert torch.equal(dX[x], (p[x].double() @ W.double()).to(dt))
        want += p[x].double().t().contiguous() @ X[x].double()
    assert torch.equal(dW, want.to(dt))


@pytest.mark.parametrize("n", [5_000_003, (1 << 30) + 100])
def test_column_sums_past_a_grid(n):
    """The sum of no rows, over more columns than one launch's workgroups take at a time."""
    b = torch.full((n,), 3.0, device="cuda")
    ld = -(-n // 8) * 8
    mp.mpgemm_run_epilogue_grad(handle().h, False, True, 0, n, 8, 1.0, None, "f16", 8, None, "f16", 8, "silu", None, ld, None, "f32",
                                ld, b, None, 0)
    torch.cuda.synchronize()
    assert not bool(b.any())


@pytest.mark.parametrize("rows", [20, 600])
def test_one_weight_for_all_experts(rows):
    """stride_b = 0 and bias_stride = 0: a grouped product of shared weights is the plain one."""
    g = torch.Generator().manual_seed(rows)
    n, k, groups = 72, 64, 5
    A, W = ref.matrix(g, rows, k, "bf16", extra=0), ref.matrix(g, n, k, "bf16", k ** -0.5, extra=0)
    bias = torch.randn(n, generator=g).cuda()
    offsets = torch.tensor([rows * e // groups for e in range(groups + 1)], dtype=torch.int32, device="cuda")
    D = torch.zeros(rows, n, device="cuda")
    mp.mpgemm_run_grouped(handle().h, True, groups, rows, n, k, 1.0, A, "bf16", k, offsets, W, "bf16", k, 0,
                          mp.Epilogue(act="silu", bias=bias), D, "f32", n)
    z, z_err = ref.product64(A, W.t(), k)
    d, err, _, _ = ref.forward64(z, z_err, "silu", bias)
    torch.cuda.synchronize()
    ref.assert_within(D, d, err + ref.rounding(d, "f32"), "D")


@pytest.mark.parametrize("values", [[-5, 10, 40, 100], [0, 1000, 20, 60], [60, 40, 20, 0], [7, 7, 7, 7], [2 ** 31 - 1, -2 ** 31, 60, 3]])
@pytest.mark.parametrize("rows", [60, 300])
def test_offsets_outside_the_contract_touch_nothing_else(values, rows):
    """Offsets are clamped to 0 .. rows on the device: whatever they hold, only rows of D, of dbias and of the
    workspace are written (A, B and the rest of the buffers stay as they were)."""
    say(f"[gpu ops] offsets {values} rows {rows}")
    g = torch.Generator().manual_seed(9)
    n, k, groups = 40, 64, 3
    A, W = ref.matrix(g, rows, k, "f16"), ref.matrix(g, groups * n, k, "f16")
    Z = ref.matrix(g, rows, n, "f16")
    offsets = torch.tensor(values, dtype=torch.int64).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda()
    dbuf, D = ref.output(rows, n, "f16")
    vbuf, V = ref.output(groups * k, n, "f32")
    size = mp.mpgemm_epilogue_grad_workspace_size(groups, rows, n)
    ws = torch.full((size + 4096,), 0x55, dtype=torch.uint8, device="cuda")
    db = torch.full((groups * n + 64,), ref.SENTINEL, device="cuda")
    mp.mpgemm_run_grouped(handle().h, True, groups, rows, n, k, 1.0, A, "f16", A.stride(0), offsets, W, "f16", W.stride(0),
                          n * W.stride(0), mp.Epilogue(), D, "f16", D.stride(0))
    mp.mpgemm_run_grouped_grad(handle().h, True, groups, rows, n, k, 1.0, A, "f16", A.stride(0), offsets, W, "f16", W.stride(0),
                               n * W.stride(0), "silu", Z, Z.stride(0), D, "f16", D.stride(0), db, ws, size)
    mp.mpgemm_run_grouped_wgrad(handle().h, groups, rows, k, n, 1.0, A, "f16", A.stride(0), Z, "f16", Z.stride(0), offsets, 0.0,
                                V, "f32", V.stride(0), k * V.stride(0))
    torch.cuda.synchronize()
    assert ref.untouched(dbuf, rows, n) and ref.untouched(vbuf, groups * k, n)
    assert bool((ws[size:] == 0x55).all()) and bool((db[groups * n:] == ref.SENTINEL).all())
    assert bool(V.isfinite().all())


def test_the_example_learns():
    import train_experts
    losses, right = train_experts.train(steps=60)
    say(f"[gpu ops] example: loss {losses[0]:.3f} -> {losses[-1]:.3f}, {right:.2f} right")
    assert abs(losses[0] - 6.9) < 1.0                      # log(1000), give or take the random head
    assert losses[-1] < 0.5 * losses[0]


def test_the_example_answers():
    """Single tokens through the trained weights: a row whose loss is below log 2 has the right answer, so that a mean
    loss of 0.05 leaves at most one in fourteen wrong."""
    import train_experts
    losses, right = train_experts.train(steps=60)
    assert losses[-1] < 0.05 and right > 0.9, (losses[-1], right)


def test_the_example_gradients_are_differences_of_its_loss():
    """The loss along the gradient of every weight, against differences in FP64 steps of the masters."""
    import train_experts
    model = train_experts.Model(vocab=96, width=64, inner=128, experts=4, seed=3)
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, 96, (256,), generator=g).cuda()
    target = torch.randint(0, 96, (256,), generator=g).cuda()
    _, grads = model.loss_and_gradients(tokens, target)
    for name, grad in grads.items():
        master = model.master[name].clone()
        step = 0.3 * grad / grad.norm()
        loss = []
        for sign in (1, -1):
            model.master[name] = master + sign * step
            model.w[name] = model.master[name].to(torch.bfloat16)
            moved = model.w[name].float() if name not in ("b1", "b2") else model.master[name]
            loss.append((float(model.loss_and_gradients(tokens, target)[0]), moved))
        model.master[name], model.w[name] = master, master.to(torch.bfloat16)
        want = float((grad.double() * (loss[0][1] - loss[1][1]).double()).sum())
        diff = loss[0][0] - loss[1][0]
        # BF16 activations and gradients: 2^-8 each over a dozen roundings on the way; the step's third order
        assert abs(diff - want) <= 0.06 * abs(want) + 2e-3, (name, diff, want)
