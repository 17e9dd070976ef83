"""Log probabilities, entropy and alternatives of stored logits on the GPU against the same in 64 bits, at
the sizes where vectors, waves and parts end and at the values where they can go wrong.

Bounds.  A lane adds at most n / 256 + 64 terms one after the other and the lanes meet in 14 more sums, each
off by 2^-24; an exponent (x - m) alpha / log 2 is rounded three times (3 2^-24 |u|), exp2 and log2 by
a unit.  log s is then off by (n / 256 + 80) 2^-24 + 2^-20 and 3 2^-24 E|u|, whose mean is taken with
the row's own p; t's terms by their own |u| more."""
import math

import pytest
import torch

import mixed_precision_dense_amd as mp
from tests import ops_reference as ref
from tests.gpu_harness import handle, say

pytestmark = pytest.mark.gpu


def rng(seed):
    return torch.Generator().manual_seed(seed)


def call(z, t, alpha=1.0, target=None, top=0, want=("logprob", "lse", "entropy")):
    """A dict of outputs; what lies past them must stay as it was."""
    m, n = z.shape
    ld_top = top + 3
    out = {name: torch.full((m + 1,), ref.SENTINEL, device="cuda") for name in want}
    at = torch.full((m + 1, ld_top), 77, dtype=torch.int64, device="cuda")
    value = torch.full((m + 1, ld_top), ref.SENTINEL, device="cuda")
    size = mp.mpgemm_logprobs_workspace_size(m, n, t, top)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_logprobs(handle().h, m, n, alpha, z, t, z.stride(0), target, out.get("logprob"), out.get("lse"), out.get("entropy"),
                           top, at, value, ld_top, ws, size)
    torch.cuda.synchronize()
    assert all(float(v[m]) == ref.SENTINEL for v in out.values())
    assert bool((at[:, top:] == 77).all()) and bool((at[m] == 77).all())
    assert bool((value[:, top:] == ref.SENTINEL).all()) and bool((value[m] == ref.SENTINEL).all())
    assert bool((ws[size:] == 0xFF).all())
    return {**{k: v[:m] for k, v in out.items()}, "top_index": at[:m, :top], "top_logprob": value[:m, :top]}


def order64(z, top):
    """Columns of the largest, equal ones by the lower column first; -1 past the columns."""
    at = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    return torch.nn.functional.pad(at, (0, top - at.shape[1]), value=-1)


def check(z, t, alpha, target, top, got, what):
    x = z.double().cpu()
    n = x.shape[1]
    y = x * alpha
    m = y.amax(1, keepdim=True)
    none = m[:, 0] == -math.inf
    # (from the maximum: beside logits of 3e38 even 64 bits would lose the logarithm of the sum)
    near = torch.where(none[:, None], torch.zeros_like(y), y - torch.where(none[:, None], torch.zeros_like(m), m))
    log_s = torch.where(none, torch.zeros_like(m[:, 0]), torch.logsumexp(near, 1))
    lse = m[:, 0] + log_s
    lp = torch.where(none[:, None], torch.full_like(y, -math.inf), near - log_s[:, None])
    p = lp.exp()
    u = torch.where(p > 0, near, torch.zeros_like(y)).abs()
    mean, square = (p * u).sum(1), (p * u * u).sum(1)
    err = (n / 256 + 80) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * mean + 2.0 ** -22 * log_s
    fin = lambda v: torch.where(v.abs() < math.inf, v.abs(), torch.zeros_like(v))   # noqa: E731
    close(got["lse"], lse, err + 2.0 ** -22 * (fin(m[:, 0]) + fin(lse)), what + " lse")
    want = torch.where(none, torch.zeros_like(lse), -torch.special.xlogy(p, p).sum(1))
    close(got["entropy"], want, err * (1 + mean) + 2.0 ** -21 * (square + mean) + 2.0 ** -22 * want.abs(), what + " entropy")
    if target is not None:
        tt = target.cpu()
        ok = (tt >= 0) & (tt < n)
        own = lp.gather(1, torch.where(ok, tt, torch.zeros_like(tt))[:, None])[:, 0]
        own = torch.where(ok, own, torch.zeros_like(own))
        close(got["logprob"], own, err + 2.0 ** -22 * (fin(own) + log_s), what + " logprob")
    if top:
        at = order64(x, top)
        assert torch.equal(got["top_index"].cpu(), at), what + " top_index"
        have = at >= 0
        v = torch.where(have, lp.gather(1, at.clamp(min=0)), torch.full(at.shape, -math.inf, dtype=torch.float64))
        close(got["top_logprob"], v, err[:, None] + 2.0 ** -22 * (fin(v) + log_s[:, None]), what + " top_logprob")


def close(got, want, bound, what):
    got = got.double().cpu()
    # (twice FP32's lowest value, 6.8e38, has no FP32 but an infinity)
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * math.inf, want)
    same_inf = (want == got) & (want.abs() == math.inf)
    ref.assert_within(torch.where(same_inf, torch.zeros_like(got), got), torch.where(same_inf, torch.zeros_like(want), want), bound, what)


def logits(gen, m, n, t, scale=3.0, extra=8):
    return ref.matrix(gen, m, n, t, scale, extra)     # (what lies past the rows is NaN)


def run(m, n, t, top, alpha=1.0, seed=0, change=None):
    say(f"[gpu logprobs] {m}x{n} {t} top={top} alpha={alpha}")
    g = rng(seed)
    z = logits(g, m, n, t)
    if change is not None:
        change(z, g)
    target = torch.randint(0, n, (m,), generator=g).cuda()
    target[::5] = torch.tensor([-1, n, -100, 1 << 40])[torch.arange(target[::5].numel()) % 4].cuda()
    check(z, t, alpha, target, top, call(z, t, alpha, target, top), f"{m}x{n} {t}")


TYPES = ["bf16", "f16", "f32"]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,n,top", [(1, 1, 1), (1, 3, 5), (2, 8, 8), (3, 9, 64), (1, 63, 64), (5, 64, 1), (4, 65, 2), (2, 255, 20),
                                     (2, 513, 33), (7, 1000, 63), (3, 2047, 20), (2, 4097, 64), (2, 8193, 5), (1, 20001, 20), (300, 129, 3)])
def test_sizes(m, n, top, t):
    run(m, n, t, top, seed=m * n)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,n,top", [(1, 100003, 20), (9, 50021, 64), (1, 600000, 1), (40, 33000, 0)])
def test_rows_in_parts(m, n, top, t):
    assert mp.mpgemm_logprobs_workspace_size(m, n, t, top) > 0
    run(m, n, t, top, alpha=1.25, seed=n)


@pytest.mark.parametrize("t", TYPES)
def test_more_rows_than_workgroups(t):
    run(70000, 9, t, 2, seed=1)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [200, 40000])
def test_masks(t, n):
    """Columns of -inf, all but fewer than top of them, rows of nothing else; the type's lowest value in their place."""
    low = torch.finfo(ref.TYPES[t]).min

    def mask(value):
        def change(z, g):
            z[0] = value
            z[1, 3:] = value
            z[2, : n - 2] = value
            z[3, torch.rand(n, generator=g).cuda() < 0.5] = value
            z[4] = value
            z[4, n - 1] = 1.0
        return change
    run(6, n, t, 20, seed=2, change=mask(-math.inf))
    run(6, n, t, 20, seed=2, change=mask(low))
    run(6, n, t, 20, alpha=2.0, seed=3, change=mask(low))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,top", [(300, 64), (40000, 64), (5000, 7)])
def test_equal_logits_and_orders(n, top, t):
    """Constant rows, few different values, both zeros, rising and falling rows: the lower column comes first."""
    def change(z, g):
        z[0] = 1.5
        z[1] = torch.randint(0, 3, (n,), generator=g).float().cuda().to(z.dtype)
        z[2] = torch.where(torch.rand(n, generator=g) < 0.5, 0.0, -0.0).cuda().to(z.dtype)
        z[3] = torch.linspace(-8, 8, n).cuda().to(z.dtype)
        z[4] = torch.linspace(8, -8, n).cuda().to(z.dtype)
        z[5] = -torch.arange(n).float().cuda().remainder(7).to(z.dtype)
    run(6, n, t, top, seed=4, change=change)


@pytest.mark.parametrize("t", TYPES)
def test_far_logits(t):
    """A single large value, values far apart, a small and a large alpha."""
    def change(z, g):
        z[0, 100] = 60000.0
        z[1] *= 1000
        z[2] = -60000.0
        z[2, ::7] = -59904.0
    for alpha in (1.0, 1e-6, 100.0):
        run(4, 700, t, 9, alpha=alpha, seed=5, change=change)


@pytest.mark.parametrize("n", [100, 70000])
def test_nan_and_infinity(n):
    """Such a row's numbers are NaN, its columns are columns; no other row is touched."""
    g = rng(6)
    z = logits(g, 6, n, "f32")
    z[1, 5], z[3, n - 1], z[4] = float("nan"), float("inf"), float("nan")
    target = torch.zeros(6, dtype=torch.int64, device="cuda")
    got = call(z, "f32", 1.0, target, 10)
    for r in (1, 3, 4):
        for name in ("logprob", "lse", "entropy"):
            assert math.isnan(float(got[name][r])), (r, name)
        at = got["top_index"][r].tolist()
        assert len(set(at)) == 10 and all(0 <= a < n for a in at)
    good = [0, 2, 5]
    check(z[good], "f32", 1.0, target[good], 10, {k: v[good] for k, v in got.items()}, "the others")


@pytest.mark.parametrize("n", [500, 50000])
def test_only_what_is_asked_for(n):
    g = rng(7)
    z = logits(g, 3, n, "bf16")
    target = torch.tensor([1, 2, 3], device="cuda")
    full = call(z, "bf16", 1.0, target, 5)
    for want in (("logprob",), ("lse",), ("entropy",), ()):
        for top in (0, 5):
            got = call(z, "bf16", 1.0, target if "logprob" in want else None, top, want)
            for name in want:
                assert torch.equal(got[name], full[name]), (want, top)
            if top:
                assert torch.equal(got["top_index"], full["top_index"]) and torch.equal(got["top_logprob"], full["top_logprob"])


def test_a_long_row_far_into_memory():
    """Rows more than 2^31 bytes apart in a buffer that is mostly not touched."""
    ld, n = (1 << 29) + 64, 1000
    buf = torch.empty(3 * ld, dtype=torch.float32, device="cuda")
    z = torch.as_strided(buf, (3, n), (ld, 1))
    z.copy_(torch.randn(3, n, generator=rng(8)))
    target = torch.tensor([5, 6, 7], device="cuda")
    check(z, "f32", 1.0, target, 4, call(z, "f32", 1.0, target, 4), "far rows")


@pytest.mark.parametrize("m,n", [(3, 60000), (200, 1000)])
def test_a_graph_between_eager_calls(m, n):
    g = rng(9)
    z = logits(g, m, n, "bf16", extra=0)
    target = torch.randint(0, n, (m,), generator=g).cuda()
    size = mp.mpgemm_logprobs_workspace_size(m, n, "bf16", 8)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda"),
            torch.zeros(m, 8, dtype=torch.int64, device="cuda"), torch.zeros(m, 8, device="cuda")]

    def step():
        mp.mpgemm_run_logprobs(handle().h, m, n, 1.0, z, "bf16", z.stride(0), target, outs[0], outs[1], outs[2], 8, outs[3], outs[4], 8,
                               ws, size)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        z.copy_(logits(rng(50 + seed), m, n, "bf16", extra=0))
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
