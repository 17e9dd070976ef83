"""Log probabilities of many long rows, where a wave has a row and takes up to sixteen turns over it, and of the
alternatives for which such rows get four waves: against 64 bits, with the bounds of
tests/test_gpu_logprobs.py.  All rows' statistics are compared, a part of the rows in every respect."""
import math

import pytest
import torch

from tests import logits_plans
from tests import ops_reference as ref
from tests.gpu_harness import say
from tests.test_gpu_logprobs import call, check, logits, rng

pytestmark = pytest.mark.gpu


def special(z, g):
    """Rows that are masked, constant, rising, falling, of few values, of one value but for the first and the last column."""
    m, n = z.shape
    low = torch.finfo(z.dtype).min
    z[0] = -math.inf
    z[1, : n - 3] = -math.inf
    z[2] = low
    z[3, 5:] = low
    z[4] = 1.5
    z[5] = torch.linspace(-8, 8, n).cuda().to(z.dtype)
    z[6] = torch.linspace(8, -8, n).cuda().to(z.dtype)
    z[7] = torch.randint(0, 3, (n,), generator=g).float().cuda().to(z.dtype)
    z[8] = -2.0
    z[8, 0] = z[8, n - 1] = 3.0
    z[9, torch.rand(n, generator=g).cuda() < 0.5] = -math.inf
    # the largest ones in one lane of one wave, turn after turn: groups of 32 elements of one lane
    z[10, ::2048] = 30.0
    z[m - 1, n - 1] = 40.0
    return list(range(11)) + [m - 1]


@pytest.mark.parametrize("t,m,n", [(t, m, n) for t in ("bf16", "f16") for m, n in
                                   ((1024, 8192), (601, 4801), (2100, 16384), (4096, 32768), (4096, 32761), (3100, 24799))] +
                         [("f32", 2048, 16384), ("f32", 1500, 11999), ("f32", 2048, 16377)])
@pytest.mark.parametrize("top", [0, 1, 20, 32, 64])
def test_rows_of_many_turns(t, m, n, top):
    if logits_plans.available():
        waves, parts, _ = logits_plans.logprobs(m, n, t, top)
        say(f"[gpu logprobs] {m}x{n} {t} top={top}: {waves} waves")
        assert (waves, parts) == (4 if top == 64 else 1, 1)
    g = rng(m + n)
    z = logits(g, m, n, t)
    rows = special(z, g)
    rows = sorted(set(rows + torch.randint(0, m, (20,), generator=g).tolist()))
    target = torch.randint(0, n, (m,), generator=g).cuda()
    got = call(z, t, 1.25, target, top)
    check(z[rows], t, 1.25, target[rows], top, {k: v[rows] for k, v in got.items()}, f"{m}x{n} {t}")
    # every row's log-sum-exp, on the device in 64 bits: 2^-18 covers the sums, 2^-21 of the value the products
    x = z.double() * 1.25
    want = torch.where(x.amax(1) == -math.inf, x.amax(1), torch.logsumexp(x - x.amax(1, keepdim=True), 1) + x.amax(1))
    live = want > -1e30
    ref.assert_within(got["lse"][live], want[live].cpu(), (2.0 ** -18 + 2.0 ** -21 * want[live].abs()).cpu(), "lse of all rows")


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(70, 2559), (70, 2560), (70, 4096), (600, 8192), (1100, 16384)])
@pytest.mark.parametrize("top", [33, 36, 37, 44, 45, 63])
def test_both_sides_of_the_rule(t, m, n, top):
    say(f"[gpu logprobs] {m}x{n} {t} top={top}")
    if t == "f32" and n > 8192:
        m = 2100
    g = rng(n + top)
    z = logits(g, m, n, t)
    rows = special(z, g) + [11, 12, 13, m - 2]
    target = torch.randint(0, n, (m,), generator=g).cuda()
    got = call(z, t, 1.0, target, top)
    check(z[rows], t, 1.0, target[rows], top, {k: v[rows] for k, v in got.items()}, f"{m}x{n} {t}")


def test_nan_and_infinity_in_rows_of_many_turns():
    """In the last of sixteen turns; no other row is touched."""
    m, n, t = 4096, 32768, "bf16"
    g = rng(4)
    z = logits(g, m, n, t)
    z[1, n - 1], z[3, n - 2], z[m - 1, 31000] = float("nan"), float("inf"), float("nan")
    target = torch.zeros(m, dtype=torch.int64, device="cuda")
    got = call(z, t, 1.0, target, 10)
    for r in (1, 3, m - 1):
        for name in ("logprob", "lse", "entropy"):
            assert math.isnan(float(got[name][r])), (r, name)
        at = got["top_index"][r].tolist()
        assert len(set(at)) == 10 and all(0 <= a < n for a in at)
    good = [0, 2, 4, 2000, m - 2]
    check(z[good], t, 1.0, target[good], 10, {k: v[good] for k, v in got.items()}, "the others")
