"""A teacher's logits scaled by nothing and by negative numbers, with entries of -infinity among them, against
64 bits.  The reference takes the scaled logits, -infinity where the logit is: the bounds are those of
tests/distill_reference.py, which count the roundings of the scaling."""
import math

import pytest
import torch

from tests import distill_reference as dref
from tests import ops_reference as ref
from tests.gpu_harness import say
from tests.test_gpu_distill import call, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.7, 0.7])
@pytest.mark.parametrize("m,n,k,top", [(9, 300, 64, 20), (150, 515, 72, 70), (5, 130, 40, 1)])
def test_entries_without_mass(m, n, k, top, scale, given, t):
    """Some logits of -infinity, rows of nothing else, entries and rows without a column."""
    say(f"[gpu distill] {m}x{n}x{k} {t} top={top} scale={scale} given={given}")
    g = rng(m + top)
    x, w = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, 2.0 * k ** -0.5)
    index, logit = dref.teacher(g, m, n, top, "mixed")
    # (float32(scale), as the library takes it)
    s = float(torch.tensor(scale, dtype=torch.float32))
    raw = logit.double().cpu()
    scaled = torch.where(raw == -math.inf, raw, raw * s)
    lse_t = None
    if given:
        lse_t = (torch.logsumexp(scaled, 1).clamp(min=-20).float() + torch.rand(m, generator=g)).cuda()
    grads = torch.randn(m, generator=g).cuda()
    got = call(x, w, t, index, logit, scale, lse_t, 1.0, grads)
    d = dref.distill64(x, w, index, scaled, 1.0, lse_t, 1.0, k)
    for name, v in zip(("lse", "picked", "loss"), (got[1], got[2], got[0])):
        ref.assert_within(v, d[name], d[name + "_err"], name)
    dx, dx_err, dw, dw_err = dref.distill_grad64(x, w, d, grads, 1.0, k, t)
    ref.assert_within(got[3], dx, dx_err, "dX")
    ref.assert_within(got[4], dw, dw_err, "dW")
    assert bool((got[0][~d["has"].any(1)] == 0).all()) and bool((got[3][~d["has"].any(1)] == 0).all())


def test_no_scale_gives_the_entries_the_same_share():
    """scale 0: q = 1 / entries, so that the loss is lse - log(entries) - the mean of the picked logits."""
    g, m, n, k, top, t = rng(3), 6, 100, 40, 8, "bf16"
    x, w = ref.matrix(g, m, k, t), ref.matrix(g, n, k, t, 0.3)
    index, logit = dref.teacher(g, m, n, top, "plain")
    loss, lse, picked = call(x, w, t, index, logit, 0.0, None, 1.0)
    want = lse.double().cpu() - math.log(top) - picked.double().cpu().mean(1)
    # log q is off by 2^-20 (see tests/distill_reference.py) and q by 2^-19, of terms of at most |lse| + |picked| + log 8 = 15
    ref.assert_within(loss, want, torch.full_like(want, 15 * 2.0 ** -18), "loss")
