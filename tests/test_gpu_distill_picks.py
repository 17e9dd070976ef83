"""The logits at the teacher's columns, formed by the kernel that joins the statistics or by one of their own: the
sizes on both sides of the rule, against 64 bits."""
import pytest

from tests import logits_plans
from tests.gpu_harness import say
from tests.test_gpu_distill import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k,top", [(300, 1500, 1024, 120), (255, 1500, 1024, 140), (256, 1100, 2048, 65), (9, 1500, 4096, 1000),
                                       (300, 700, 504, 300), (300, 700, 513, 300), (40, 700, 513, 32), (40, 700, 513, 33)])
def test_both_sides(m, n, k, top, t):
    say(f"[gpu distill] itself: {logits_plans.merge_picks(m, top, k) if logits_plans.available() else '?'}")
    run(m, n, k, t, top, train=False, seed=m + top)
