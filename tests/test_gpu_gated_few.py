"""The gated product at a size of each of its kernels (tests/gated_cases.py; a host test holds that none is left out),
against 64 bits, with both factors kept."""
import pytest

from tests import gated_cases, gated_plans
from tests.gpu_harness import say
from tests.test_gpu_gated import run_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("groups,m,n,k", gated_cases.SIZES)
def test_every_kernel(groups, m, n, k, t, tb):
    say(f"[gpu gated] kernel {gated_plans.gated(groups, m, n, k, tb, 'silu', True) if gated_plans.available() else '?'}")
    out = "f32" if m % 2 else t
    run_forward(m, n, k, t, out, tb, "silu", "beside" if n % 2 else "after", (t, t) if m % 3 else (None, "f32"), "beside", seed=n,
                shares=gated_cases.shares(groups, m))
