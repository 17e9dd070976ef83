"""Which kernels the losses and the log probabilities take, where the rules turn.  CPU only."""
import pytest

from tests import logits_plans

pytestmark = pytest.mark.skipif(not logits_plans.available(), reason="g++ builds the rules")
BIG = 2 ** 31 - 257


@pytest.mark.parametrize("m,top,k", [(1, 1024, 8192), (8, 1000, 4096), (8, 1024, 4096), (8, 1024, 8192), (16, 512, 4096), (64, 128, 4096),
                                     (64, 512, 4096), (128, 512, 4096), (255, 1024, 8192), (1, 1024, BIG), (4096, 40, 256)])
def test_few_rows_of_many_entries_are_picked_by_a_kernel_of_their_own(m, top, k):
    """A workgroup a row would leave the other CUs idle (or, at a short k, half of each wave)."""
    assert not logits_plans.merge_picks(m, top, k)


@pytest.mark.parametrize("m,top,k", [(256, 128, 4096), (512, 64, 2048), (1024, 64, 1024), (4096, 64, 4096), (BIG, 1024, BIG)])
def test_many_rows_pick_for_themselves(m, top, k):
    assert logits_plans.merge_picks(m, top, k)


def test_a_turn_of_entries_and_little_work():
    for m in (1, 8, 300):
        for k in (0, 64, 4096):
            assert logits_plans.merge_picks(m, 32, k) and logits_plans.merge_picks(m, 1, k)
    assert not logits_plans.merge_picks(300, 33, 0) and not logits_plans.merge_picks(300, 33, 512)
