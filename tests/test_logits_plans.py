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


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_many_alternatives_of_long_rows_get_four_waves(t):
    """64 lanes' maxima do not bound them: see how many elements of random rows reach the bound."""
    for m, n, top in [(16, 4096, 48), (4096, 4096, 64), (4096, 2560, 64), (4096, 3000, 48), (1024, 8192, 40), (2048, 16384, 36),
                      (4096, 16384, 33), (512, 4096, 56)]:
        assert logits_plans.logprobs(m, n, t, top)[0] == 4, (m, n, top)
    if t != "f32":
        assert logits_plans.logprobs(4096, 32000, t, 64)[0] == 4 and logits_plans.logprobs(4096, 32768, t, 33)[0] == 4


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_one_wave_of_short_rows_and_of_many(t):
    for m, n, top in [(1, 1, 64), (16, 2559, 64), (4096, 2559, 64), (16, 4096, 44), (4096, 4096, 20), (1024, 8192, 36), (2048, 16384, 32),
                      (4096, 16384, 0)]:
        assert logits_plans.logprobs(m, n, t, top)[0] == 1, (m, n, top)
    assert logits_plans.logprobs(4096, 32768, t, 32)[0] == (4 if t == "f32" else 1)
    assert logits_plans.logprobs(4096, 32769, t, 0)[0] == 4 and logits_plans.logprobs(16, 4097, t, 0)[0] == 4


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("top", [0, 1, 20, 64])
def test_no_wave_has_more_turns_than_places_for_their_maxima(t, top):
    """16 turns of a wave, 32 elements a lane each."""
    per = 4 if t == "f32" else 8
    for m in (1, 2, 16, 255, 256, 1000, 4096, 100000):
        for n in (1, 2048, 2559, 2560, 4096, 4097, 8192, 16384, 16385, 32768, 32769, 128000, 131072, 131073, 500000, 10 ** 7):
            waves, parts, vectors = logits_plans.logprobs(m, n, t, top)
            assert vectors * per <= 16 * 32 * 64 * waves and parts * vectors * per >= n and (parts - 1) * vectors * per < n, (m, n)
