"""What the products of language models take as a scalar argument: numbers, and no text.  CPU only."""
from decimal import Decimal
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.test_distill_host import forward
from tests.test_distill_host import grad as distill_grad
from tests.test_gated_host import ALL
from tests.test_logprobs_host import check as logprobs
from tests.test_ops_host import OK, ce, ce_grad, epilogue, epilogue_grad, grouped, grouped_grad, wgrad

CALLS = [*ALL, forward, distill_grad, logprobs, ce, ce_grad, epilogue, epilogue_grad, grouped, grouped_grad, wgrad]


@pytest.mark.parametrize("check", CALLS)
def test_text_is_no_number(check):
    for v in ("1.5", "1", "nan", b"1.5", bytearray(b"1"), np.str_("2"), None, [1.0]):
        for name in {"alpha", "beta"} & check.names:
            with pytest.raises(TypeError):
                check(**{name: v})


@pytest.mark.parametrize("check", CALLS)
def test_numbers_of_any_kind(check):
    for v in (1, True, 0.5, np.float32(0.5), np.float64(2.0), np.int64(3), np.array(0.5), torch.tensor(0.5), torch.tensor(2),
              Decimal("0.5"), Fraction(1, 2)):
        assert check(alpha=v) == OK, v
