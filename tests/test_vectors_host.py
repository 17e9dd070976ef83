"""What the binding refuses where the library takes an address alone: values that do not follow each other
in memory, or of another type than the one that is read there.  CPU only (refused before any address is taken)."""
import pytest
import torch

import mixed_precision_dense_amd as mp
from tests.test_ops_host import P


def logprobs(target=None, logprob=None, lse=None, entropy=None, top=0, top_index=None, top_logprob=None):
    return mp.mpgemm_check_logprobs(4, 8, 1.0, P, "f32", 8, target, logprob, lse, entropy, top, top_index, top_logprob, 8, P, 1 << 20)


def teacher(index=P, logit=P, lse=None):
    return mp.Teacher(3, index, logit, 8, lse=lse)


def distill(loss=P, lse=P, picked=P):
    return mp.mpgemm_check_linear_distill(4, 8, 8, 1.0, P, "bf16", 8, P, 8, teacher(), loss, lse, picked, P, 1 << 20)


def distill_grad(lse=P, picked=P, grad=P):
    return mp.mpgemm_check_linear_distill_grad(4, 8, 8, 1.0, P, "bf16", 8, P, 8, teacher(), lse, picked, grad, P, 8, P, 8, P, 1 << 20)


def experts(offsets):
    return mp.mpgemm_check_grouped_gated(True, 3, 4, 8, 8, 1.0, P, "bf16", 8, offsets, P, "bf16", 8, 128, 64, mp.Gated(), P, "bf16", 8)


def experts_grad(offsets):
    return mp.mpgemm_check_grouped_gated_grad(True, 3, 4, 8, 8, 1.0, P, "bf16", 8, offsets, P, "bf16", 8, 64,
                                              mp.GatedGrad(kept=P, ld_kept=16, stride_kept=8), P, "bf16", 16, 8, None, 0)


CALLS = [(logprobs, "target", torch.int64), (logprobs, "logprob", None), (logprobs, "lse", None), (logprobs, "entropy", None),
         (teacher, "lse", None), (distill, "loss", None), (distill, "lse", None), (distill_grad, "lse", None),
         (distill_grad, "grad", None), (experts, "offsets", torch.int32), (experts_grad, "offsets", torch.int32)]
ROWS = [(logprobs, "top_index", torch.int64), (logprobs, "top_logprob", None), (teacher, "index", torch.int64), (teacher, "logit", None),
        (distill, "picked", None), (distill_grad, "picked", None)]
TYPES = [torch.float32, torch.bfloat16, torch.float16, torch.float64, torch.int64, torch.int32]


@pytest.mark.parametrize("call,name,dtype", CALLS + ROWS)
def test_other_types_are_refused(call, name, dtype):
    for t in TYPES:
        x = torch.zeros(4, 8, dtype=t)
        # (of its own type the tensor is refused for where it lies, as everywhere)
        with pytest.raises(ValueError, match="tensor on cpu" if t is (dtype or torch.float32) else f"must be {dtype or torch.float32}"):
            call(**{name: x})


@pytest.mark.parametrize("call,name,dtype", CALLS)
def test_columns_are_refused(call, name, dtype):
    x = torch.zeros(4, 3, dtype=dtype or torch.float32)
    with pytest.raises(ValueError, match="strides"):
        call(**{name: x[:, 0]})


@pytest.mark.parametrize("call,name,dtype", ROWS)
def test_rows_of_strided_values_are_refused_and_distant_rows_are_not(call, name, dtype):
    x = torch.zeros(8, 16, dtype=dtype or torch.float32)
    with pytest.raises(ValueError, match="strides"):
        call(**{name: x.t()[:4]})
    with pytest.raises(ValueError, match="tensor on cpu"):
        call(**{name: x[:4, :3]})


@pytest.mark.parametrize("name", ["bias_gate", "bias_up"])
def test_biases_are_rows(name):
    for t in (torch.bfloat16, torch.float32):
        x = torch.zeros(8, 16, dtype=t)
        with pytest.raises(ValueError, match="strides"):
            mp.Gated(**{name: x[:, 0]})
        with pytest.raises(ValueError, match="tensor on cpu"):
            mp.Gated(**{name: x[:, :8]})
    with pytest.raises(ValueError, match="must be torch.float32"):
        mp.GatedGrad(dbias=torch.zeros(2, 8, dtype=torch.bfloat16))


def test_addresses_are_taken_as_they_are():
    assert logprobs(target=P, logprob=P, lse=P, entropy=P, top=3, top_index=P, top_logprob=P) == 0
    assert distill() == 0 and distill_grad() == 0 and experts(P) == 0 and experts_grad(P) == 0
