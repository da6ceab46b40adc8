"""Whole-number arguments of the expert-layer calls: what does not fit is
refused, never cut off."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn

BIG = [2 ** 32, 2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1, -2 ** 32, 2 ** 64, 2 ** 70]
DEV = "cuda:0"


@pytest.mark.parametrize("value", BIG)
def test_numbers_that_do_not_fit(value):
    from allreduce_sum_residual_gb300 import experts
    with pytest.raises(ValueError, match="first must be"):
        experts._whole(value, "first")
    with pytest.raises(ValueError, match="act must be"):
        experts._option(arn.ACTS, value, "act")


@pytest.mark.parametrize("value", [2.0, 2.7, "2", None, torch.tensor([1, 2])])
def test_what_is_no_whole_number(value):
    from allreduce_sum_residual_gb300 import experts
    with pytest.raises(TypeError):
        experts._whole(value, "k")


def test_numbers_that_fit():
    import numpy as np
    from allreduce_sum_residual_gb300 import experts
    for v in (0, 1, -1, 2 ** 31 - 1, -2 ** 31, np.int64(7), np.uint8(3), torch.tensor(5)):
        assert experts._whole(v, "k") == int(v)
    assert experts._option(arn.ACTS, "silu_mul", "act") == arn.AR_ACT_SILU_MUL
    assert experts._option(arn.ACTS, np.int32(1), "act") == 1


@pytest.mark.gpu
@pytest.mark.parametrize("value", BIG)
@pytest.mark.parametrize("own_stream", [False, True])
def test_calls_refuse_numbers_that_do_not_fit(value, own_stream):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((2, 8, 32), dtype=torch.uint8, device=DEV)
    s = torch.zeros((2, 8, 1), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    st = torch.cuda.current_stream() if own_stream else None
    for name in ("groups", "topk_groups", "scoring", "group_score"):
        with pytest.raises(ValueError, match=f"{name} must be"):
            arn.ar_route_experts(x, 2, stream=st, **{name: value})
    with pytest.raises(ValueError, match="k must be"):
        arn.ar_route_experts(x, value, stream=st)
    with pytest.raises(ValueError, match="first must be"):
        arn.ar_w4_matvec_experts(x, ids, q, s, first=value, stream=st)
    with pytest.raises(ValueError, match="act must be"):
        arn.ar_w4_matvec_experts(x, ids, q, s, act=value, stream=st)
    with pytest.raises(ValueError, match="act must be"):
        arn.ar_w4_matvec(x, q[0], s[0], act=value, stream=st)


@pytest.mark.gpu
@pytest.mark.parametrize("own_stream", [False, True])
def test_calls_refuse_fractions(own_stream):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    st = torch.cuda.current_stream() if own_stream else None
    with pytest.raises(TypeError):
        arn.ar_route_experts(x, 2.7, stream=st)
    with pytest.raises(TypeError):
        arn.ar_route_experts(x, 2, groups=2.0, stream=st)


@pytest.mark.gpu
def test_a_row_of_more_logits_than_an_int_counts():
    """2^32 + 64 logits are not 64."""
    x = torch.empty((1, 2 ** 32 + 64), dtype=torch.bfloat16, device=DEV)
    for st in (None, torch.cuda.current_stream()):
        with pytest.raises(arn.ArError) as e:
            arn.ar_route_experts(x, 2, stream=st)
        assert e.value.status == arn.AR_ERR_UNSUPPORTED
    ids = torch.zeros((1, 2 ** 32 + 2), dtype=torch.int32, device=DEV)  # 2^32 + 2 choices are not 2
    q = torch.zeros((2, 1, 32), dtype=torch.uint8, device=DEV)
    s = torch.zeros((2, 1, 1), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((1, 2 ** 32 + 2, 1), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(arn.ArError) as e:
        arn.ar_w4_matvec_experts(x[:, :64].contiguous(), ids, q, s, out=out)
    assert e.value.status == arn.AR_ERR_UNSUPPORTED
