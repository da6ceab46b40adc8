"""The ways out of the 8-bit products' kernels when a wait runs out: on valid
operands, with loads that stop, as the library's self-test makes them."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_dense import DEV, F32, bytes_
from test_gpu_experts import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [500, 3000])
def test_waits_that_run_out_end_with_a_status_and_leave_nothing_behind(limit_us):
    g = gen(1)
    x, w = bytes_(g, 200, 2048), bytes_(g, 512, 2048)
    one = torch.ones(512, device=DEV)
    want = arn.ar_i8_matmul(x, one[:200], w, one, dtype=F32)
    assert arn.ar_selftest_i8_waits(0, limit_us) == arn.AR_OK
    assert arn.ar_device_status(0) == arn.AR_OK
    assert torch.equal(arn.ar_i8_matmul(x, one[:200], w, one, dtype=F32), want)
