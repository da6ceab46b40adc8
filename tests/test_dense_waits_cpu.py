"""The self-test of the 8-bit products' waits: what it refuses."""
import allreduce_sum_residual_gb300 as arn


def test_refusals():
    for device, limit_us in ((-1, 1000), (64, 1000), (0, 0), (0, 100001)):
        assert arn.ar_selftest_i8_waits(device, limit_us) == arn.AR_ERR_ARG
