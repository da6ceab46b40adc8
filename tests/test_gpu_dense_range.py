"""Norms in bytes of rows near fp32's end: what the 16-bit norm of the same row
gives is what the bytes stand for."""
import math

import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_dense import BF, DEV, F32, HF
from test_gpu_experts import gen, normal

pytestmark = pytest.mark.gpu


# Clusters with one and with four packs a thread, one CTA with two and with four.
@pytest.mark.parametrize("m,H,post", [(6, 4096, False), (6, 65600, False), (700, 1024, False), (700, 1024, True),
                                      (700, 5128, False)])
@pytest.mark.parametrize("rtype", [BF, F32])
def test_squares_past_fp32(m, H, post, rtype):
    """The mean square is infinite, so the norm of a finite row is 0: zeros and a
    scale of 0, whether or not the row times the weight passes fp32's end too."""
    g = gen(m + H)
    residual = normal(g, m, H, dtype=rtype)
    partial = normal(g, m, H, dtype=BF)
    weight = (torch.randn(H, generator=g, device=DEV) * 0.1 + 3).to(BF)  # 3e38 times 3
    pw = torch.ones(H, device=DEV, dtype=BF) if post else None
    residual[1] *= 1e25
    residual[2] = 3e38
    residual[3, 5] = -3.3e38
    residual[4] = 3e38
    residual[4, H - 1] = math.inf
    residual[5] = 3e38
    residual[5, 0] = math.nan
    q, s, r = arn.ar_block_rmsnorm_i8([partial], residual, weight, 1e-6, post_weight=pw)
    y, r2 = arn.ar_block_rmsnorm([partial], residual, weight, 1e-6, post_weight=pw)
    assert torch.equal(r.view(torch.uint8), r2.view(torch.uint8))
    for row in (1, 2, 3):
        assert not bool(y[row].any())
        assert float(s[row]) == 0.0 and not bool(q[row].any()), (row, float(s[row]))
    for row in (4, 5):
        assert bool(torch.isnan(y[row]).any())
        assert math.isnan(float(s[row])) and not bool(q[row].any())
    others = torch.tensor([i for i in range(m) if i not in (1, 2, 3, 4, 5)], device=DEV)
    assert bool((s[others] > 0).all()) and bool((q[others].abs().amax(1) == 127).all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_of_the_smallest_numbers(dtype):
    """Rows that are zeros but for the type's least numbers keep their bytes."""
    m, H = 4, 1024
    residual = torch.zeros((m, H), device=DEV, dtype=dtype)
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    residual[1, 3] = tiny
    residual[2, 4], residual[2, 9] = tiny, -tiny
    weight = torch.ones(H, device=DEV, dtype=dtype)
    q, s, _ = arn.ar_block_rmsnorm_i8([torch.zeros_like(residual)], residual, weight, 1e-6)
    assert not bool(q[0].any()) and float(s[0]) == 0.0
    assert int(q[1, 3]) == 127 and int(q[1].abs().sum()) == 127
    assert int(q[2, 4]) == 127 and int(q[2, 9]) == -127
    want = tiny / math.sqrt(1e-6) / 127  # its square is far below eps
    # A bf16 row's scale (7e-40) is below fp32's normal numbers, a multiple of 2^-149:
    # the last of its roundings is off by 2^-150 there.
    assert abs(float(s[1]) - want) <= 2.0 ** -20 * want + 2.0 ** -150
