"""The 4-bit products through the checking build at the shapes that walk all
of their shared memory: several phases, many column sets, teams of every
size, ranges of items over many blocks, outputs taken again."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_experts import DEV, gen, normal, weights4
from test_gpu_experts_check import checklib  # noqa: F401

pytestmark = pytest.mark.gpu

DENSE = [  # m, K, N, group, zeros, act, scale
    (1, 7168, 2048, 128, False, "none", 1), (1, 32736, 50, 32, True, "none", 1),
    (3, 1024, 50000, 64, True, "none", 1), (16, 32768, 64, 32, True, "none", 1),
    (64, 32768, 40, 128, False, "silu_mul", 1), (16, 6144, 20480, 128, False, "silu_mul", 1),
    (33, 512, 66, 64, False, "silu_mul", 1), (16, 4128, 1001, 32, True, "none", 1),
    (9, 8192, 300, 64, True, "silu_mul", 2.0 ** 122), (40, 640, 5000, 128, False, "none", 2.0 ** 124),
]
EXPERTS = [  # m, E, k, K, N, group, zeros, act, x per pair, scale
    (4096, 300, 1, 64, 20, 32, False, "none", False, 1), (256, 9, 16, 64, 18, 64, False, "none", True, 1),
    (16, 3, 2, 16384, 40, 64, True, "none", True, 1), (24, 64, 8, 2048, 4096, 128, False, "silu_mul", False, 1),
    (16, 512, 16, 128, 48, 128, False, "none", False, 1), (16, 64, 8, 7168, 40, 128, False, "silu_mul", False, 1),
    (64, 2, 1, 1152, 2000, 128, True, "none", False, 1), (1, 64, 8, 7168, 256, 128, False, "none", False, 1),
    (40, 5, 2, 384, 700, 64, True, "none", True, 2.0 ** 122),
]


def both(checklib, call):  # noqa: F811
    normal_lib = arn.lib()
    want = call()
    arn._lib = checklib
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        arn._lib = normal_lib
    assert checklib.ar_device_status(0, 1) == arn.AR_OK
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("m,K,N,group,zeros,act,scale", DENSE)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_dense(checklib, kind, m, K, N, group, zeros, act, scale):  # noqa: F811
    g = gen(m + K)
    x = normal(g, m, K)
    q, s, z = weights4(g, (N,), K, group, kind, zeros)
    both(checklib, lambda: arn.ar_w4_matvec(x, q, s * scale, zeros=z, act=act))


@pytest.mark.parametrize("m,E,k,K,N,group,zeros,act,per_pair,scale", EXPERTS)
def test_experts(checklib, m, E, k, K, N, group, zeros, act, per_pair, scale):  # noqa: F811
    g = gen(m + E)
    x = normal(g, m, k, K) if per_pair else normal(g, m, K)
    ids = torch.randint(-1, E + 1, (m, k), generator=g, device=DEV, dtype=torch.int32)
    q, s, z = weights4(g, (E, N), K, group, "bf16", zeros)
    both(checklib, lambda: arn.ar_w4_matvec_experts(x, ids, q, s * scale, zeros=z, act=act))
    ids[:] = E - 1  # one expert alone
    both(checklib, lambda: arn.ar_w4_matvec_experts(x, ids, q, s * scale, zeros=z, act=act))
