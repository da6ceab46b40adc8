"""The expert-layer kernels through the checking build: no check fires on small
and ragged shapes, and the results are the normal build's bit for bit."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_experts import DEV, gen, normal, weights4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checklib():
    from allreduce_sum_residual_gb300 import _build
    L = arn.load(_build.build(check=True))
    assert L.ar_checks_bounds() == 1 and L.ar_device_status(0, 1) == arn.AR_OK
    return L


def calls():
    g = gen(61)
    for m, E, kind, kw in ((1, 3, torch.float32, {}), (37, 60, torch.float16, dict(groups=6, topk_groups=3)),
                           (130, 256, torch.bfloat16, dict(scoring="sigmoid", groups=8, topk_groups=4,
                                                           group_score="top2"))):
        x = normal(g, m, E, dtype=kind)
        yield lambda x=x, kw=kw: arn.ar_route_experts(x, 2, **kw)
    for m, K, N, group, zeros, act in ((1, 32, 1, 32, True, "none"), (5, 1088, 515, 64, False, "none"),
                                       (16, 6144, 4096, 128, True, "silu_mul"), (33, 256, 70, 32, True, "none")):
        x, w = normal(g, m, K), weights4(g, (N,), K, group, "bf16", zeros)
        yield lambda x=x, w=w, act=act: arn.ar_w4_matvec(x, *w, act=act)
    for m, E, k, K, N in ((1, 4, 2, 128, 18), (40, 7, 3, 512, 200)):
        x, w = normal(g, m, K), weights4(g, (E, N), K, 128, "f16", False)
        ids = torch.randint(-1, E + 1, (m, k), generator=g, device=DEV, dtype=torch.int32)
        yield lambda x=x, w=w, ids=ids: arn.ar_w4_matvec_experts(x, ids, *w)
    for m, k, H in ((1, 1, 8), (19, 8, 7168), (300, 2, 1032), (2, 3, 131072)):
        y, w = normal(g, m, k, H), normal(g, m, k, dtype=torch.float32)
        res, gain = normal(g, m, H), normal(g, H)
        yield lambda y=y, w=w: arn.ar_combine(y, w)
        yield lambda y=y, w=w, res=res, gain=gain: arn.ar_combine_rmsnorm(y, w, res, gain, 1e-6, shared=res)


def test_no_check_fires_and_results_match_the_normal_build(checklib):
    normal_lib = arn.lib()
    for call in calls():
        want = call()
        arn._lib = checklib
        try:
            got = call()
            torch.cuda.synchronize()
        finally:
            arn._lib = normal_lib
        assert checklib.ar_device_status(0, 0) == arn.AR_OK
        for a, b in zip(want if isinstance(want, tuple) else (want,),
                        got if isinstance(got, tuple) else (got,)):
            assert torch.equal(a, b)
