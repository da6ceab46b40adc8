"""The expert-layer calls in one step (_binding.so) and the long way through
ctypes: the same checks, the same outputs."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from allreduce_sum_residual_gb300 import experts
from test_gpu_experts import DEV, gen, normal, weights4

pytestmark = pytest.mark.gpu


def operands():
    g = gen(71)
    m, E, k, K, N, H = 5, 12, 3, 256, 40, 64
    ids = torch.randint(-1, E + 1, (m, k), generator=g, device=DEV, dtype=torch.int32)
    logits, bias = normal(g, m, E), normal(g, E, dtype=torch.float32)
    x, xk = normal(g, m, K), normal(g, m, k, K)
    w, we = weights4(g, (N,), K, 64, "bf16", True), weights4(g, (E, N), K, 128, "f32", False)
    y, rows = normal(g, m, k, H), normal(g, 9, H)
    slots = torch.randint(-1, 10, (m, k), generator=g, device=DEV, dtype=torch.int32)
    cw, res, gain = normal(g, m, k, dtype=torch.float32), normal(g, m, H), normal(g, H)
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    new = lambda *shape, dtype=bf: torch.full(shape, -7, device=DEV, dtype=dtype)
    wide = normal(g, m, E + 5)[:, :E]
    return {
        "route": lambda **s: arn.ar_route_experts(logits, k, **s),
        "route_all": lambda **s: arn.ar_route_experts(
            wide, k, bias=bias, scoring="sigmoid", groups=4, topk_groups=2, group_score="top2",
            renorm=False, scale=2, weights=new(m, k, dtype=f32), ids=new(m, k, dtype=i32), **s),
        "matvec": lambda **s: arn.ar_w4_matvec(x, *w, **s),
        "matvec_out": lambda **s: arn.ar_w4_matvec(x, *w, act="silu_mul", out=new(m, N // 2), **s),
        "experts": lambda **s: arn.ar_w4_matvec_experts(x, ids, *we, **s),
        "experts_pairs": lambda **s: arn.ar_w4_matvec_experts(
            xk, ids, *we, act=arn.AR_ACT_SILU_MUL, first=1, out=new(m, k, N // 2), **s),
        "combine": lambda **s: arn.ar_combine(y, cw, **s),
        "combine_slots": lambda **s: arn.ar_combine(rows, cw, shared=res, slots=slots,
                                                    out=new(m, H), **s),
        "norm": lambda **s: arn.ar_combine_rmsnorm(y, cw, res, gain, 1e-6, **s),
        "norm_all": lambda **s: arn.ar_combine_rmsnorm(rows, cw, res, gain, 1, shared=res, slots=slots,
                                                       out=new(m, H), residual_out=new(m, H), **s),
    }


def as_tuple(r):
    return r if isinstance(r, tuple) else (r,)


def test_one_step_is_the_long_way(monkeypatch):
    long_way = experts._call
    for name, call in operands().items():
        used = []
        monkeypatch.setattr(experts, "_call", lambda *a: used.append(a) or long_way(*a))
        want = as_tuple(call(stream=torch.cuda.current_stream()))
        assert len(used) == 1, name
        got = as_tuple(call())
        assert len(used) == 1, f"{name}: not made in one step"
        for a, b in zip(want, got):
            assert a.shape == b.shape and a.dtype == b.dtype and a.device == b.device
            assert torch.equal(a, b), name
            assert not (b.float() == -7).any(), f"{name}: an output not written"


def test_one_step_runs_on_the_current_stream_and_in_a_graph():
    calls = operands()
    want = {name: as_tuple(call()) for name, call in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = {name: as_tuple(call()) for name, call in calls.items()}
    graph.replay()
    torch.cuda.synchronize()
    for name in calls:
        for a, b in zip(want[name], got[name]):
            assert torch.equal(a, b), name


def test_what_is_wrong_is_named():
    g = gen(72)
    x, w = normal(g, 2, 256), weights4(g, (8,), 256, 64, "bf16", False)
    with pytest.raises(ValueError, match="q must be on"):
        arn.ar_w4_matvec(x, w[0].cpu(), *w[1:])
    with pytest.raises(ValueError, match="act must be one of"):
        arn.ar_w4_matvec(x, *w, act="gelu")
    with pytest.raises(ValueError, match="out must have shape"):
        arn.ar_w4_matvec(x, *w, out=normal(g, 2, 9))
    with pytest.raises(arn.ArError) as e:
        arn.ar_w4_matvec(x, *w, act=9)
    assert e.value.status == arn.AR_ERR_ARG
    with pytest.raises(arn.ArError) as e:
        arn.ar_route_experts(x, 300)
    assert e.value.status == arn.AR_ERR_UNSUPPORTED
    with pytest.raises(TypeError, match="bias must be a torch.Tensor"):
        arn.ar_route_experts(x, 2, bias=3)
    with pytest.raises(TypeError):
        arn.ar_combine(None, None)
    with pytest.raises(TypeError, match="arguments"):
        experts._fast().combine(x)
