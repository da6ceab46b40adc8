"""ExpertLayer: the calls of an expert layer in a row, for one rank and for the
ranks of a group."""
import math

import pytest
import torch

import experts_ref as ref

DEV = "cuda:0"


def make(g, E=16, H=512, I=128, shared=True):
    def w4(lead, K, group):
        q = torch.randint(0, 256, (*lead, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s = ((torch.rand((*lead, K // group), generator=g, device=DEV) - 0.4) / math.sqrt(K)).bfloat16()
        return q, s, None
    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()
    w = dict(router=normal(E, H, std=0.05), up=w4((E, 2 * I), H, 64), down=w4((E, H), I, 32))
    sh = dict(shared_up=w4((2 * I,), H, 128), shared_down=w4((H,), I, 128)) if shared else {}
    return w, sh, normal


def exact(x, y, weights, shared, residual, weight, k):
    r, mag = ref.combine(y, weights, shared, None, x.shape[0] * k, k)
    return r + residual.double(), mag + residual.double().abs()


class OneProcessGroup:
    """Stands in for the group object: the ranks of one process take turns,
    the epilogue runs over all partials once the last has written its own."""

    def __init__(self, world, m, H):
        self.partials = [torch.zeros((m, H), dtype=torch.bfloat16, device=DEV) for _ in range(world)]
        self.rank = 0

    def partial(self, m):
        return self.partials[self.rank][:m]

    def __call__(self, residual, weight, eps):
        import allreduce_sum_residual_gb300 as arn
        m = residual.shape[0]
        return arn.ar_rmsnorm([p[:m] for p in self.partials], residual, weight, eps)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5, 33])
def test_one_rank(m):
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    w, sh, normal = make(g)
    bias = torch.randn(16, generator=g, device=DEV) * 0.1
    layer = ExpertLayer(**w, **sh, top_k=3, bias=bias, scoring="sigmoid", groups=4, topk_groups=2,
                        group_score="top2", scale=2.5)
    x, residual, weight = normal(m, 512), normal(m, 512), normal(512)
    out, rout = layer(x, residual, weight, 1e-6)
    y, weights, shared = layer.outputs(x)
    r, mag = exact(x, y, weights, shared, residual, weight, 3)
    ref.close(rout, r, 4 * ref.F32 * mag)
    ref.close(out, *ref.norm(r, 4 * ref.F32 * mag, weight, 1e-6))
    ref.close(layer.partial(x), *(lambda s, a: (s, 3 * ref.F32 * a))(
        *ref.combine(y, weights, shared, None, m * 3, 3)))


@pytest.mark.gpu
def test_ranks_of_a_group_hold_the_experts_between_them():
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    m, world = 6, 4
    w, _, normal = make(g, shared=False)
    x, residual, weight = normal(m, 512), normal(m, 512), normal(512)
    group = OneProcessGroup(world, 8, 512)
    r, mag = residual.double(), residual.double().abs()
    for rank in range(world):
        sl = slice(4 * rank, 4 * rank + 4)
        layer = ExpertLayer(w["router"], [t if t is None else t[sl] for t in w["up"]],
                            [t if t is None else t[sl] for t in w["down"]], 3, first=4 * rank,
                            group=group)
        group.rank = rank
        out, rout = layer(x, residual, weight, 1e-6)
        y, weights, _ = layer.outputs(x)
        s, a = ref.combine(y, weights, None, None, m * 3, 3)
        r, mag = r + s, mag + a
    err = world * ref.BF16 * mag + 16 * ref.F32 * mag  # every partial rounds once to bf16
    ref.close(rout, r, err)
    ref.close(out, *ref.norm(r, err, weight, 1e-6))


@pytest.mark.gpu
def test_replays_from_a_graph():
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    w, sh, normal = make(g)
    layer = ExpertLayer(**w, **sh, top_k=2)
    xs = [normal(4, 512) for _ in range(3)]
    residual, weight = normal(4, 512), normal(512)
    want = [layer(x, residual, weight, 1e-6) for x in xs]
    live = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(live, residual, weight, 1e-6)
    for x, (o, r) in zip(xs, want):
        live.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], r)


def test_refusals():
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    router = torch.zeros((8, 64), dtype=torch.bfloat16)
    up = (torch.zeros((4, 64, 32), dtype=torch.uint8), torch.zeros((4, 64, 1)), None)
    down = (torch.zeros((4, 64, 16), dtype=torch.uint8), torch.zeros((4, 64, 1)), None)
    with pytest.raises(ValueError, match="both"):
        ExpertLayer(router, up, down, 2, shared_up=up)
    with pytest.raises(ValueError, match="among"):
        ExpertLayer(router, up, down, 2, first=5)
    with pytest.raises(ValueError, match="router"):
        ExpertLayer(router[0], up, down, 2)
    assert ExpertLayer(router, up, down, 2, first=4).first == 4
