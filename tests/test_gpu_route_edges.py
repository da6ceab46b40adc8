"""Routing where equal choices and choices closer than fp32 resolves meet."""
import math

import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import experts_ref as ref
from test_gpu_experts import DEV, TYPES, check_route, gen

pytestmark = pytest.mark.gpu


def order64(x, k, bias=None, groups=1, topk_groups=1, group_score="max"):
    """ids of sigmoid routing in 64 bits, with stable sorts (equals: lowest index)."""
    m, E = x.shape
    c = 1 / (1 + torch.exp(-x.double()))
    if bias is not None:
        c = c + bias.double()
    if topk_groups < groups:
        best = torch.sort(c.view(m, groups, E // groups), dim=2, descending=True).values
        score = best[..., 0] if group_score == "max" else best[..., 0] + best[..., 1]
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        inside = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(inside.repeat_interleave(E // groups, dim=1), c, -math.inf)
    return torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k].int()


@pytest.mark.parametrize("row,want", [
    # 17 and 18 are equal scores in fp32, not in 64 bits; the third 18 lies
    # behind the first four experts.
    ([17, 17, 18, 18, 18, 0, 0, 0], [2, 3, 4]),
    ([17, 17.125, 17.5, 17.5, 17.5, -1, -1, -1], [2, 3, 4]),
    ([18, 17, 17, 18, 17, 18, 18, 0], [0, 3, 5]),
    ([-30, -30, -29, -29, -29, -40, -40, -29], [2, 3, 4]),
    ([17, 17, 17, 17, 17, 17, 17, 17], [0, 1, 2]),
    ([17, 18, 18, 17, 18, 17, 18, 18], [1, 2, 4]),
])
@pytest.mark.parametrize("kind", sorted(TYPES))
def test_equals_of_the_last_choice_behind_near_ones(row, want, kind):
    x = torch.tensor([row], device=DEV).to(TYPES[kind])
    zero = torch.zeros(8, device=DEV)
    for bias in (zero, zero + 0.5):
        kw = dict(bias=bias, scoring="sigmoid")
        w, ids = arn.ar_route_experts(x, 3, **kw)
        assert ids.tolist() == [want]
        check_route(x, 3, w, ids, **kw)
    # Without a bias, with groups by their two best: the scores themselves.
    far = torch.full((1, 8), -90, device=DEV).to(TYPES[kind])
    x2 = torch.cat((far, x), dim=1)
    kw = dict(scoring="sigmoid", groups=2, topk_groups=1, group_score="top2")
    _, ids = arn.ar_route_experts(x2, 3, **kw)
    assert ids.tolist() == [[8 + i for i in want]]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("groups", [1, 4])
def test_few_near_choices_before_runs_of_equals(kind, groups):
    """The near, lower ones all among the first choices by index, the equals of
    the last choice going on behind them; the other experts far away."""
    g = gen(21)
    m, per = 4096, 64 // groups
    for k in (2, 3, 5, 9):
        x = torch.rand((m, 64), generator=g, device=DEV) - 4  # far below
        place = torch.rand((m, 64), generator=g, device=DEV).argsort(1)
        if groups > 1:  # all that matters in the first group
            place = torch.where(place < per, place, 64 + place)
        near = torch.randint(1, k + 1, (m, 1), generator=g, device=DEV)
        equal = torch.randint(1, k + 4, (m, 1), generator=g, device=DEV)
        rank = place.argsort(1).argsort(1)
        x = torch.where(rank < near + equal, 18.0, x)
        x = torch.where(rank < near, 16 + (rank % 3) * 0.5, x).to(TYPES[kind])
        kw = dict(groups=groups, topk_groups=1, group_score="top2")
        for bias in (torch.zeros(64, device=DEV), torch.full((64,), -0.5, device=DEV)):
            _, ids = arn.ar_route_experts(x, k, bias=bias, scoring="sigmoid", **kw)
            assert torch.equal(ids, order64(x, k, bias, **kw))


@pytest.mark.parametrize("k", [1, 3, 8, 16])
@pytest.mark.parametrize("lo,hi", [(-20, 20), (13, 30), (-60, -13)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("E", [64, 256])
def test_saturated_logits_with_many_equals(E, kind, lo, hi, k):
    """16-bit logits, many of them equal, whose scores fp32 cannot tell apart."""
    g = gen(E + k)
    x = ((torch.randn((4096, E), generator=g, device=DEV) * 16 + (lo + hi) / 2).clamp(lo, hi)
         .to(TYPES[kind]))
    for bias in (torch.zeros(E, device=DEV), torch.full((E,), 0.25, device=DEV)):
        _, ids = arn.ar_route_experts(x, k, bias=bias, scoring="sigmoid")
        assert torch.equal(ids, order64(x, k, bias))
        for score in ("max", "top2"):
            kw = dict(groups=8, topk_groups=4, group_score=score)
            _, ids = arn.ar_route_experts(x, k, bias=bias, scoring="sigmoid", **kw)
            assert torch.equal(ids, order64(x, k, bias, **kw))
    kw = dict(groups=8, topk_groups=4, group_score="top2")
    _, ids = arn.ar_route_experts(x, k, scoring="sigmoid", **kw)
    assert torch.equal(ids, order64(x, k, **kw))


def test_equals_and_near_softmax_scores():
    """The same for softmax, whose near rows are decided whole."""
    g = gen(9)
    x = (torch.randn((500, 64), generator=g, device=DEV) * 4).round().to(torch.bfloat16)
    x[:, 0] = 40  # the others' scores lie far under it
    kw = dict(bias=torch.full((64,), 0.5, device=DEV))
    w, ids = arn.ar_route_experts(x, 6, **kw)
    rw, rids = ref.route(x, 6, **kw)
    assert torch.equal(ids.cpu(), rids)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("lo,hi", [(-690, -88), (-200, -90), (-120, -60), (-89, -87), (-500, 3)])
@pytest.mark.parametrize("grouped", [False, True])
def test_sigmoid_weights_far_below_zero(kind, lo, hi, grouped):
    """Scores that fp32 cannot hold, whose weights it can: as in 64 bits.  Two
    roundings (the weight, and nothing before it but fp64): 2^-23, and half of
    fp32's smallest step."""
    g = gen(31)
    x = (torch.rand((40, 64), generator=g, device=DEV) * (hi - lo) + lo).to(TYPES[kind])
    x[1, 3:] = -math.inf   # fewer on than are chosen
    x[2] = lo              # equal weights
    x[3, ::2] = torch.finfo(TYPES[kind]).min
    kw = dict(groups=8, topk_groups=4, group_score="top2") if grouped else {}
    for bias in (None, (torch.rand(64, generator=g, device=DEV) - 0.5)):
        for renorm, scale in ((True, 1.0), (True, 2.5), (False, 1.0), (False, 1e30)):
            k = dict(bias=bias, scoring="sigmoid", renorm=renorm, scale=scale, **kw)
            w, ids = arn.ar_route_experts(x, 6, **k)
            rw, rids = ref.route(x, 6, **k)
            assert torch.equal(ids.cpu(), rids)
            # Rows with no score near fp32's end keep its roundings (2^-18).
            cx = x.gather(1, ids.long()).cpu()
            far = ((cx < -80) & (cx > -math.inf)).any(1, keepdim=True)
            tol = torch.where(far, 2.0 ** -23, 2.0 ** -18)
            err = (w.cpu().double() - rw).abs()
            assert bool((err <= tol * rw.abs() + 2.0 ** -150).all()), float((err / rw.abs()).nan_to_num().max())


def test_sigmoid_weights_where_64_bits_have_none():
    """Logits of the type's lowest value: a score of 0 in 64 bits too, and
    weights of 0 where there is nothing else."""
    for kind in TYPES.values():
        x = torch.full((2, 16), torch.finfo(kind).min, device=DEV, dtype=kind)
        x[1, 5] = -600
        for bias in (None, torch.zeros(16, device=DEV)):
            w, ids = arn.ar_route_experts(x, 4, bias=bias, scoring="sigmoid")
            assert ids.tolist() == [[0, 1, 2, 3], [5, 0, 1, 2]]
            assert w.tolist() == [[0.0] * 4, [1.0, 0.0, 0.0, 0.0]]
