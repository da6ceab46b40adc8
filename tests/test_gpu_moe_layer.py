"""ExpertLayer against a layer written out in 64 bits from its weights alone,
on one rank and on the ranks of a group."""
import math

import pytest
import torch

import experts_ref as ref
from test_moe import DEV, OneProcessGroup

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 128, 16, 3
ROUTING = [dict(), dict(scoring="sigmoid", groups=4, topk_groups=2, group_score="top2", scale=2.5),
           dict(scoring="sigmoid", renorm=False)]


def weights(g, bias):
    def w4(lead, k, group, zeros):
        q = torch.randint(0, 256, (*lead, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s = ((torch.rand((*lead, k // group), generator=g, device=DEV) - 0.4) / math.sqrt(k)).bfloat16()
        z = (torch.randint(0, 16, (*lead, k // group), generator=g, device=DEV, dtype=torch.uint8)
             if zeros else None)
        return q, s, z
    w = dict(router=(torch.randn((E, H), generator=g, device=DEV) * 0.05).bfloat16(),
             up=w4((E, 2 * I), H, 64, True), down=w4((E, H), I, 32, False))
    shared = dict(shared_up=w4((2 * I,), H, 128, False), shared_down=w4((H,), I, 128, True))
    return w, shared, (torch.randn(E, generator=g, device=DEV) * 0.2 if bias else None)


def mlp(x, up, down):
    """(rows, error) of one expert: up and gate, rounded to bf16, down, rounded."""
    wu = ref.unpack(*up)
    y, e = ref.product(x, *up)
    gate, value = x.double() @ wu[:I].T, x.double() @ wu[I:].T
    assert torch.equal(y, torch.cat((gate, value), 1))
    h = gate / (1 + torch.exp(-gate)) * value
    _, eh = ref.act(y, e, "silu_mul")
    eh = ref.BF16 * h.abs() + (1 + ref.BF16) * eh
    wd = ref.unpack(*down).abs()
    out = h @ ref.unpack(*down).T
    e2 = (h.abs() + eh) @ wd.T * 512 * ref.F32 + eh @ wd.T   # far more roundings than K / 16 + 128
    return out, ref.BF16 * out.abs() + (1 + ref.BF16) * e2


def layer64(x, w, shared, bias, ids, residual, kw):
    """(sum with the residual, its error, weights) for the experts `ids`."""
    logits = x.double() @ w["router"].double().T
    score = (torch.softmax(logits, 1) if kw.get("scoring", "softmax") == "softmax"
             else 1 / (1 + torch.exp(-logits)))
    weight = score.gather(1, ids.long())
    if kw.get("renorm", True):
        weight = weight / weight.sum(1, keepdim=True)
    weight = weight * kw.get("scale", 1.0)
    r, err = residual.double(), torch.zeros((x.shape[0], H), dtype=torch.float64, device=DEV)
    mag = r.abs()
    if shared:
        y, e = mlp(x, shared["shared_up"], shared["shared_down"])
        r, err, mag = r + y, err + e, mag + y.abs()
    part = lambda t, i: tuple(None if a is None else a[i] for a in t)
    for i in range(E):
        rows, at = (ids == i).nonzero(as_tuple=True)
        if len(rows):
            y, e = mlp(x[rows], part(w["up"], i), part(w["down"], i))
            a = weight[rows, at].unsqueeze(1)
            r[rows] += a * y
            mag[rows] += (a * y).abs()
            # Logits as fp32 sums are off by 2^-14 at most here, and so are the weights, relatively.
            err[rows] += a * e + 2.0 ** -13 * (a * y).abs()
    return r, err + 16 * ref.F32 * mag


def check_ids(x, w, bias, ids, kw):
    """The experts are the 64-bit form's but for choices closer than fp32
    logits tell apart."""
    logits = x.double() @ w["router"].double().T
    _, want = ref.route(logits, K, bias=bias, **kw)
    differ = (ids.cpu().sort(1).values != want.sort(1).values).any(1)
    assert int(differ.sum()) == 0 or int(differ.sum()) <= x.shape[0] // 50


@pytest.mark.parametrize("m", [1, 7, 33])
@pytest.mark.parametrize("case", range(len(ROUTING)))
@pytest.mark.parametrize("with_shared", [False, True])
def test_a_layer_and_its_ranks_against_64_bits(m, case, with_shared):
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(100 * m + case)
    w, shared, bias = weights(g, case > 0)
    shared = shared if with_shared else {}
    kw = ROUTING[case]
    x, residual, gain = ((torch.randn((m, H), generator=g, device=DEV)).bfloat16() for _ in range(3))
    gain = gain[0].contiguous()
    one = ExpertLayer(**w, **shared, top_k=K, bias=bias, **kw)
    _, ids = one.route(x)
    check_ids(x, w, bias, ids, kw)
    r, err = layer64(x, w, shared, bias, ids, residual, kw)
    out, rout = one(x, residual, gain, 1e-6)
    ref.close(rout, r, err)
    ref.close(out, *ref.norm(r, err, gain, 1e-6))

    world = 4
    group = OneProcessGroup(world, max(m, 8), H)
    share = lambda t, n: tuple(None if a is None else a[n].contiguous() for a in t)
    for rank in range(world):
        n = slice(4 * rank, 4 * rank + 4)
        sh = shared if rank == 1 else {}  # one rank adds the shared expert
        layer = ExpertLayer(w["router"], share(w["up"], n), share(w["down"], n), K, first=4 * rank,
                            group=group, bias=bias, **sh, **kw)
        group.rank = rank
        out4, rout4 = layer(x, residual, gain, 1e-6)
    # Every rank's partial rounds once more.
    mag = r.abs() + residual.double().abs()
    err4 = err + 16 * ref.F32 * mag + sum(ref.BF16 * (1 + ref.BF16) * p[:m].double().abs()
                                          for p in group.partials)
    ref.close(rout4, r, err4)
    ref.close(out4, *ref.norm(r, err4, gain, 1e-6))
    assert bool(((rout4.double() - rout.double()).abs() <= err + err4 + 2 * ref.BF16 * r.abs()).all())


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_logits_keep_what_bf16_would_lose(kind):
    """Experts whose logits differ by less than bf16 resolves: the larger one
    is chosen, also where it has the higher index."""
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    w, _, _ = weights(g, False)
    x = torch.zeros((E - 1, H), dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1] = 64, 2.0 ** -4
    router = torch.zeros((E, H), dtype=kind, device=DEV)
    router[:, 0] = 1                       # logits of 64 ...
    router[:, 1] = torch.arange(E, device=DEV) / 16   # ... and up to 2^-4 more
    layer = ExpertLayer(router, w["up"], w["down"], K)
    _, ids = layer.route(x)
    assert ids.tolist() == [[E - 1, E - 2, E - 3]] * (E - 1)


def test_an_fp32_router_and_parameters():
    """A router in fp32 is used as it is; parameters and inputs that autograd
    follows are read like others; no token at all."""
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    w, _, _ = weights(g, False)
    x = torch.randn((9, H), generator=g, device=DEV).bfloat16()
    residual, gain = x.roll(1, 0).contiguous(), x[0].clone()
    want = ExpertLayer(**w, top_k=K)(x, residual, gain, 1e-6)
    fine = torch.randn((E, H), generator=g, device=DEV) * 0.05
    weights32, ids = ExpertLayer(fine, w["up"], w["down"], K).route(x)
    rw, rids = ref.route(x.double() @ fine.double().T, K)
    assert torch.equal(ids.cpu(), rids) and bool(((weights32.cpu() - rw).abs() <= 1e-5).all())
    for router in (w["router"], w["router"].float()):
        layer = ExpertLayer(torch.nn.Parameter(router), w["up"], w["down"], K)
        xg = x.clone().requires_grad_(True)
        got = layer(xg, residual, gain, 1e-6)
        if router is w["router"]:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        # fp32 products add up in another order: 512 terms, each way off by 512 2^-24 of
        # sum |x router| < 128, so weights by less than 2^-7.
        (wa, ia), (wb, ib) = layer.route(xg), ExpertLayer(**w, top_k=K).route(x)
        assert torch.equal(ia, ib) and bool(((wa - wb).abs() <= 2.0 ** -7).all())
        none = layer(x[:0], residual[:0], gain, 1e-6)
        assert [t.shape for t in none] == [(0, H), (0, H)]
    with pytest.raises(ValueError, match="router must be"):
        ExpertLayer(w["router"].half(), w["up"], w["down"], K)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_autocast_leaves_the_logits_alone(kind):
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    w, _, _ = weights(g, False)
    layer = ExpertLayer(w["router"].to(kind), w["up"], w["down"], K)
    x = torch.randn((33, H), generator=g, device=DEV).bfloat16()
    want = layer.route(x)
    for to in (torch.bfloat16, torch.float16):
        with torch.autocast("cuda", dtype=to):
            got = layer.route(x)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
