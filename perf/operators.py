"""The expert-layer operators, as cases to measure.

Four operators: routing to experts, products with 4-bit weights (dense, and
of the routed experts), and the weighted sum of the experts' outputs with
the residual add and RMSNorm.  ``run`` computes each in its plain form
(elementary torch operations) or, where ``own`` is true, through the
package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
LOGITS = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------- cases

def _route(name, m, E, k, scoring="softmax", groups=1, topk_groups=1, group_score="max",
           bias=False, renorm=True, scale=1.0, dtype="bfloat16", masked=0.0):
    return dict(name=name, op="route", m=m, E=E, k=k, scoring=scoring, groups=groups,
                topk_groups=topk_groups, group_score=group_score, bias=bias, renorm=renorm,
                scale=scale, dtype=dtype, masked=masked)


def _matvec(name, m, K, N, group=128, zeros=False, scales="bfloat16", act="none"):
    return dict(name=name, op="matvec", m=m, K=K, N=N, group=group, zeros=zeros, scales=scales,
                act=act)


def _experts(name, m, E, k, K, N, group=128, zeros=False, scales="bfloat16", act="none",
             per_pair=False, missing=0.0):
    return dict(name=name, op="experts", m=m, E=E, k=k, K=K, N=N, group=group, zeros=zeros,
                scales=scales, act=act, per_pair=per_pair, missing=missing)


def _combine(name, m, k, H, norm=True, shared=False, slots=False, missing=0.0):
    return dict(name=name, op="combine", m=m, k=k, H=H, norm=norm, shared=shared, slots=slots,
                missing=missing)


def listed():
    return [
        # One decode step of a small batch: 8 of 128 experts per token.
        _route("route_decode", 16, 128, 8),
        # A long prompt: sigmoid scores with a balance bias, 4 of 8 groups kept by their two
        # best experts, renormalised and scaled.
        _route("route_prompt_groups", 16384, 256, 8, scoring="sigmoid", groups=8, topk_groups=4,
               group_score="top2", bias=True, scale=2.5, dtype="float32"),
        # A ragged chunk with an odd expert count, some experts switched off (-inf logits).
        _route("route_ragged", 1023, 60, 6, groups=6, topk_groups=3, renorm=False,
               dtype="float16", masked=0.1),
        # One token through a square projection of the decode hidden size.
        _matvec("matvec_token", 1, 7168, 7168),
        # A decode batch through a gate-up projection with its activation: weights above L2 size
        # for two states.
        _matvec("matvec_gate_up", 16, 6144, 32768, act="silu_mul"),
        # Odd sizes: a K that ends inside a tile, an odd number of outputs, zero points.
        _matvec("matvec_ragged", 5, 4128, 1001, group=32, zeros=True, scales="float32"),
        # One token through the gate-up products of its 8 experts.
        _experts("experts_gate_up_token", 1, 64, 8, 7168, 4096, act="silu_mul"),
        # A decode batch through the down products: most experts have one to four tokens.
        _experts("experts_down_batch", 32, 128, 8, 1024, 6144, per_pair=True),
        # Odd sizes, and a quarter of the choices on other ranks.
        _experts("experts_ragged", 7, 17, 3, 1056, 515, group=32, zeros=True, missing=0.25),
        # The layer's end in a decode step, with a shared expert.
        _combine("combine_norm_decode", 16, 8, 7168, shared=True),
        # The layer's end for a prompt whose expert outputs lie in expert order.
        _combine("combine_norm_prompt", 8192, 8, 6144, slots=True),
        # A rank's partial: only the choices that this rank computed.
        _combine("combine_partial", 777, 6, 7168, norm=False, slots=True, missing=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "matvec", "experts", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 6, 8))
        E = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        c = _route(None, _log(rng, 1, 16384), E, k, rng.choice(("softmax", "sigmoid")), groups,
                   topk_groups, rng.choice(("max", "top2")), rng.random() < 0.5,
                   rng.random() < 0.7, rng.choice((1.0, 2.5)), rng.choice(sorted(LOGITS)),
                   rng.choice((0.0, 0.0, 0.1)))
    elif op == "matvec":
        group = rng.choice((32, 64, 128))
        act = rng.choice(("none", "silu_mul"))
        N = _log(rng, 256, 16384)
        c = _matvec(None, _log(rng, 1, 32), group * _log(rng, 512 // group, 8192 // group),
                    N + N % 2 if act == "silu_mul" else N, group, rng.random() < 0.5,
                    rng.choice(sorted(LOGITS)), act)
    elif op == "experts":
        group = rng.choice((32, 64, 128))
        act = rng.choice(("none", "silu_mul"))
        E, N = rng.randint(8, 64), _log(rng, 256, 4096)
        c = _experts(None, _log(rng, 1, 24), E, rng.randint(1, 8),
                     group * _log(rng, 512 // group, 4096 // group),
                     N + N % 2 if act == "silu_mul" else N, group, rng.random() < 0.5,
                     rng.choice(sorted(LOGITS)), act, rng.random() < 0.5,
                     rng.choice((0.0, 0.0, 0.5)))
    else:
        c = _combine(None, _log(rng, 1, 4096), rng.randint(1, 8), 8 * _log(rng, 128, 1024),
                     rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.5,
                     rng.choice((0.0, 0.0, 0.5)))
        c["missing"] = c["missing"] if c["slots"] else 0.0
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _weights4(g, shape, K, case):
    """Packed 4-bit weights [*shape, K/2] with their group scales and zero points.  The scales
    make the outputs about as large as the inputs."""
    dev, ng = g.device, K // case["group"]
    q = torch.randint(0, 256, (*shape, K // 2), generator=g, device=dev, dtype=torch.uint8)
    s = (torch.rand((*shape, ng), generator=g, device=dev) + 0.5) / (4.6 * math.sqrt(K))
    z = (torch.randint(5, 12, (*shape, ng), generator=g, device=dev, dtype=torch.uint8)
         if case["zeros"] else None)
    return q, s.to(LOGITS[case["scales"]]), z


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = g.device

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    def chosen(m, E, k):
        return torch.rand((m, E), generator=g, device=dev).topk(k, dim=1).indices.int()

    st = dict(case=case)
    if case["op"] == "route":
        m, E = case["m"], case["E"]
        st["logits"] = normal(m, E, std=1.5, dtype=LOGITS[case["dtype"]])
        if case["masked"]:
            off = torch.rand(E, generator=g, device=dev) < case["masked"]
            st["logits"][:, off] = -math.inf
        st["bias"] = normal(E, std=0.1, dtype=torch.float32) if case["bias"] else None
    elif case["op"] == "matvec":
        st["x"] = normal(case["m"], case["K"])
        st["q"], st["s"], st["z"] = _weights4(g, (case["N"],), case["K"], case)
    elif case["op"] == "experts":
        m, E, k, K = case["m"], case["E"], case["k"], case["K"]
        st["x"] = normal(m, k, K) if case["per_pair"] else normal(m, K)
        st["ids"] = chosen(m, E, k)
        if case["missing"]:
            st["ids"][torch.rand((m, k), generator=g, device=dev) < case["missing"]] = -1
        st["q"], st["s"], st["z"] = _weights4(g, (E, case["N"]), K, case)
    else:
        m, k, H = case["m"], case["k"], case["H"]
        if case["slots"]:
            slots = torch.randperm(m * k, generator=g, device=dev)
            live = torch.rand(m * k, generator=g, device=dev) >= case["missing"]
            # The rows that are not computed here have no place in y.
            place = torch.cumsum(live.int(), 0) - 1
            st["slots"] = torch.where(live, place, -1)[slots].view(m, k).int()
            st["y"] = normal(max(1, int(live.sum())), H)
        else:
            st["slots"] = None
            st["y"] = normal(m, k, H)
        w = torch.rand((m, k), generator=g, device=dev) + 0.1
        st["weights"] = w / w.sum(1, keepdim=True)
        st["shared"] = normal(m, H) if case["shared"] else None
        if case["norm"]:
            st["residual"] = normal(m, H)
            st["weight"] = (torch.randn(H, generator=g, device=dev) * 0.1 + 1).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- the plain forms

def _plain_route(st):
    case = st["case"]
    m, E, k, G = case["m"], case["E"], case["k"], case["groups"]
    x = st["logits"].double()  # choices next to a border are decided in 64 bits
    off = x == -math.inf
    if case["scoring"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        s = e / e.sum(1, keepdim=True)
        s = torch.where(off, 0.0, s)
    else:
        s = 1 / (1 + torch.exp(-x))
    if st["bias"] is not None:
        c = s + st["bias"].double()
    else:
        c = x if case["group_score"] == "max" or G == 1 else s  # the scores' order is the logits'
    c = torch.where(off, -math.inf, c)
    if G > 1:
        best = torch.sort(c.view(m, G, E // G), dim=2, descending=True).values
        score = best[..., 0] if case["group_score"] == "max" else best[..., 0] + best[..., 1]
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        inside = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        inside = inside.repeat_interleave(E // G, dim=1)
        c = torch.where(inside, c.clamp(min=-1e300), -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return (w * case["scale"]).float(), ids.int()


def _dequantised(q, s, z, group):
    low_high = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()
    w = low_high.unflatten(-1, (-1, group))
    w = w - (8.0 if z is None else z.float().unsqueeze(-1))
    return (w * s.float().unsqueeze(-1)).flatten(-2)


def _activated(y, act):
    if act == "none":
        return y
    gate, up = y.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_matvec(st):
    case = st["case"]
    w = _dequantised(st["q"], st["s"], st["z"], case["group"])
    return _activated(st["x"].float() @ w.T, case["act"]).bfloat16()


def _plain_experts(st):
    case = st["case"]
    m, k = case["m"], case["k"]
    ids = st["ids"].flatten().long()
    here = ids >= 0
    ids = ids.clamp(min=0)
    z = st["z"][ids] if st["z"] is not None else None
    w = _dequantised(st["q"][ids], st["s"][ids], z, case["group"])
    x = st["x"].flatten(0, 1) if case["per_pair"] else st["x"].repeat_interleave(k, dim=0)
    y = torch.matmul(w, x.float().unsqueeze(-1)).squeeze(-1)
    y = torch.where(here.unsqueeze(-1), _activated(y, case["act"]), 0.0)
    return y.bfloat16().view(m, k, -1)


def _plain_combine(st):
    case = st["case"]
    y = st["y"]
    w = st["weights"]
    if st["slots"] is not None:
        w = torch.where(st["slots"] >= 0, w, 0.0)
        y = y[st["slots"].clamp(min=0).long()]
    r = (w.unsqueeze(-1) * y.float()).sum(1)
    if st["shared"] is not None:
        r = r + st["shared"].float()
    if not case["norm"]:
        return r.bfloat16()
    r = r + st["residual"].float()
    out = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * st["weight"].float()
    return out.bfloat16(), r.bfloat16()


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        plain = {"route": _plain_route, "matvec": _plain_matvec, "experts": _plain_experts,
                 "combine": _plain_combine}
        return plain[op](state)
    import allreduce_sum_residual_gb300 as arn
    if op == "route":
        return arn.ar_route_experts(
            state["logits"], case["k"], bias=state["bias"], scoring=case["scoring"],
            groups=case["groups"], topk_groups=case["topk_groups"],
            group_score=case["group_score"], renorm=case["renorm"], scale=case["scale"])
    if op == "matvec":
        return arn.ar_w4_matvec(state["x"], state["q"], state["s"], zeros=state["z"],
                                act=case["act"])
    if op == "experts":
        return arn.ar_w4_matvec_experts(state["x"], state["ids"], state["q"], state["s"],
                                        zeros=state["z"], act=case["act"])
    if case["norm"]:
        return arn.ar_combine_rmsnorm(state["y"], state["weights"], state["residual"],
                                      state["weight"], EPS, shared=state["shared"],
                                      slots=state["slots"])
    return arn.ar_combine(state["y"], state["weights"], shared=state["shared"],
                          slots=state["slots"])


# ---------------------------------------------------------------- what a pass has to do

def work(case):
    op = case["op"]
    if op == "route":
        m, E = case["m"], case["E"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": m * E * size + m * case["k"] * 8 + (4 * E if case["bias"] else 0),
                "flops": 6 * m * E}
    if op in ("matvec", "experts"):
        K, N, m = case["K"], case["N"], case["m"]
        ng = K // case["group"]
        size = 4 if case["scales"] == "float32" else 2
        matrix = N * K // 2 + N * ng * (size + (1 if case["zeros"] else 0))
        width = N // 2 if case["act"] == "silu_mul" else N
        if op == "matvec":
            return {"bytes": matrix + 2 * m * K + 2 * m * width, "flops": 2 * m * N * K}
        E, k = case["E"], case["k"]
        hit = (k / E) * (1 - case["missing"])  # an expert's chance to be one token's here
        distinct = E * (1 - (1 - hit) ** m)
        pairs = m * k
        rows = pairs if case["per_pair"] else m
        return {"bytes": distinct * matrix + 2 * rows * K + 2 * pairs * width + 4 * pairs,
                "flops": 2 * pairs * (1 - case["missing"]) * N * K}
    m, k, H = case["m"], case["k"], case["H"]
    rows = k * (1 - case["missing"]) + (1 if case["shared"] else 0) + (3 if case["norm"] else 1)
    return {"bytes": 2 * m * H * rows + m * k * (8 if case["slots"] else 4)
            + (2 * H if case["norm"] else 0), "flops": 2 * m * H * (k + (4 if case["norm"] else 0))}


# ---------------------------------------------------------------- 64 bits, from the definition

def _exact_route(st, case):
    x, k = st["logits"].double(), case["k"]
    m, E = x.shape
    G = case["groups"]
    alive = torch.isfinite(x)
    if case["scoring"] == "softmax":
        s = torch.where(alive, torch.softmax(x, dim=1), 0.0)
    else:
        s = torch.sigmoid(x)
    choice = s if st["bias"] is None else s + st["bias"].double()
    choice = choice.masked_fill(~alive, -1e9)
    if G > 1:
        per = choice.reshape(m, G, E // G)
        first = per.max(2)
        score = first.values
        if case["group_score"] == "top2":
            score = score + per.scatter(2, first.indices.unsqueeze(2), -1e9).max(2).values
        score = score.masked_fill(score < -1e8, -math.inf)  # too few experts that are on
        for _ in range(G - case["topk_groups"]):  # drop the worst group; the last of equals goes
            worst = G - 1 - score.flip(1).argmin(1)
            score[torch.arange(m), worst] = math.inf
            choice.view(m, G, E // G)[torch.arange(m), worst] = -math.inf
    w = []
    for _ in range(k):
        best = choice == choice.amax(1, keepdim=True)
        at = torch.argmax(best.to(torch.uint8), dim=1, keepdim=True)
        w.append(s.gather(1, at))
        choice.scatter_(1, at, -math.inf)
    w = torch.cat(w, dim=1)
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    return w * case["scale"], None


def _exact_product(x, q, s, z, group):
    """x [r, K] times the weights [N, K/2]: per group, sum(q x) - z sum(x), then the scale."""
    r, N = x.shape[0], q.shape[0]
    xg = x.double().reshape(r, -1, group)
    even, odd = xg[..., 0::2], xg[..., 1::2]
    out = x.new_zeros((r, N), dtype=torch.float64)
    for a in range(0, N, 1024):
        b = q[a:a + 1024].reshape(-1, xg.shape[1], group // 2)
        lo, hi = (b % 16).double(), torch.div(b, 16, rounding_mode="floor").double()
        d = torch.einsum("rgi,ngi->rng", even, lo) + torch.einsum("rgi,ngi->rng", odd, hi)
        zero = 8.0 if z is None else z[a:a + 1024].double()
        d = d - xg.sum(-1).unsqueeze(1) * zero
        out[:, a:a + 1024] = (d * s[a:a + 1024].double()).sum(-1)
    return out


def _exact_act(y, act):
    if act == "none":
        return y
    half = y.shape[-1] // 2
    return y[..., :half] * torch.sigmoid(y[..., :half]) * y[..., half:]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st, case)
    if op == "matvec":
        return _exact_act(_exact_product(st["x"], st["q"], st["s"], st["z"], case["group"]),
                          case["act"])
    if op == "experts":
        m, k = case["m"], case["k"]
        width = case["N"] // 2 if case["act"] == "silu_mul" else case["N"]
        out = torch.zeros((m * k, width), dtype=torch.float64, device="cuda")
        ids = st["ids"].flatten()
        for e in range(case["E"]):
            pairs = torch.nonzero(ids == e).flatten()
            if len(pairs) == 0:
                continue
            x = st["x"].reshape(m * k, -1)[pairs] if case["per_pair"] else st["x"][pairs // k]
            y = _exact_product(x, st["q"][e], st["s"][e],
                               None if st["z"] is None else st["z"][e], case["group"])
            out[pairs] = _exact_act(y, case["act"])
        return out.view(m, k, width)
    r = st["shared"].double() if case["shared"] else 0.0
    y = st["y"].double().reshape(-1, case["H"])
    for j in range(case["k"]):
        at = (torch.arange(case["m"], device=y.device) * case["k"] + j if st["slots"] is None
              else st["slots"][:, j].long())
        live = (at >= 0).double() * st["weights"][:, j].double()
        r = r + live.unsqueeze(1) * y[at.clamp(min=0)]
    if not case["norm"]:
        return r
    r = r + st["residual"].double()
    rms = torch.sqrt((r * r).sum(1, keepdim=True) / case["H"] + EPS)
    return r / rms * st["weight"].double(), r
