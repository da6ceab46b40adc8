"""The expert-layer calls on the GPU against their plain 64-bit forms, at the
sizes, types and masks where they can go wrong.  Tolerances count roundings
(experts_ref.py); ids and zero rows are exact."""
import math

import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import experts_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def guarded(shape, dtype):
    """An output inside a buffer of canaries, and a check that they survived."""
    n = math.prod(shape)
    pad = 256
    size = torch.empty((), dtype=dtype).element_size()
    buf = torch.full(((n + 2 * pad) * size,), 0x5A, dtype=torch.uint8, device=DEV)
    out = buf[pad * size:(pad + n) * size].view(dtype).view(shape)

    def intact():
        return bool((buf[:pad * size] == 0x5A).all()) and bool((buf[(pad + n) * size:] == 0x5A).all())
    return out, intact


# ---------------------------------------------------------------- routing

ROUTE = [
    # m, E, k, type, scoring, groups, topk_groups, group_score, bias, renorm, scale
    (1, 1, 1, "f32", "softmax", 1, 1, "max", False, True, 1.0),
    (5, 8, 8, "bf16", "softmax", 1, 1, "max", False, False, 1.0),
    (16, 128, 8, "bf16", "softmax", 1, 1, "max", False, True, 1.0),
    (33, 128, 8, "bf16", "sigmoid", 1, 1, "max", True, True, 2.5),
    (64, 60, 6, "f16", "softmax", 6, 3, "max", False, False, 1.0),
    (64, 61, 4, "f32", "softmax", 1, 1, "max", True, True, 1.0),
    (70, 256, 8, "f32", "sigmoid", 8, 4, "top2", True, True, 2.5),
    (70, 256, 8, "bf16", "sigmoid", 8, 4, "top2", False, True, 1.0),
    (70, 160, 6, "bf16", "softmax", 8, 3, "max", True, False, 16.0),
    (33, 512, 16, "f32", "softmax", 1, 1, "max", False, True, 1.0),
    (33, 512, 16, "bf16", "sigmoid", 32, 9, "top2", True, True, 1.0),
    (33, 493, 7, "f16", "sigmoid", 17, 5, "top2", True, False, 1.0),
    (33, 510, 16, "bf16", "softmax", 17, 17, "top2", False, True, 1.0),
    (9, 64, 4, "f32", "softmax", 2, 1, "top2", False, True, 1.0),
    (9, 34, 2, "bf16", "sigmoid", 17, 1, "top2", True, True, 1.0),
]


def check_route(x, k, w, ids, **kw):
    rw, rids = ref.route(x, k, **kw)
    assert torch.equal(ids.cpu(), rids)
    # exp within 1 ulp, sums of up to 37 adds, two divides, the scale: 2^-18.
    err = (w.cpu().double() - rw).abs()
    assert bool((err <= 2.0 ** -18 * rw.abs() + 1e-37).all()), float(err.max())


@pytest.mark.parametrize("m,E,k,kind,scoring,groups,topk_groups,group_score,bias,renorm,scale", ROUTE)
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_route(m, E, k, kind, scoring, groups, topk_groups, group_score, bias, renorm, scale, masked):
    g = gen(m * 1000 + E)
    x = normal(g, m, E, std=2.0, dtype=TYPES[kind])
    if masked:
        x[torch.rand((m, E), generator=g, device=DEV) < masked] = -math.inf
        x[0] = -math.inf  # a row with nothing on
    b = normal(g, E, std=0.3, dtype=torch.float32) if bias else None
    wbuf, wok = guarded((m, k), torch.float32)
    ibuf, iok = guarded((m, k), torch.int32)
    kw = dict(bias=b, scoring=scoring, groups=groups, topk_groups=topk_groups,
              group_score=group_score, renorm=renorm, scale=scale)
    w, ids = arn.ar_route_experts(x, k, weights=wbuf, ids=ibuf, **kw)
    torch.cuda.synchronize()
    assert wok() and iok()
    check_route(x, k, w, ids, **kw)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("width,offset", [(64, 0), (80, 8), (73, 3), (200, 100)])
def test_route_takes_strided_and_unaligned_logits(kind, width, offset):
    g = gen(width)
    wide = normal(g, 21, width + 64, dtype=TYPES[kind])
    x = wide[:, offset:offset + 64]
    for kw in (dict(), dict(scoring="sigmoid", groups=4, topk_groups=2, group_score="top2")):
        w, ids = arn.ar_route_experts(x, 6, **kw)
        check_route(x, 6, w, ids, **kw)


def test_route_ties_go_to_the_lowest_index():
    """Few distinct logits, with and without equal biases, and -0 beside 0."""
    g = gen(3)
    x = torch.randint(-1, 2, (64, 96), generator=g, device=DEV).to(torch.bfloat16) * 0.5
    x[0] = 0.0
    x[0, ::2] = -0.0
    for kw in (dict(), dict(scoring="sigmoid", bias=torch.zeros(96, device=DEV)),
               dict(scoring="softmax", bias=torch.full((96,), 0.25, device=DEV)),
               dict(groups=8, topk_groups=3), dict(groups=8, topk_groups=3, group_score="top2"),
               dict(groups=8, topk_groups=3, group_score="top2", scoring="sigmoid",
                    bias=torch.full((96,), -2.0, device=DEV))):
        w, ids = arn.ar_route_experts(x, 8, **kw)
        check_route(x, 8, w, ids, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_decides_near_ties_as_64_bits_do(scoring):
    """Biases that undo the scores of row 0 to within a rounding of fp32: its
    order is the order of those roundings, below what fp32 scores resolve."""
    g = gen(4)
    x = normal(g, 40, 256, dtype=torch.float32)
    s = (torch.softmax(x[0].double(), 0) if scoring == "softmax" else torch.sigmoid(x[0].double()))
    b = (0.5 - s).float()
    kw = dict(bias=b, scoring=scoring)
    w, ids = arn.ar_route_experts(x, 8, **kw)
    check_route(x, 8, w, ids, **kw)
    kw.update(groups=8, topk_groups=4, group_score="top2")
    w, ids = arn.ar_route_experts(x, 8, **kw)
    check_route(x, 8, w, ids, **kw)


def test_route_many_rows_agree_with_64_bits():
    """65536 rows: some hundred have a border that fp32 cannot call."""
    g = gen(5)
    x = normal(g, 65536, 256, std=1.5, dtype=torch.float32)
    b = normal(g, 256, std=0.1, dtype=torch.float32)
    _, ids = arn.ar_route_experts(x, 8, bias=b, scoring="sigmoid", groups=8, topk_groups=4,
                                  group_score="top2", renorm=True)
    c = torch.sigmoid(x.double()) + b.double()
    best = torch.sort(c.view(-1, 8, 32), dim=2, descending=True).values
    score = best[..., 0] + best[..., 1]
    kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :4]
    inside = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
    c = torch.where(inside.repeat_interleave(32, dim=1), c, -math.inf)
    want = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :8].int()
    assert torch.equal(ids, want)


@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_decides_near_group_borders_as_64_bits_do(group_score):
    """Groups whose scores differ by less than fp32 resolves, in every row:
    eight groups hold the same choices up to a few 2^-25, in another order."""
    g = gen(14)
    m, per = 200, 32
    x = normal(g, 1, per, std=1.0, dtype=torch.float32).repeat(m, 8)
    x = x.view(m, 8, per)
    for j in range(8):
        x[:, j] = x[:, j, torch.randperm(per, generator=g, device=DEV)]
    s = torch.sigmoid(x.double())
    s = s + (torch.rand(s.shape, generator=g, device=DEV).double() - 0.5) * 2.0 ** -23
    x = torch.log(s / (1 - s)).float().reshape(m, 8 * per)
    b = torch.full((8 * per,), 0.5, device=DEV)
    kw = dict(bias=b, scoring="sigmoid", groups=8, topk_groups=4, group_score=group_score)
    w, ids = arn.ar_route_experts(x, 8, **kw)
    check_route(x, 8, w, ids, **kw)


def test_route_nan_and_infinite_values_keep_ids_valid():
    g = gen(6)
    x = normal(g, 32, 64, dtype=torch.float32)
    x[1, 5] = math.nan
    x[2] = math.nan
    x[3, 7] = math.inf
    x[4, :2] = math.inf
    b = normal(g, 64, dtype=torch.float32)
    b2 = b.clone()
    b2[3], b2[4], b2[5] = math.inf, -math.inf, math.nan
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, b, b2):
            for kw in (dict(), dict(groups=8, topk_groups=2), dict(groups=8, topk_groups=2,
                                                                   group_score="top2")):
                for renorm in (True, False):
                    w, ids = arn.ar_route_experts(x, 8, bias=bias, scoring=scoring, renorm=renorm, **kw)
                    i = ids.cpu()
                    assert int(i.min()) >= 0 and int(i.max()) < 64
                    assert all(len(set(r)) == 8 for r in i.tolist())
                    if scoring == "softmax":
                        assert bool(w[1].isnan().all() and w[2].isnan().all() and w[4].isnan().all())
                    assert bool(w[5:].isfinite().all())
                    if bias is not b2:
                        _, want = ref.route(x[5:], 8, bias=bias, scoring=scoring, renorm=renorm, **kw)
                        assert torch.equal(i[5:], want)


# ---------------------------------------------------------------- 4-bit products

def weights4(g, lead, K, group, kind, zeros):
    ng = K // group
    q = torch.randint(0, 256, (*lead, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = ((torch.rand((*lead, ng), generator=g, device=DEV) - 0.4) / math.sqrt(K)).to(TYPES[kind])
    z = (torch.randint(0, 256, (*lead, ng), generator=g, device=DEV, dtype=torch.uint8)
         if zeros else None)
    return q, s, z


MATVEC = [
    # m, K, N, group, scale type, zeros, act
    (1, 32, 1, 32, "bf16", False, "none"),
    (1, 64, 2, 64, "f32", True, "silu_mul"),
    (1, 128, 17, 128, "f16", True, "none"),
    (2, 96, 33, 32, "f32", True, "none"),
    (3, 160, 34, 32, "f16", True, "silu_mul"),
    (7, 192, 515, 64, "bf16", True, "none"),
    (8, 1056, 514, 32, "bf16", True, "silu_mul"),
    (9, 1088, 100, 64, "f16", False, "none"),
    (16, 4128, 1001, 32, "f32", True, "none"),
    (16, 640, 4096, 128, "bf16", False, "silu_mul"),
    (17, 384, 130, 128, "f32", True, "none"),
    (33, 512, 66, 64, "bf16", False, "silu_mul"),
    (64, 2048, 300, 128, "bf16", True, "none"),
    (1, 7168, 2048, 128, "bf16", False, "none"),
    (16, 7168, 512, 64, "f16", True, "none"),
    (16, 6144, 20480, 128, "bf16", False, "silu_mul"),   # tall items
    (3, 1024, 50000, 64, "bf16", True, "none"),
    (4, 1024, 30002, 32, "f32", True, "silu_mul"),
    (16, 32768, 64, 32, "bf16", True, "none"),           # longest, most shared memory
    (64, 32768, 40, 128, "f32", False, "silu_mul"),
    (1, 32736, 50, 32, "f16", True, "none"),
]


@pytest.mark.parametrize("m,K,N,group,kind,zeros,act", MATVEC)
def test_w4_matvec(m, K, N, group, kind, zeros, act):
    g = gen(m + K + N)
    x = normal(g, m, K)
    q, s, z = weights4(g, (N,), K, group, kind, zeros)
    out, intact = guarded((m, N // 2 if act == "silu_mul" else N), torch.bfloat16)
    arn.ar_w4_matvec(x, q, s, zeros=z, act=act, out=out)
    torch.cuda.synchronize()
    assert intact()
    y, err = ref.act(*ref.product(x, q, s, z), act)
    ref.close(out, y, err)


EXPERTS = [
    # m, E, k, K, N, group, scale type, zeros, act, x per pair, missing
    (1, 1, 1, 32, 3, 32, "bf16", False, "none", False, 0.0),
    (1, 64, 8, 256, 130, 128, "bf16", False, "silu_mul", False, 0.0),
    (3, 7, 2, 160, 33, 32, "f32", True, "none", True, 0.3),
    (7, 17, 3, 1056, 515, 32, "bf16", True, "none", False, 0.25),
    (8, 4, 3, 448, 100, 64, "f16", True, "silu_mul", True, 0.0),
    (16, 512, 16, 128, 48, 128, "bf16", False, "none", False, 0.5),
    (32, 128, 8, 1024, 200, 128, "bf16", False, "none", True, 0.0),
    (40, 2, 1, 256, 70, 64, "f32", True, "none", False, 0.0),       # sets of more than 16
    (70, 5, 4, 384, 50, 128, "bf16", True, "silu_mul", True, 0.1),
    (4096, 300, 1, 64, 20, 32, "bf16", False, "none", False, 0.0),
    (256, 9, 16, 64, 18, 64, "bf16", False, "none", True, 0.9),
    (5, 6, 2, 512, 64, 128, "bf16", False, "none", False, 1.0),     # nobody here
    (24, 64, 8, 2048, 4096, 128, "bf16", False, "silu_mul", False, 0.0),
    (16, 3, 2, 16384, 40, 64, "bf16", True, "none", True, 0.0),
    (16, 64, 8, 7168, 40, 128, "bf16", False, "silu_mul", False, 0.0),  # sets of 7, one phase
    (12, 40, 4, 7040, 34, 64, "f16", True, "none", False, 0.1),         # a part behind the row's end
    (64, 2, 1, 1152, 2000, 128, "bf16", True, "none", False, 0.0),      # two row and two column tiles
    (300, 3, 1, 384, 700, 64, "f32", True, "silu_mul", True, 0.0),
]


def expert_rows(x, ids, q, s, z, act):
    """(result, error) of every pair, expert by expert."""
    m, k = ids.shape
    K = x.shape[-1]
    width = q.shape[1] // (2 if act == "silu_mul" else 1)
    y = torch.zeros((m * k, width), dtype=torch.float64, device=DEV)
    e = torch.zeros_like(y)
    rows = x.reshape(m * k, K) if x.dim() == 3 else x.repeat_interleave(k, 0)
    flat = ids.flatten()
    for ex in range(q.shape[0]):
        at = (flat == ex).nonzero().flatten()
        if len(at):
            y[at], e[at] = ref.act(*ref.product(rows[at], q[ex], s[ex],
                                                None if z is None else z[ex]), act)
    return y.view(m, k, -1), e.view(m, k, -1)


@pytest.mark.parametrize("m,E,k,K,N,group,kind,zeros,act,per_pair,missing", EXPERTS)
def test_w4_matvec_experts(m, E, k, K, N, group, kind, zeros, act, per_pair, missing):
    g = gen(m + E + K)
    x = normal(g, m, k, K) if per_pair else normal(g, m, K)
    ids = torch.randint(0, E, (m, k), generator=g, device=DEV, dtype=torch.int32)  # repeats too
    gone = torch.rand((m, k), generator=g, device=DEV) < missing
    bad = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    ids[gone] = bad[torch.randint(0, 4, (int(gone.sum()),), generator=g, device=DEV)]
    q, s, z = weights4(g, (E, N), K, group, kind, zeros)
    out, intact = guarded((m, k, N // 2 if act == "silu_mul" else N), torch.bfloat16)
    arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z, act=act, out=out)
    torch.cuda.synchronize()
    assert intact()
    y, err = expert_rows(x, ids, q, s, z, act)
    ref.close(out, y, err)
    assert not bool(out[gone].any())


@pytest.mark.parametrize("level", [2.0 ** -133, 2.0 ** -126, 1e-30, 1.0, 1e30])
def test_w4_matvec_holds_over_the_range_of_x(level):
    """Rows from bf16's smallest to its largest numbers, and rows whose values
    spread over sixty powers of two (scales bring the results back)."""
    g = gen(13)
    x = torch.randint(-8, 9, (6, 512), generator=g, device=DEV).double() * level
    x[1] *= torch.exp2(-torch.randint(0, 60, (512,), generator=g, device=DEV).double())
    x[2, 100] *= 2.0 ** 6
    x[3] = 0
    x = x.bfloat16()
    q, s, z = weights4(g, (64,), 512, 64, "f32", True)
    s = (s.double() / max(level, 2.0 ** -100)).float() if level < 1 else s
    ref.close(arn.ar_w4_matvec(x, q, s, zeros=z), *ref.product(x, q, s, z))


def test_w4_matvec_experts_of_a_rank():
    """`first`: the whole layer's numbers, of which this rank holds some."""
    g = gen(15)
    x = normal(g, 9, 256)
    q, s, z = weights4(g, (12, 40), 256, 64, "bf16", True)
    ids = torch.randint(-3, 15, (9, 4), generator=g, device=DEV, dtype=torch.int32)
    ids[0, :2] = torch.tensor([-2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    for first, count in ((0, 5), (5, 4), (9, 3)):
        sl = slice(first, first + count)
        got = arn.ar_w4_matvec_experts(x, ids, q[sl], s[sl], zeros=z[sl], first=first)
        local = torch.where((ids >= first) & (ids < first + count), ids - first, -1).int()
        ref.close(got, *expert_rows(x, local, q[sl], s[sl], z[sl], "none"))
        assert not bool(got[local < 0].any())


@pytest.mark.parametrize("m,K,N", [(16, 7168, 24), (9, 1024, 5000)])
def test_w4_matvec_experts_with_every_token_on_one_expert(m, K, N):
    """More tokens than a set has columns, all on one expert; the others idle."""
    g = gen(16)
    x = normal(g, m, K)
    q, s, z = weights4(g, (32, N), K, 128, "bf16", False)
    ids = torch.full((m, 4), 7, device=DEV, dtype=torch.int32)
    ids[3, 1:] = torch.tensor([0, 31, 32], dtype=torch.int32)
    ref.close(arn.ar_w4_matvec_experts(x, ids, q, s), *expert_rows(x, ids, q, s, z, "none"))


@pytest.mark.parametrize("m", [1, 9])
@pytest.mark.parametrize("K,group", [(128, 128), (384, 128), (192, 64), (320, 64), (64, 64), (96, 32)])
def test_w4_scales_behind_a_rows_end_take_no_part(m, K, group):
    """The next row's NaN scales lie where a row's last, unfinished unit ends."""
    g = gen(17)
    x = normal(g, m, K)
    for kind in ("f32", "bf16", "f16"):
        for zeros in (False, True):
            q, s, z = weights4(g, (50,), K, group, kind, zeros)
            clean = arn.ar_w4_matvec(x, q, s, zeros=z)
            s2 = s.clone()
            s2[1::2] = math.nan
            out = arn.ar_w4_matvec(x, q, s2, zeros=z)
            assert torch.equal(out[:, ::2], clean[:, ::2]) and bool(out[:, 1::2].isnan().all())


def test_w4_nan_and_infinite_rows_stay_their_own():
    """A NaN or an infinity in one row of x, or one scale, reaches no other
    row or output; the group behind a row's end takes no part."""
    g = gen(9)
    x = normal(g, 5, 96)
    q, s, z = weights4(g, (40,), 96, 32, "f32", True)
    clean = arn.ar_w4_matvec(x, q, s, zeros=z)
    x2, s2 = x.clone(), s.clone()
    x2[1, 7], x2[3, 0] = math.nan, math.inf
    s2[11, 0] = math.nan  # row 10 ends in front of it
    out = arn.ar_w4_matvec(x2, q, s2, zeros=z)
    keep = [0, 2, 4]
    cols = [i for i in range(40) if i != 11]
    assert torch.equal(out[keep][:, cols], clean[keep][:, cols])
    assert bool(out[1].isnan().all()) and bool(out[:, 11].isnan().all())


# ---------------------------------------------------------------- combine

COMBINE = [
    # m, k, H, shared, slots, missing
    (1, 1, 8, False, False, 0.0),
    (1, 8, 7168, True, False, 0.0),
    (3, 5, 1032, False, True, 0.3),
    (16, 8, 7168, True, True, 0.5),
    (33, 9, 24, True, True, 0.0),
    (40, 16, 4096, False, True, 0.0),
    (200, 6, 2056, True, False, 0.0),
    (300, 2, 8192, False, True, 1.0),
    (5, 3, 16384, True, True, 0.2),
    (2, 4, 65536, False, False, 0.0),
    (2, 3, 131072, True, True, 0.2),
]


def combine_inputs(m, k, H, shared, slots, missing, seed):
    g = gen(seed)
    rows = m * k + 3 if slots else m * k
    y = normal(g, rows, H) if slots else normal(g, m, k, H)
    st = None
    if slots:
        st = torch.randint(0, rows, (m, k), generator=g, device=DEV, dtype=torch.int32)
        gone = torch.rand((m, k), generator=g, device=DEV) < missing
        bad = torch.tensor([-1, rows, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        st[gone] = bad[torch.randint(0, 4, (int(gone.sum()),), generator=g, device=DEV)]
    w = normal(g, m, k, dtype=torch.float32)
    if slots and missing:
        w[gone] = math.nan  # the weight of a choice that is not here does not count
    sh = normal(g, m, H) if shared else None
    return y, w, sh, st, rows


@pytest.mark.parametrize("m,k,H,shared,slots,missing", COMBINE)
def test_combine(m, k, H, shared, slots, missing):
    y, w, sh, st, rows = combine_inputs(m, k, H, shared, slots, missing, m + H)
    out, intact = guarded((m, H), torch.bfloat16)
    arn.ar_combine(y, w, shared=sh, slots=st, out=out)
    torch.cuda.synchronize()
    assert intact()
    r, mag = ref.combine(y, w, sh, st, rows, k)
    ref.close(out, r, k * ref.F32 * mag)


@pytest.mark.parametrize("m,k,H,shared,slots,missing", COMBINE)
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_rmsnorm(m, k, H, shared, slots, missing, in_place):
    y, w, sh, st, rows = combine_inputs(m, k, H, shared, slots, missing, m + H + 1)
    g = gen(7)
    res, wt = normal(g, m, H), (normal(g, H, std=0.1, dtype=torch.float32) + 1).bfloat16()
    r, mag = ref.combine(y, w, sh, st, rows, k)
    r, mag = r + res.double(), mag + res.double().abs()
    out, intact = guarded((m, H), torch.bfloat16)
    rout, rintact = guarded((m, H), torch.bfloat16)
    if in_place:
        rout.copy_(res)
        res = rout
    arn.ar_combine_rmsnorm(y, w, res, wt, 1e-6, shared=sh, slots=st, out=out, residual_out=rout)
    torch.cuda.synchronize()
    assert intact() and rintact()
    err = (k + 1) * ref.F32 * mag
    ref.close(rout, r, err)
    ref.close(out, *ref.norm(r, err, wt, 1e-6))
    assert arn.ar_device_status(0) == arn.AR_OK


def test_combine_of_nothing():
    """No row of y at all: the shared rows, or zeros."""
    g = gen(8)
    y = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    st = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    w = torch.ones((4, 2), device=DEV)
    sh = normal(g, 4, 64)
    assert torch.equal(arn.ar_combine(y, w, shared=sh, slots=st), sh)
    assert not bool(arn.ar_combine(y, w, slots=st).any())


# ---------------------------------------------------------------- together

def layer(x, router, bias, up, down, residual, weight, shared=None):
    w, ids = arn.ar_route_experts(x @ router.T, 4, bias=bias, scoring="sigmoid", groups=4,
                                  topk_groups=2, group_score="top2", scale=2.5)
    h = arn.ar_w4_matvec_experts(x, ids, *up, act="silu_mul")
    y = arn.ar_w4_matvec_experts(h, ids, *down)
    return arn.ar_combine_rmsnorm(y, w, residual, weight, 1e-6, shared=shared), w, ids, h, y


def layer_inputs(m, seed, H=1024, I=256, E=32):
    g = gen(seed)
    return dict(x=normal(g, m, H), router=normal(g, E, H, std=0.03),
                bias=normal(g, E, std=0.1, dtype=torch.float32),
                up=weights4(g, (E, 2 * I), H, 128, "bf16", True),
                down=weights4(g, (E, H), I, 64, "bf16", False),
                residual=normal(g, m, H), weight=normal(g, H), shared=normal(g, m, H))


@pytest.mark.parametrize("m", [1, 6, 40])
def test_a_layer_from_routing_to_the_norm(m):
    """The calls in a row, each checked against 64 bits on what it was given."""
    inp = layer_inputs(m, m)
    (out, rout), w, ids, h, y = layer(**inp)
    check_route(inp["x"] @ inp["router"].T, 4, w, ids, bias=inp["bias"], scoring="sigmoid", groups=4,
                topk_groups=2, group_score="top2", scale=2.5)
    ref.close(h, *expert_rows(inp["x"], ids, *inp["up"], "silu_mul"))
    ref.close(y, *expert_rows(h, ids, *inp["down"], "none"))
    r, mag = ref.combine(y, w, inp["shared"], None, m * 4, 4)
    r, mag = r + inp["residual"].double(), mag + inp["residual"].double().abs()
    ref.close(rout, r, 5 * ref.F32 * mag)
    ref.close(out, *ref.norm(r, 5 * ref.F32 * mag, inp["weight"], 1e-6))


def test_ranks_partials_reach_the_epilogue():
    """Two ranks hold half of the experts each: their combined partials go
    through ar_rmsnorm.  Each product is checked on what it was given; the
    partials' sum is off by their own roundings."""
    m, inp = 6, layer_inputs(6, 11)
    _, w, ids, _, _ = layer(**inp)
    partials = []
    r, mag = inp["residual"].double(), inp["residual"].double().abs()
    for rank in range(2):
        mine = torch.where((ids >= 16 * rank) & (ids < 16 * (rank + 1)), ids - 16 * rank, -1).int()
        sl = slice(16 * rank, 16 * (rank + 1))
        up = [None if t is None else t[sl] for t in inp["up"]]
        down = [None if t is None else t[sl] for t in inp["down"]]
        shared = inp["shared"] if rank == 0 else None
        h = arn.ar_w4_matvec_experts(inp["x"], ids, *up, act="silu_mul", first=16 * rank)
        y = arn.ar_w4_matvec_experts(h, ids, *down, first=16 * rank)
        ref.close(h, *expert_rows(inp["x"], mine, *up, "silu_mul"))
        ref.close(y, *expert_rows(h, mine, *down, "none"))
        assert not bool(y[mine < 0].any())
        partials.append(arn.ar_combine(y, w, shared=shared))
        c, cmag = ref.combine(y, w, shared, None, m * 4, 4)
        r, mag = r + c, mag + cmag
    out, rout = arn.ar_rmsnorm(partials, inp["residual"], inp["weight"], 1e-6)
    err = 2 * ref.BF16 * mag + 8 * ref.F32 * mag  # each partial rounds once to bf16
    ref.close(rout, r, err)
    ref.close(out, *ref.norm(r, err, inp["weight"], 1e-6))


def test_captured_and_replayed_with_new_inputs():
    """The layer in a CUDA graph: replays follow what its inputs hold then,
    and equal the eager calls bit for bit."""
    a, b = layer_inputs(5, 21), layer_inputs(5, 22)
    want = [layer(**d)[0] for d in (a, b)]
    live = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in a.items()}
    live["up"], live["down"] = a["up"], a["down"]
    b.update(up=a["up"], down=a["down"])
    want[1] = layer(**b)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(**live)[0]
    for d, w in ((b, want[1]), (a, want[0]), (b, want[1])):
        for k in ("x", "router", "bias", "residual", "weight", "shared"):
            live[k].copy_(d[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def test_two_graphs_and_two_streams_at_once():
    """No call keeps state: two graphs replayed on two streams, interleaved
    and overlapping, give what each gives alone."""
    ins = [layer_inputs(3, 31), layer_inputs(17, 32)]
    want = [layer(**d)[0] for d in ins]
    graphs, outs = [], []
    for d in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(**d)[0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_a_given_stream_owns_its_outputs():
    """stream= as a torch stream and as a raw handle; outputs made by the call
    belong to that stream."""
    d = layer_inputs(4, 41)
    want, ids0 = arn.ar_route_experts(d["x"] @ d["router"].T, 4)
    side = torch.cuda.Stream()
    logits = d["x"] @ d["router"].T
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        w, ids = arn.ar_route_experts(logits, 4, stream=s)
        h = arn.ar_w4_matvec_experts(d["x"], ids, *d["up"], act="silu_mul", stream=s)
        y = arn.ar_w4_matvec_experts(h, ids, *d["down"], stream=s)
        o = arn.ar_combine(y, w, stream=s)
        side.synchronize()
        assert torch.equal(w, want) and torch.equal(ids, ids0) and bool(o.isfinite().all())


def test_results_repeat_bit_for_bit():
    """No atomics in any sum: the same call gives the same bits."""
    g = gen(51)
    x = normal(g, 16, 1024)
    q, s, z = weights4(g, (8, 96), 1024, 128, "bf16", True)
    ids = torch.randint(0, 8, (16, 2), generator=g, device=DEV, dtype=torch.int32)
    full = arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z)
    again = arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z)
    assert torch.equal(full, again)


def test_binding_errors_on_the_gpu():
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((8, 128), dtype=torch.uint8, device=DEV)
    s = torch.zeros((8, 2), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="rows of logits"):
        arn.ar_route_experts(x.T, 2)
    with pytest.raises(TypeError, match="logits must be float32"):
        arn.ar_route_experts(q, 2)
    with pytest.raises(arn.ArError) as e:
        arn.ar_route_experts(x[:, :64], 17)
    assert e.value.status == arn.AR_ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="scoring"):
        arn.ar_route_experts(x[:, :64], 2, scoring="relu")
    with pytest.raises(ValueError, match="K/2"):
        arn.ar_w4_matvec(x, q[:, :64].contiguous(), s)
    with pytest.raises(ValueError, match="one value per group"):
        arn.ar_w4_matvec(x, q, torch.zeros((8, 3), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError, match="q must be uint8"):
        arn.ar_w4_matvec(x, q.int(), s)
    with pytest.raises(ValueError, match="contiguous"):
        arn.ar_w4_matvec(x, torch.zeros((8, 256), dtype=torch.uint8, device=DEV)[:, ::2], s)
    with pytest.raises(arn.ArError) as e:
        arn.ar_w4_matvec(x, q, torch.zeros((8, 16), dtype=torch.bfloat16, device=DEV))
    assert e.value.status == arn.AR_ERR_ARG
    with pytest.raises(TypeError, match="ids must be int32"):
        arn.ar_w4_matvec_experts(x, ids.long(), q[None], s[None])
    with pytest.raises(ValueError, match="x must have shape"):
        arn.ar_w4_matvec_experts(x[:3].contiguous(), ids, q[None], s[None])
    w = torch.zeros((4, 2), device=DEV)
    with pytest.raises(ValueError, match="without slots"):
        arn.ar_combine(x, w)
    with pytest.raises(ValueError, match="slots must have shape"):
        arn.ar_combine(x, w, slots=ids[:2].contiguous())
    with pytest.raises(arn.ArError) as e:
        arn.ar_combine(x, w, slots=ids, out=x)
    assert e.value.status == arn.AR_ERR_ALIAS
    out = arn.ar_combine(torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV),
                         torch.empty((0, 2), device=DEV))
    assert out.shape == (0, 64)
