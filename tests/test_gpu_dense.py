"""The 8-bit layer's calls on the GPU against their plain 64-bit forms, at the
sizes, types and values where they can go wrong.  Tolerances count roundings
(dense_ref.py); bytes of ar_i8_quantize are exact."""
import math

import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import dense_ref as ref
from test_gpu_experts import DEV, gen, guarded, normal

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF, "f16": HF, "f32": F32}


def within(got, want, bound, dtype):
    err = (got.double() - want).abs()
    tol = bound + ref.rounding(want, dtype) * (1 + 2 ** -8) + ref.half(dtype) * bound
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err - tol)[bad].max()), torch.nonzero(bad)[:4].tolist())


# ---------------------------------------------------------------- block norms

def block_inputs(g, m, H, n, dtype, rtype, post, gate, offset):
    around = 1.0 - offset

    def weight():
        return (torch.randn(H, generator=g, device=DEV) * 0.2 + around).to(dtype)
    kw = dict(post_weight=weight() if post else None, gate=None, weight_offset=offset)
    if gate == "channel":
        kw["gate"] = normal(g, H, dtype=dtype)
    elif gate == "token":
        kw["gate"] = normal(g, m, H, dtype=dtype)
    elif gate:  # rows of a wider tensor, one for each of `gate` sequences
        kw["gate"] = normal(g, gate, 3 * H + 8, dtype=dtype)[:, H + 8:2 * H + 8]
    partials = [normal(g, m, H, dtype=dtype) for _ in range(n)]
    return partials, normal(g, m, H, std=2.0, dtype=rtype or dtype), weight(), kw


def check_block(partials, residual, weight, eps, **kw):
    m, H = residual.shape
    dtype = partials[0].dtype
    y, ey, r, er = ref.block(partials, residual, weight, eps, **kw)
    out, ok1 = guarded((m, H), dtype)
    rout, ok2 = guarded((m, H), residual.dtype)
    a, b = arn.ar_block_rmsnorm(partials, residual, weight, eps, out=out, residual_out=rout, **kw)
    torch.cuda.synchronize()
    assert a is out and b is rout and ok1() and ok2()
    within(rout, r, er, residual.dtype)
    within(out, y, ey, dtype)
    q, ok3 = guarded((m, H), torch.int8)
    s, ok4 = guarded((m,), F32)
    rout2, ok5 = guarded((m, H), residual.dtype)
    arn.ar_block_rmsnorm_i8(partials, residual, weight, eps, q=q, scales=s, residual_out=rout2, **kw)
    torch.cuda.synchronize()
    assert ok3() and ok4() and ok5()
    assert torch.equal(rout2, rout)
    check_bytes(q, s, y, ey)


def check_bytes(q, s, y, ey):
    top = y.abs().amax(1)
    etop = ey.amax(1)
    assert bool(((s.double() - top / 127).abs() <= etop / 127 + 4 * ref.U * top / 127 + 2.0 ** -149).all())
    assert int(q.int().abs().max()) <= 127
    assert bool(((q.int().abs().amax(1) == 127) | (top == 0)).all())
    step = (top / 127).unsqueeze(1)
    err = (q.double() * step - y).abs()
    tol = step * (0.5 + 2.0 ** -13) + ey + y.abs() * (etop / top.clamp(min=1e-300)).unsqueeze(1)
    assert bool((err <= tol).all()), float((err - tol).max())


BLOCKS = [
    # m, H, n, type, residual, post, gate, offset, block scale, residual scale
    (1, 8, 1, "bf16", None, True, None, 0.0, 1.0, 1.0),
    (3, 8, 16, "f16", "f32", True, "token", 1.0, 0.5, 2.0),
    (1, 7168, 8, "bf16", None, True, "channel", 0.0, 1.0, 1.0),
    (16, 7168, 8, "bf16", None, True, None, 1.0, 1.0, 1.0),
    (19, 2048, 4, "f16", None, False, 1, 0.0, 0.22, 1.0),
    (5, 6152, 5, "bf16", "f32", True, 5, 0.0, 1.0, 0.5),
    (77, 1024, 1, "bf16", None, True, 7, 0.0, 1.0, 1.0),
    (153, 4096, 3, "f16", "f32", False, None, 0.0, 1.0, 1.0),
    (400, 5128, 2, "bf16", "f32", True, 8, 1.0, 0.22, 0.5),
    (400, 6144, 1, "f16", None, True, "token", 0.0, 1.0, 1.0),
    (310, 8192, 9, "bf16", None, True, "channel", 0.0, 1.0, 1.0),
    (310, 8192, 2, "f16", "f32", False, "token", 1.0, 1.0, 1.0),
    (2, 8200, 2, "bf16", None, True, None, 0.0, 1.0, 1.0),
    (200, 12296, 3, "bf16", "f32", True, "channel", 0.0, 1.0, 1.0),
    (2, 65544, 1, "bf16", None, True, "token", 0.0, 1.0, 1.0),
    (3, 131072, 2, "f16", "f32", True, None, 0.0, 1.0, 1.0),
    (2500, 264, 3, "bf16", None, True, 2, 0.0, 1.0, 1.0),
]


@pytest.mark.parametrize("m,H,n,kind,rkind,post,gate,offset,bs,rs", BLOCKS)
def test_block(m, H, n, kind, rkind, post, gate, offset, bs, rs):
    g = gen(m * 7 + H)
    if isinstance(gate, int):
        m = m // gate * gate
    p, res, w, kw = block_inputs(g, m, H, n, TYPES[kind], TYPES.get(rkind), post, gate, offset)
    check_block(p, res, w, 1e-6, block_scale=bs, residual_scale=rs, **kw)


@pytest.mark.parametrize("m,H,n", [(4, 7168, 8), (300, 5120, 3), (2, 16384, 1)])
def test_plain_block_is_the_fused_epilogue(m, H, n):
    """Without a norm after the block, gate, scales or offset: ar_rmsnorm's
    residual bit for bit, its output within the two roundings."""
    g = gen(H)
    p, res, w, _ = block_inputs(g, m, H, n, BF, None, False, None, 0.0)
    want, rwant = arn.ar_rmsnorm(p, res, w, 1e-6, mode="one_stage")
    out, rout = arn.ar_block_rmsnorm(p, res, w, 1e-6)
    assert torch.equal(rout, rwant)
    assert bool(((out.double() - want.double()).abs() <= 2 ** -7 * want.double().abs()).all())


def test_block_and_residual_that_cancel():
    """r is the difference of nearly equal numbers; its norm is still r's own."""
    g = gen(5)
    m, H = 9, 4096
    res = normal(g, m, H, dtype=F32)
    p = [-res.to(BF)]
    w = torch.ones(H, device=DEV, dtype=BF)
    check_block(p, res, w, 1e-12)
    check_block(p, p[0].float().neg(), w, 1e-6)  # to zeros


@pytest.mark.parametrize("m", [3, 600])
def test_block_in_place_and_rows_of_zeros(m):
    g = gen(6)
    H = 1024
    p, res, w, kw = block_inputs(g, m, H, 2, BF, None, True, "channel", 0.0)
    for t in (*p, res):
        t[1] = 0
    want, rwant = arn.ar_block_rmsnorm(p, res, w, 1e-6, **kw)
    mine = res.clone()
    out, rout = arn.ar_block_rmsnorm(p, mine, w, 1e-6, residual_out=mine, **kw)
    assert rout is mine and torch.equal(mine, rwant) and torch.equal(out, want)
    assert not out[1].any() and not mine[1].any()
    mine = res.clone()
    q, s, _ = arn.ar_block_rmsnorm_i8(p, mine, w, 1e-6, residual_out=mine, **kw)
    assert torch.equal(mine, rwant) and not q[1].any() and float(s[1]) == 0.0


@pytest.mark.parametrize("m", [4, 700])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_block_rows_that_are_not_finite_stay_their_own(m, bad):
    g = gen(7)
    H = 2048
    p, res, w, kw = block_inputs(g, m, H, 3, BF, None, False, None, 0.0)
    want = arn.ar_block_rmsnorm(p, res, w, 1e-6, **kw)
    wantq = arn.ar_block_rmsnorm_i8(p, res, w, 1e-6, **kw)
    p[1][2, 77] = bad
    got = arn.ar_block_rmsnorm(p, res, w, 1e-6, **kw)
    gotq = arn.ar_block_rmsnorm_i8(p, res, w, 1e-6, **kw)
    others = torch.arange(m, device=DEV) != 2
    for a, b in zip(got + gotq, want + wantq):
        assert torch.equal(a[others], b[others])
    assert not torch.isfinite(got[1][2, 77]) and bool(torch.isnan(got[0][2, 77]))
    assert bool(torch.isnan(gotq[1][2])) and not gotq[0][2].any()


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,K", [(1, 8), (3, 16), (1, 7168), (5, 1000), (33, 8192), (300, 8200),
                                 (2, 16384), (160, 16392), (3, 32776), (2, 131072), (1000, 520)])
def test_quantise(kind, m, K):
    g = gen(K)
    x = normal(g, m, K, std=3.0, dtype=TYPES[kind])
    q, ok1 = guarded((m, K), torch.int8)
    s, ok2 = guarded((m,), F32)
    arn.ar_i8_quantize(x, q=q, scales=s)
    torch.cuda.synchronize()
    assert ok1() and ok2()
    rq, rs = ref.quantise(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_quantise_decides_every_border_exactly(kind):
    """Every finite value of the type against many maxima: ties to even, and
    quotients as near a border as the type has them."""
    dtype = TYPES[kind]
    bits = torch.arange(0, 1 << 15, device=DEV, dtype=torch.int32).to(torch.int16)
    values = bits.view(dtype)
    values = values[torch.isfinite(values)]
    tops = values[values > 0]
    pick = torch.cat([tops[:300:7], tops[::97], tops[-300::7]])
    for top in pick.tolist():
        x = values[values <= top]
        x = x[-32768:]
        x = torch.cat([x, -x])
        x = torch.cat([x, torch.zeros(-x.numel() % 8, device=DEV, dtype=dtype)]).view(1, -1)
        q, s = arn.ar_i8_quantize(x)
        rq, rs = ref.quantise(x)
        assert torch.equal(s, rs), top
        assert torch.equal(q, rq), (top, x[q != rq][:5], q[q != rq][:5])


def test_quantise_strided_rows_and_rows_without_values():
    g = gen(8)
    wide = normal(g, 37, 4096, dtype=BF)
    x = wide[:, 1024:1024 + 2008]
    x[3] = 0
    x[5, 9] = math.nan
    x[6, 2007] = -math.inf
    x[7] = 2.0 ** -133
    q, s = arn.ar_i8_quantize(x)
    rq, rs = ref.quantise(x)
    assert torch.equal(q, rq) and torch.equal(s[~torch.isnan(rs)], rs[~torch.isnan(rs)])
    assert torch.equal(torch.isnan(s), torch.isnan(rs)) and int(torch.isnan(s).sum()) == 2
    assert float(s[3]) == 0.0 and bool((q[7] == 127).all())


# ---------------------------------------------------------------- products

def bytes_(g, *shape, std=32.0):
    x = torch.randn(shape, generator=g, device=DEV) * std
    return x.round_().clamp_(-128, 127).to(torch.int8)


def scale(g, n):
    return (torch.rand(n, generator=g, device=DEV) + 0.5) / 64


def check_product(x, xs, w, ws, act, dtype):
    m, N = x.shape[0], w.shape[0]
    y, ey = ref.product(x, xs, w, ws, act)
    out, ok = guarded((m, N // 2 if act == "silu_mul" else N), dtype)
    arn.ar_i8_matmul(x, xs, w, ws, act=act, out=out)
    torch.cuda.synchronize()
    assert ok()
    within(out, y, ey, dtype)


MS = [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 513]
SHAPES = [(16, 1), (32, 2), (128, 64), (144, 130), (528, 257), (1040, 300), (2048, 1001), (4112, 514)]


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("m", MS)
def test_product(m, K, N):
    g = gen(m * 131 + K)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N)
    check_product(x, xs, w, ws, "none", [BF, F32, HF][(m + N) % 3])
    if N % 2 == 0:
        # Smaller scales: gates of both signs in the range where they matter.
        check_product(x, xs / (4 * math.sqrt(K)), w, ws, "silu_mul", [F32, BF, HF][(m + N // 2) % 3])


@pytest.mark.parametrize("m,K,N,act", [(1, 7168, 7168, "none"), (7, 8192, 4096, "silu_mul"),
                                       (24, 6144, 8192, "silu_mul"), (48, 16384, 1024, "none"),
                                       (96, 8192, 2056, "none"), (150, 5120, 5120, "silu_mul"),
                                       (700, 4096, 3000, "none"), (1111, 2048, 2222, "silu_mul"),
                                       (2048, 1024, 4096, "none")])
def test_product_of_layer_sizes(m, K, N, act):
    g = gen(m + K + N)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N) / math.sqrt(K)
    check_product(x, xs, w, ws, act, BF)


@pytest.mark.parametrize("m", [1, 6, 40, 100, 300])
def test_product_every_byte_against_every_byte(m):
    """Each pair of bytes, one at a time: the 256 x 256 table."""
    v = torch.arange(-128, 128, device=DEV, dtype=torch.int32).to(torch.int8)
    K = 32
    one = torch.ones(1, device=DEV)
    for at in (0, 5, 18, 31):
        w = torch.zeros((256, K), dtype=torch.int8, device=DEV)
        w[:, at] = v
        for a in range(0, 256, m):
            x = torch.zeros((m, K), dtype=torch.int8, device=DEV)
            part = v[a:a + m]
            x[:len(part), at] = part
            out = arn.ar_i8_matmul(x, one.expand(m).contiguous(), w, one.expand(256).contiguous(),
                                   dtype=F32)
            want = torch.zeros((m, 256), device=DEV)
            want[:len(part)] = part.float().unsqueeze(1) * v.float()
            assert torch.equal(out, want)


@pytest.mark.parametrize("m", [1, 8, 20, 130, 400])
@pytest.mark.parametrize("K", [1024, 16384])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (127, 127)])
def test_product_of_the_largest_bytes(m, K, a, b):
    """Sums to 2^14 K: exact up to 2^24, and within K / 16 truncations of a
    half-sized unit beyond."""
    N = 200
    x = torch.full((m, K), a, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), b, dtype=torch.int8, device=DEV)
    one = torch.ones(max(m, N), device=DEV)
    out = arn.ar_i8_matmul(x, one[:m], w, one[:N], dtype=F32)
    want = float(a * b * K)
    off = 0.0 if abs(want) <= 2 ** 24 else (K / 16) * 2.0 ** -23 * abs(want)
    assert float((out.double() - want).abs().max()) <= off


def test_product_scales_that_are_zero_infinite_or_nan():
    g = gen(9)
    for m in (3, 40, 300):
        x, xs, w, ws = bytes_(g, m, 64), scale(g, m), bytes_(g, 96, 64), scale(g, 96)
        want = arn.ar_i8_matmul(x, xs, w, ws, dtype=F32)
        xs[1], ws[70] = math.nan, 0.0
        got = arn.ar_i8_matmul(x, xs, w, ws, dtype=F32)
        assert bool(torch.isnan(got[1]).all())
        rows = torch.arange(m, device=DEV) != 1
        cols = torch.arange(96, device=DEV) != 70
        assert not got[rows][:, 70].any()
        assert torch.equal(got[rows][:, cols], want[rows][:, cols])


# ---------------------------------------------------------------- together, and how they are called

def layer(st):
    """A block in 8 bits, from one epilogue to the next."""
    q, s, r = arn.ar_block_rmsnorm_i8(st["partials"], st["residual"], st["weight"], 1e-6,
                                      post_weight=st["post"], gate=st["gate"])
    h = arn.ar_i8_matmul(q, s, *st["up"], act="silu_mul")
    hq, hs = arn.ar_i8_quantize(h)
    y = arn.ar_i8_matmul(hq, hs, *st["down"])
    return (q, s, r, h, hq, hs, y) + arn.ar_block_rmsnorm([y], r, st["next"], 1e-6,
                                                          post_weight=st["post"], block_scale=0.5)


def layer_inputs(g, m, H=1024, I=1536, n=2):
    def weights(N, K):
        return bytes_(g, N, K), (torch.rand(N, generator=g, device=DEV) + 0.5) / (32 * math.sqrt(K))
    ones = [(torch.randn(H, generator=g, device=DEV) * 0.1 + 1).to(BF) for _ in range(3)]
    return dict(partials=[normal(g, m, H) for _ in range(n)], residual=normal(g, m, H),
                weight=ones[0], post=ones[1], next=ones[2], gate=normal(g, H),
                up=weights(2 * I, H), down=weights(H, I))


def check_layer(st, got):
    """Each call against the 64-bit form of what it was given."""
    q, s, r, h, hq, hs, y, out, rout = got
    b = ref.block(st["partials"], st["residual"], st["weight"], 1e-6, post_weight=st["post"],
                  gate=st["gate"])
    check_bytes(q, s, b[0], b[1])
    within(r, b[2], b[3], BF)
    within(h, *ref.product(q, s, *st["up"], "silu_mul"), BF)
    rq, rs = ref.quantise(h)
    assert torch.equal(hq, rq) and torch.equal(hs, rs)
    within(y, *ref.product(hq, hs, *st["down"], "none"), BF)
    b = ref.block([y], r, st["next"], 1e-6, post_weight=st["post"], block_scale=0.5)
    within(rout, b[2], b[3], BF)
    within(out, b[0], b[1], BF)


@pytest.mark.parametrize("m", [1, 7, 60, 130, 600])
def test_a_layer(m):
    st = layer_inputs(gen(m), m)
    check_layer(st, layer(st))


@pytest.mark.parametrize("m", [1, 60, 300])
def test_a_layer_in_a_graph_takes_new_inputs(m):
    st = layer_inputs(gen(m), m)
    layer(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(st)
    for seed in (1, 2):
        new = layer_inputs(gen(seed), m)
        for k in ("residual", "weight", "post", "next", "gate"):
            st[k].copy_(new[k])
        for k in ("partials", "up", "down"):
            for a, b in zip(st[k], new[k]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        check_layer(st, got)


def test_streams_do_not_share_anything():
    """Layers on four streams at once, each with its own inputs."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    states = [layer_inputs(gen(40 + i), m) for i, m in enumerate((1, 33, 140, 500))]
    want = [layer(st) for st in states]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(states[i]))
    torch.cuda.synchronize()
    for i in range(4):
        for g in got[i]:
            for a, b in zip(want[i], g):
                assert torch.equal(a, b)


@pytest.mark.parametrize("how", ["given", "handle"])
def test_given_streams_and_the_long_way_give_the_same(how):
    st = layer_inputs(gen(50), 20)
    s = torch.cuda.Stream()
    want = layer(st)
    torch.cuda.synchronize()
    on = s if how == "given" else s.cuda_stream
    q, sc, r = arn.ar_block_rmsnorm_i8(st["partials"], st["residual"], st["weight"], 1e-6,
                                       post_weight=st["post"], gate=st["gate"], stream=on)
    h = arn.ar_i8_matmul(q, sc, *st["up"], act="silu_mul", stream=on)
    hq, hs = arn.ar_i8_quantize(h, stream=on)
    y = arn.ar_i8_matmul(hq, hs, *st["down"], stream=on)
    out, rout = arn.ar_block_rmsnorm([y], r, st["next"], 1e-6, post_weight=st["post"],
                                     block_scale=0.5, stream=on)
    s.synchronize()
    for a, b in zip(want, (q, sc, r, h, hq, hs, y, out, rout)):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_one_step_is_taken(monkeypatch):
    from allreduce_sum_residual_gb300 import dense
    st = layer_inputs(gen(51), 4)
    monkeypatch.setattr(dense, "_call", lambda *a: pytest.fail("the long way"))
    layer(st)


def test_empty_batches():
    st = layer_inputs(gen(52), 0)
    st["gate"] = st["gate"].view(1, -1)
    for t in layer(st):
        assert t.shape[0] == 0
