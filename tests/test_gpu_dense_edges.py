"""The 8-bit layer's calls at the ends of their ranges: arrays past 2^31
elements, the longest products and rows, batches that take other kernels,
threads, and the checking build."""
import threading

import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import dense_ref as ref
from test_gpu_dense import BF, DEV, F32, HF, block_inputs, bytes_, check_block, check_product, layer, \
    layer_inputs, scale, within
from test_gpu_experts import gen, guarded, normal
from test_gpu_experts_check import checklib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N,act", [(512, 300, "none"), (1024, 2000, "silu_mul"), (4096, 1001, "none"),
                                     (2992, 8192, "silu_mul")])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_a_row_does_not_depend_on_its_batch(K, N, act, dtype):
    """Every kernel and split gives the same bits where the sums are exact."""
    N -= N % 2 if act == "silu_mul" else 0
    g = gen(K + N)
    x, xs, w, ws = bytes_(g, 700, K), scale(g, 700), bytes_(g, N, K), scale(g, N) / 30
    want = arn.ar_i8_matmul(x, xs, w, ws, act=act, dtype=dtype)
    for m in (1, 2, 3, 7, 12, 16, 30, 64, 100, 128, 190, 256, 400, 513):
        got = arn.ar_i8_matmul(x[:m], xs[:m], w, ws, act=act, dtype=dtype)
        assert torch.equal(got, want[:m]), m


@pytest.mark.parametrize("m,K,N,act", [(5000, 4096, 4096, "none"), (3001, 5120, 5122, "silu_mul")])
def test_a_prompt_in_two_launches(m, K, N, act):
    """A prompt whose last tokens take a launch of their own."""
    g = gen(m)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N) / 300
    out, ok = guarded((m, N // 2 if act == "silu_mul" else N), BF)
    arn.ar_i8_matmul(x, xs, w, ws, act=act, out=out)
    torch.cuda.synchronize()
    assert ok()
    for a in range(0, m, 500):
        assert torch.equal(out[a:a + 500], arn.ar_i8_matmul(x[a:a + 500], xs[a:a + 500], w, ws, act=act))
    y, ey = ref.product(x[-300:], xs[-300:], w, ws, act)
    within(out[-300:], y, ey, BF)


@pytest.mark.parametrize("K", [16, 128, 144, 384, 400, 528])
@pytest.mark.parametrize("N,act", [(20011, "none"), (20016, "none"), (20012, "silu_mul"), (20016, "silu_mul")])
def test_many_tiles_of_few_stages(K, N, act):
    """One to five stages a tile, and several tiles for each pair of CTAs."""
    m = 1500
    g = gen(K + N)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m) / (4 * K ** 0.5), bytes_(g, N, K), scale(g, N)
    check_product(x, xs, w, ws, act, [BF, F32, HF][K // 16 % 3])


@pytest.mark.parametrize("m", [2, 5, 20, 60, 140])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
def test_longest_products(m, act):
    K, N = arn.AR_I8_MAX_K, 130
    g = gen(m)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N) / 300
    check_product(x, xs, w, ws, act, F32)


@pytest.mark.parametrize("m,N,act,dtype", [(70000, 32768, "none", BF), (140001, 32772, "silu_mul", HF),
                                           (5, 1048576, "none", F32), (40, 1048575, "none", BF)])
def test_outputs_past_32_bits_and_the_widest(m, N, act, dtype):
    K = 32
    g = gen(N)
    x, xs, w, ws = bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N) / 8
    out = arn.ar_i8_matmul(x, xs, w, ws, act=act, dtype=dtype)
    for rows in (slice(0, 3), slice(m // 2, m // 2 + 3), slice(m - 3, m)):
        y, ey = ref.product(x[rows], xs[rows], w, ws, act)
        within(out[rows], y, ey, dtype)


def test_quantise_past_32_bits():
    m, K = 38000, 57344
    x = torch.empty((m, K), dtype=BF, device=DEV).normal_(generator=gen(1))
    q, s = arn.ar_i8_quantize(x)
    for rows in (slice(0, 2), slice(37448, 37452), slice(m - 2, m)):  # 2^31 elements: row 37449
        rq, rs = ref.quantise(x[rows])
        assert torch.equal(q[rows], rq) and torch.equal(s[rows], rs)


@pytest.mark.parametrize("post", [False, True])
def test_block_past_32_bits(post):
    m, H = 270000, 8192
    g = gen(2)
    p, res, w, kw = block_inputs(g, m, H, 1, BF, None, post, "channel", 0.0)
    out, rout = arn.ar_block_rmsnorm(p, res, w, 1e-6, **kw)
    q, s, rout2 = arn.ar_block_rmsnorm_i8(p, res, w, 1e-6, **kw)
    for rows in (slice(0, 2), slice(262143, 262146), slice(m - 2, m)):
        y, ey, r, er = ref.block([p[0][rows]], res[rows], w, 1e-6, **kw)
        within(out[rows], y, ey, BF)
        within(rout[rows], r, er, BF)
        assert torch.equal(rout2[rows], rout[rows])
        step = s[rows].double().unsqueeze(1)
        assert bool(((q[rows].double() * step - y).abs() <= step * 0.5001 + 2 * ey + 2 ** -20 * y.abs()).all())


@pytest.mark.parametrize("m,H,n,rkind", [(90, 73728, 2, None), (100, 131072, 1, "f32"), (300, 16392, 3, None),
                                         (400, 8200, 1, "f32"), (2000, 64, 2, None), (700, 8, 3, "f32"),
                                         (76, 2048, 16, None), (77, 1032, 16, None)])
@pytest.mark.parametrize("post", [False, True])
def test_block_long_and_short_rows_of_large_batches(m, H, n, rkind, post):
    g = gen(m + H)
    p, res, w, kw = block_inputs(g, m, H, n, BF, F32 if rkind else None, post, "token", 1.0)
    check_block(p, res, w, 1e-6, block_scale=0.5, **kw)


def test_the_largest_gate_stride_and_a_gate_for_each_token():
    g = gen(3)
    m, H = 6, 512
    p, res, w, _ = block_inputs(g, m, H, 1, BF, None, True, None, 0.0)
    wide = normal(g, 3, 1 << 20)
    check_block(p, res, w, 1e-6, gate=wide[:, 4096:4096 + H])
    check_block(p, res, w, 1e-6, gate=normal(g, m, 2 * H)[:, H:])
    check_block(p, res, w, 1e-6, gate=normal(g, 1, H))


def test_fp16_results_beyond_its_range_are_infinite():
    x = torch.full((20, 64), 127, dtype=torch.int8, device=DEV)
    w = torch.cat([x, -x])[:32]
    one = torch.ones(32, device=DEV)
    for m in (2, 20):
        out = arn.ar_i8_matmul(x[:m], one[:m], w, one, dtype=HF)
        assert bool(torch.isinf(out).all())
        assert bool((out[:, :20] > 0).all()) and bool((out[:, 20:] < 0).all())


def test_gates_far_from_zero():
    """SiLU of gates to +-3e38 and of infinite ones."""
    v = [0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 80.0, -80.0, 88.5, -88.5, 104.0, -104.0, 1e30, -1e30, 3e38, -3e38]
    for m in (3, 40, 300):
        x = torch.zeros((m, 16), dtype=torch.int8, device=DEV)
        x[:, 0] = 1
        w = torch.zeros((32, 16), dtype=torch.int8, device=DEV)
        w[:, 0] = 1
        ws = torch.tensor(v + [1.0] * 16, device=DEV)
        out = arn.ar_i8_matmul(x, torch.ones(m, device=DEV), w, ws, act="silu_mul", dtype=F32)
        g = ws[:16].double()
        want = g * torch.sigmoid(g)
        err = (out.double() - want).abs()
        assert bool((err <= want.abs() * (2 * ref.U * (2 + g.abs()) + 10 * ref.U) + 2.0 ** -126).all()), err


def test_two_threads():
    states = [layer_inputs(gen(60 + i), m) for i, m in enumerate((3, 200))]
    want = [layer(st) for st in states]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = layer(states[i])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_products_beside_other_tensor_core_work():
    """Library products on another stream at the same time."""
    g = gen(70)
    cases = [(20, 4096, 8192), (150, 4096, 8192), (1000, 4096, 8192)]
    inputs = [(bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N)) for m, K, N in cases]
    want = [arn.ar_i8_matmul(*i) for i in inputs]
    a = normal(g, 4096, 4096)
    prod = a @ a
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s):
            others = [a @ a for _ in range(4)]
        got = [arn.ar_i8_matmul(*i) for i in inputs]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and all(torch.equal(prod, o) for o in others)
    assert arn.ar_device_status(0) == arn.AR_OK


def test_no_check_fires_and_results_match_the_normal_build(checklib):  # noqa: F811
    g = gen(80)
    calls = []
    for m, K, N, act in ((1, 32, 1, "none"), (7, 4096, 300, "silu_mul"), (16, 8192, 512, "none"), (30, 144, 64, "none"),
                         (60, 2048, 1001, "none"), (120, 4112, 2050, "silu_mul"), (192, 8192, 4096, "none"),
                         (333, 4112, 1001, "none"), (700, 1040, 5000, "silu_mul"), (3000, 512, 3004, "none")):
        i = (bytes_(g, m, K), scale(g, m), bytes_(g, N, K), scale(g, N))
        calls.append(lambda i=i, act=act: (arn.ar_i8_matmul(*i, act=act),))
    for m, H, n, r in ((1, 7168, 8, None), (3, 131072, 2, F32), (100, 12296, 3, None), (500, 4104, 1, F32), (900, 1024, 5, None)):
        i = block_inputs(g, m, H, n, BF, r, n != 5, "channel", 0.0)
        calls.append(lambda i=i: arn.ar_block_rmsnorm(*i[:3], 1e-6, **i[3]) + arn.ar_block_rmsnorm_i8(*i[:3], 1e-6, **i[3]))
    for m, K in ((1, 8), (77, 5120), (400, 16392), (3, 40000)):
        x = normal(g, m, K)
        calls.append(lambda x=x: arn.ar_i8_quantize(x))
    normal_lib = arn.lib()
    for call in calls:
        want = call()
        arn._lib = checklib
        try:
            got = call()
            torch.cuda.synchronize()
        finally:
            arn._lib = normal_lib
        assert checklib.ar_device_status(0, 0) == arn.AR_OK
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_canaries_around_small_outputs():
    g = gen(90)
    for m in (1, 5, 17, 33, 65, 129, 257):
        for N in (1, 3, 62, 127, 129):
            x, xs, w, ws = bytes_(g, m, 48), scale(g, m), bytes_(g, N, 48), scale(g, N)
            for dtype in (BF, HF, F32):
                out, ok = guarded((m, N), dtype)
                arn.ar_i8_matmul(x, xs, w, ws, out=out)
                assert ok(), (m, N, dtype)
