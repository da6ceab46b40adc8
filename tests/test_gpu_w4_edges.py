"""The 4-bit products at the ends of their arguments' ranges."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import experts_ref as ref
from test_gpu_experts import DEV, expert_rows, gen, normal, weights4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,E", [(2 ** 31 - 1, 4), (2 ** 31 - 3, 8), (2 ** 31 - 512, 512), (1, 3)])
def test_no_id_wraps_into_the_experts_of_a_rank(first, E):
    """`first` near the end of int32: only ids from `first` on are here, not
    those that wrap around to behind it."""
    g = gen(81)
    x = normal(g, 6, 128)
    q, s, z = weights4(g, (E, 24), 128, 64, "bf16", True)
    low = -2 ** 31
    ids = torch.tensor([[first, low], [low + 1, 2 ** 31 - 1], [low + E - 1, first - 1],
                        [-1, low + 2], [0, low + 5], [min(first + 1, 2 ** 31 - 1), low + 7]],
                       dtype=torch.int64, device=DEV).int()
    here = (ids.long() >= first) & (ids.long() < first + E)
    local = torch.where(here, ids.long() - first, -1).int()
    for st in (None, torch.cuda.current_stream()):
        out = arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z, first=first, stream=st)
        ref.close(out, *expert_rows(x, local, q, s, z, "none"))
        assert not bool(out[~here].any())


@pytest.mark.parametrize("kind,big", [("f32", 2.0 ** 126), ("bf16", 2.0 ** 126), ("f32", 2.0 ** -120),
                                      ("bf16", 2.0 ** -120), ("f32", 2.0 ** 100), ("bf16", 2.0 ** 112)])
@pytest.mark.parametrize("m,K,group", [(1, 256, 32), (3, 192, 64), (9, 384, 128), (16, 1024, 64),
                                       (1, 7168, 128), (16, 7168, 128)])
def test_scales_at_one_end_of_their_range_and_x_at_the_other(kind, big, m, K, group):
    """Ordinary results from scales that fp32 just holds: no sum on the way
    leaves its range, in one phase or several."""
    g = gen(82)
    x = (torch.randint(-8, 9, (m, K), generator=g, device=DEV).double() / big).bfloat16()
    for N, act in ((40, "none"), (64, "silu_mul")):
        q, s, z = weights4(g, (N,), K, group, "f32", True)
        s = (s.double() * big).to(torch.float32 if kind == "f32" else torch.bfloat16)
        for zeros in (None, z):
            out = arn.ar_w4_matvec(x, q, s, zeros=zeros, act=act)
            y, err = ref.act(*ref.product(x, q, s, zeros), act)
            assert bool(y.isfinite().all())
            ref.close(out, y, err)


def test_results_next_to_the_largest_number():
    """Results of 2^120 and more, which the row's power of two once passed."""
    g = gen(83)
    x = normal(g, 5, 512)
    q, s, z = weights4(g, (48,), 512, 64, "f32", True)
    s = s * 2.0 ** 122
    ids = torch.randint(0, 3, (5, 2), generator=g, device=DEV, dtype=torch.int32)
    out = arn.ar_w4_matvec(x, q, s, zeros=z)
    y, err = ref.product(x, q, s, z)
    assert float(y.abs().max()) > 2.0 ** 121
    ref.close(out, y, err)
    qe, se, ze = (t.expand(3, *t.shape).contiguous() for t in (q, s, z))
    ref.close(arn.ar_w4_matvec_experts(x, ids, qe, se, zeros=ze), *expert_rows(x, ids, qe, se, ze, "none"))


@pytest.mark.parametrize("per_pair,act", [(False, "none"), (True, "silu_mul")])
@pytest.mark.parametrize("m,K,N,group,zeros", [(40, 256, 400, 128, False), (20, 96, 5000, 32, True),
                                               (9, 8192, 30, 64, False)])
def test_experts_with_scales_at_the_end_of_their_range(m, K, N, group, zeros, per_pair, act):
    """Several column sets of an expert, ranges of items over many blocks,
    several phases; a row of ordinary numbers and ids that are not here."""
    g = gen(85)
    x = torch.randint(-8, 9, (m, 2, K) if per_pair else (m, K), generator=g, device=DEV).double()
    x = (x * 2.0 ** -110).bfloat16()
    q, s, z = weights4(g, (3, N), K, group, "f32", True)
    s = s * 2.0 ** 112
    s[1, ::2] *= 2.0 ** -60
    z = z if zeros else None
    ids = torch.randint(-1, 3, (m, 2), generator=g, device=DEV, dtype=torch.int32)
    out = arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z, act=act)
    y, err = expert_rows(x, ids, q, s, z, act)
    ref.close(out, y, err)
    assert not bool(out[ids < 0].any())
    assert torch.equal(out, arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z, act=act))
    x2 = x.reshape(-1, K)[:33]
    ref.close(arn.ar_w4_matvec(x2, q[0], s[0], zeros=None if z is None else z[0], act=act),
              *ref.act(*ref.product(x2, q[0], s[0], None if z is None else z[0]), act))


def test_rows_without_a_number_stay_so():
    """NaN and infinite x, scales and results come out as the formula has
    them, beside outputs that had to be computed again."""
    g = gen(84)
    x = normal(g, 6, 320) * 2.0 ** -20
    q, s, z = weights4(g, (70,), 320, 64, "f32", True)
    s = s.abs() + 0.01
    s[3] = 2.0 ** 110   # past fp32's end on the way for the small rows
    s[7, 2] = float("nan")
    s[9, 1] = float("inf")
    s[11] = 2.0 ** 127
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    x[4] = normal(g, 320)
    q[:, :] = (q & 0x77) | 0x88          # codes 8 .. 15
    z[:] = 2                             # weights are positive
    x = x.abs()
    x[5] *= 2.0 ** -40
    out = arn.ar_w4_matvec(x, q, s, zeros=z)
    y, err = ref.product(x, q, s, z)
    plain = [0, 3, 5]
    rows = [i for i in range(70) if i not in (7, 9)]
    big = y[plain][:, rows].abs() > 3.39e38
    got = out[plain][:, rows]
    ref.close(torch.where(big, 0, got), torch.where(big, 0.0, y[plain][:, rows]),
              torch.where(big, 1.0, err[plain][:, rows]))
    assert bool((got[big] == float("inf")).all())
    assert bool(out[1].isnan().all()) and bool(out[:, 7].isnan().all())
    assert bool((out[2, rows] == float("inf")).all())
    assert bool((out[plain, 9] == float("inf")).all())


def test_overflow_keeps_its_sign_next_to_the_largest_x():
    """x so large that a group's sum of products alone passes fp32's end: the
    result is infinite or a number as the scaled sums have it, never NaN."""
    x = torch.full((2, 128), 2.0 ** 126, dtype=torch.bfloat16, device=DEV)
    q = torch.full((4, 64), 0xFF, dtype=torch.uint8, device=DEV)   # 7
    q[1:, 32:] = 0                                                # -8 behind 64
    s = torch.tensor([[1.0, 1.0], [1.0, 0.25], [2.0 ** -60, 2.0 ** -60], [8.0, 7.0]], device=DEV)
    out = arn.ar_w4_matvec(x, q, s)
    inf = float("inf")
    assert out[:, [0, 1]].tolist() == [[inf, inf]] * 2
    assert bool((out[:, 2] == -64 * 2.0 ** 66).all()) and not bool(out[:, 3].isnan().any())


@pytest.mark.parametrize("m,K,N,act", [(16, 6144, 32768, "silu_mul"), (16, 2048, 32768, "none"),
                                       (1, 7168, 7168, "none")])
def test_rows_of_nan_take_no_more_time(m, K, N, act):
    """A padded batch's garbage: its outputs are not taken for sums that passed
    fp32's end, in whichever phase it lies."""
    g = gen(86)
    x = normal(g, m, K)
    bad = x.clone()
    bad[m // 2:, [3, K - 5]] = float("nan")
    bad[m // 2:, 40] = float("inf")
    only_first, only_last = x.clone(), x.clone()
    only_first[0, 3], only_last[0, K - 5] = float("nan"), float("inf")
    q, s, _ = weights4(g, (N,), K, 128, "bf16", False)

    def time(x):
        best = float("inf")
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(3):
                arn.ar_w4_matvec(x, q, s, act=act)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    usual = time(x)
    for other in (bad, only_first, only_last):
        assert time(other) < 2 * usual
