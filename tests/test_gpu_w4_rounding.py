"""The 4-bit products within the roundings that their sums take.

Of one output: a group's products, sixteen at a time, each step of which may
lose 2^-23 of the magnitudes so far (2 half-steps of fp32); one rounding of
the group's sum times its scale added to the sum so far, K / G of them at
most, in one warp; up to 15 adds that join a team's warps; an add a phase, of
which there are at most as many as units of 128 k.  That is 2 G / 16 + K / G +
15 + K / 128 half-steps of sum |q - z| |s| |x|.  The power of two of a column
and its way back are exact; of elements under 2^-30 of their row's largest up
to 2^-39 of that is lost."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
import experts_ref as ref
from test_gpu_experts import DEV, EXPERTS, MATVEC, gen, normal, weights4

pytestmark = pytest.mark.gpu


def product(x, q, s, z):
    K = x.shape[1]
    group = K // s.shape[-1]
    w, x = ref.unpack(q, s, z), x.double()
    steps = 2 * group / 16 + K / group + 15 + K / 128
    tiny = 2.0 ** -39 * 15 * x.abs().amax(1, keepdim=True) * group * s.double().abs().sum(1)
    return x @ w.T, steps * ref.F32 * (x.abs() @ w.abs().T) + tiny


@pytest.mark.parametrize("m,K,N,group,kind,zeros,act", MATVEC)
def test_dense(m, K, N, group, kind, zeros, act):
    g = gen(7 * m + K + N)
    x = normal(g, m, K)
    q, s, z = weights4(g, (N,), K, group, kind, zeros)
    ref.close(arn.ar_w4_matvec(x, q, s, zeros=z, act=act), *ref.act(*product(x, q, s, z), act))


@pytest.mark.parametrize("m,E,k,K,N,group,kind,zeros,act,per_pair,missing", EXPERTS)
def test_experts(m, E, k, K, N, group, kind, zeros, act, per_pair, missing):
    g = gen(7 * m + E + K)
    x = normal(g, m, k, K) if per_pair else normal(g, m, K)
    ids = torch.randint(0, E, (m, k), generator=g, device=DEV, dtype=torch.int32)
    q, s, z = weights4(g, (E, N), K, group, kind, zeros)
    out = arn.ar_w4_matvec_experts(x, ids, q, s, zeros=z, act=act).flatten(0, 1)
    rows = x.reshape(m * k, K) if per_pair else x.repeat_interleave(k, 0)
    for e in range(E):
        at = (ids.flatten() == e).nonzero().flatten()
        if len(at):
            y, err = product(rows[at], q[e], s[e], None if z is None else z[e])
            ref.close(out[at], *ref.act(y, err, act))
