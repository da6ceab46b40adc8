"""8-bit products and the sums on the way to them: whole numbers up to 2^24
whatever the launch shape, for one and two tokens at any size, and beyond that
within the bound that the header gives.

With scales of 1 an fp32 output is the sum itself.  Each of K / 16 additions to
an fp32 sum, and of up to seven between parts of K, is off by at most a step,
2^-23 of a sum that no sum of magnitudes is below."""
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_dense import DEV, F32
from test_gpu_experts import gen, guarded

pytestmark = pytest.mark.gpu

# Batches and matrices that take dot products, one CTA a tile and pairs of every
# size, alone and in parts of K.
MS = (1, 2, 3, 8, 16, 20, 32, 40, 64, 100, 130, 200, 256, 400, 600)


def between(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int8)


def sums(x, w):
    """Whole numbers, exact in 64 bits."""
    total = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    for a in range(0, x.shape[1], 1024):  # at most 2^24 each: exact in fp32 in any order
        total += (x[:, a:a + 1024].float() @ w[:, a:a + 1024].float().T).double()
    return total


def product(x, w):
    one = torch.ones(max(x.shape[0], w.shape[0]), device=DEV)
    out, ok = guarded((x.shape[0], w.shape[0]), F32)
    arn.ar_i8_matmul(x, one[:x.shape[0]], w, one[:w.shape[0]], out=out)
    torch.cuda.synchronize()
    assert ok()
    return out


@pytest.mark.parametrize("lo", [64, 126])
@pytest.mark.parametrize("N", [96, 1000, 4098])
def test_any_1024_products_add_up_exactly(lo, N):
    g = gen(N + lo)
    x, w = between(g, lo, 127, max(MS), 1024), between(g, lo, 127, N, 1024)
    S = sums(x, w).float()
    for m in MS:
        assert torch.equal(product(x[:m], w), S[:m]), m


@pytest.mark.parametrize("K,N", [(2048, 1000), (7168, 2000), (16384, 200)])
def test_sums_that_go_out_to_2_24_and_back(K, N):
    """Blocks of 512 k of one sign: no sum passes 2^24 wherever it starts."""
    g = gen(K)
    x, w = between(g, 100, 127, max(MS), K), between(g, 100, 127, N, K)
    for a in range(512, K, 1024):
        w[:, a:a + 512] = -w[:, a:a + 512]
    w[:, K - 1] = 1
    S = sums(x, w).float()
    for m in MS:
        assert torch.equal(product(x[:m], w), S[:m]), m


@pytest.mark.parametrize("kind", ["one sign", "cancelling", "odd"])
@pytest.mark.parametrize("K,N", [(1040, 1000), (4096, 512), (7168, 2000), (16384, 200), (131056, 96)])
def test_sums_past_2_24(K, N, kind):
    """One and two tokens exactly, more within K / 16 + 8 steps; equal calls equal."""
    g = gen(K + N)
    x, w = between(g, 64, 127, max(MS), K), between(g, 64, 127, N, K)
    if kind == "cancelling":  # far out and back again
        w[:, K // 2:] *= -1
    elif kind == "odd":       # a 1 that a step of more than 1 would drop
        x.fill_(127)
        w.fill_(127)
        w[:, K - 1] = 126
    S = sums(x, w)
    bound = (K / 16 + 8) * 2.0 ** -23 * sums(x, w.abs())
    for m in MS:
        got = product(x[:m], w)
        if m <= 2:
            assert torch.equal(got, S[:m].float()), m
        else:
            assert bool(((got.double() - S[:m]).abs() <= bound[:m]).all()), m
            assert torch.equal(product(x[:m], w), got)


@pytest.mark.parametrize("m", [1, 5, 40, 130, 500])
def test_bytes_of_either_sign_stay_exact_at_any_length(m):
    """Bytes spread evenly over all values: sums grow with the root of K."""
    g = gen(m)
    for K, N in ((16384, 400), (131056, 80)):
        x, w = between(g, -128, 127, m, K), between(g, -128, 127, N, K)
        assert torch.equal(product(x, w), sums(x, w).float())
