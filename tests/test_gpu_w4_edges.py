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
