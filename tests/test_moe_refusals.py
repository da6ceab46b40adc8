"""What an ExpertLayer is not made of."""
import pytest
import torch


def operands(up_experts, down_experts):
    def w4(*shape):
        return torch.zeros(shape, dtype=torch.uint8), torch.zeros((*shape[:2], 1)), None
    return torch.zeros((8, 64), dtype=torch.bfloat16), w4(up_experts, 64, 32), w4(down_experts, 64, 16)


@pytest.mark.parametrize("up,down", [(4, 3), (3, 4), (8, 1)])
def test_up_and_down_hold_the_same_experts(up, down):
    """The missing ones' rows would be zeros, as another rank's are."""
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    router, u, d = operands(up, down)
    with pytest.raises(ValueError, match="experts and down"):
        ExpertLayer(router, u, d, 2)


def test_what_is_taken():
    from allreduce_sum_residual_gb300.moe import ExpertLayer
    layer = ExpertLayer(*operands(4, 4), 2, first=4)
    assert layer.first == 4 and layer.group is None
