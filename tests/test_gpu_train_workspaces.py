"""One workspace, of the size for a larger batch, serves smaller ones: equal bits, and nothing behind its end."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.train_util import rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def guarded(size):
    """A workspace of size bytes and the 4096 marked ones behind it."""
    whole = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole[:size], whole[size:]


@pytest.mark.parametrize("small,large", [(1039, 1040), (1040, 2080), (700, 33000), (32831, 32832)])
def test_activation_gradient(small, large):
    N = 2048
    z, dy = rand((small, N), BF, 1).cuda(), rand((small, N), BF, 2).cuda()
    ws, behind = guarded(Q.moe_expert_act_backward_workspace_size(1, N, large))
    roomy = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    got = []
    for w in (ws, roomy):
        dz, db = torch.zeros_like(z), torch.zeros((1, N), device="cuda")
        Q.moe_expert_act_backward(dy, z, None, dz, db, act=Q.MOE_ACT_RELU, ws=w)
        got.append((dz, db))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.equal(got[0][0], torch.where(z > 0, dy, torch.zeros_like(dy)))
    assert (behind == 0xA5).all()
