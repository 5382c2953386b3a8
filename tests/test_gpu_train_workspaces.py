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


@pytest.mark.parametrize("E,small,large", [(256, 32831, 32832), (1000, 4111, 4112), (16, 100, 40000), (256, 300, 301)])
def test_router_losses(E, small, large):
    G, k = 8, 4
    l = rand((small, E), F32, 1).cuda()
    ids = torch.randint(0, E, (small, k), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    off = torch.linspace(0, small, G + 1).int().cuda()
    ws, behind = guarded(Q.moe_balance_loss_workspace_size(large, E, G))
    roomy = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    got = []
    for w in (ws, roomy):
        counts = torch.zeros((G, E), dtype=torch.int32, device="cuda")
        probs, losses = torch.zeros((G, E), device="cuda"), torch.zeros(2, device="cuda")
        Q.moe_balance_loss(l, ids, Q.MOE_SCORE_SOFTMAX, counts, probs, losses, off, ws=w)
        got.append((counts, probs, losses))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert int(got[0][0].sum()) == small * k and (behind == 0xA5).all()
