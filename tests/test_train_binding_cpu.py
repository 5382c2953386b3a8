"""The binding of the products and gradient lists on host tensors, without a GPU: every call here is refused, or stops,
before anything is enqueued."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q

LATER = [Q.MOE_ACT_SILU, Q.MOE_ACT_GELU, Q.MOE_ACT_GELU_TANH, Q.MOE_ACT_RELU]


@pytest.fixture(autouse=True)
def host(monkeypatch):
    """Host tensors count as the current device's (theirs is -1)."""
    Q._op_types()
    monkeypatch.setattr(Q, "_op_device", lambda: -1)


@pytest.mark.parametrize("act", LATER)
@pytest.mark.parametrize("width", [32, 16])
def test_products_name_an_activation_they_do_not_take(act, width):
    """Not y's shape: that is N wide for all of them."""
    x, y = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, width), dtype=torch.bfloat16)
    with pytest.raises(Q.QmoeError, match="act"):
        Q.moe_expert_gemm(x, torch.zeros((1, 32, 64), dtype=torch.bfloat16), None, y, act=act, stream=0)
    with pytest.raises(Q.QmoeError, match="act"):
        Q.moe_expert_gemv_w4(x, torch.zeros((1, 32, 32), dtype=torch.uint8), torch.zeros((1, 32, 2)), None, 32, None, y,
                             act=act, stream=0)
