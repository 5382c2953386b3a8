"""The binding of the products and gradient lists on host tensors, without a GPU: every call here is refused, or stops,
before anything is enqueued."""
import weakref

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


def test_a_kept_list_does_not_keep_its_outputs():
    """Gradients and outputs are compared once for a pair of kept lists; what is remembered of it holds no memory."""
    grads = Q._TensorList([torch.zeros(5), torch.zeros(7)])
    outs = Q._TensorList([torch.zeros(5), torch.zeros(7)])
    gone = weakref.ref(outs)
    Q._op_apart(grads, outs)
    del outs
    assert gone() is None
    gone = weakref.ref(grads)
    Q._op_apart(grads, grads)  # in place
    del grads
    assert gone() is None


def test_lists_are_compared_once(monkeypatch):
    """A pair of kept lists is not looked at again; another list, also one that overlaps, is."""
    monkeypatch.setattr(Q, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(Q, "_check", lambda status: None)
    flat, looked = torch.zeros(32), []
    apart = Q._op_apart
    monkeypatch.setattr(Q, "_op_apart", lambda a, b: (looked.append(b), apart(a, b))[1])

    class Silent:
        moe_grad_clip = staticmethod(lambda *a: 0)

    monkeypatch.setattr(Q, "lib", lambda: Silent)
    kept = object.__new__(Q.moe_tensor_list)
    Q._TensorList.__init__(kept, [flat[:8], flat[8:16]])
    total, first, second = torch.zeros(1), object.__new__(Q.moe_tensor_list), object.__new__(Q.moe_tensor_list)
    Q._TensorList.__init__(first, [torch.zeros(8), torch.zeros(8)])
    Q._TensorList.__init__(second, [flat[:8], flat[8:16]])
    for outs, times in ((first, 1), (first, 1), (second, 2), (second, 2), (first, 3)):
        Q.moe_grad_clip(kept, total, 1.0, outs=outs)
        assert len(looked) == times
    del first, second, outs
    looked.clear()
    for _ in range(3):  # plain lists are new each time, wherever their objects lie
        with pytest.raises(ValueError, match="overlaps"):
            Q.moe_grad_clip(kept, total, 1.0, outs=[flat[4:12], torch.zeros(8)])
    assert len(looked) == 3
