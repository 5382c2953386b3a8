"""The expert products, block norms and SwiGLU refuse a tensor that requires
a gradient while gradients are enabled: no call records itself for autograd,
so the gradient would silently end there."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device(monkeypatch):
    """CPU tensors pass the device check, and a call that passes every check of the binding ends before the library."""
    monkeypatch.setattr(Q, "_op_device", lambda: (Q._op_types(), -1)[1])

    class Reached(Exception):
        pass

    def reached():
        raise Reached

    monkeypatch.setattr(Q, "lib", reached)
    return Reached


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


CALLS = {
    "moe_expert_gemm": (dict(x=t(4, 16), w=t(2, 8, 16), slot_offsets=i32(3), y=t(4, 8)), ("x", "w", "y")),
    "moe_expert_gemm_wgrad": (dict(dy=t(4, 8), x=t(4, 16), slot_offsets=i32(3), dw=t(2, 8, 16)), ("dy", "x", "dw")),
    "moe_expert_gemv_w4": (dict(x=t(4, 64), q=t(2, 8, 32, dtype=torch.uint8), scales=t(2, 8, 2), zeros=None, group=32,
                                slot_offsets=i32(3), y=t(4, 8)), ("x", "scales", "y")),
    "moe_block_norm": (dict(x=t(4, 64), y=t(4, 64), w_post=t(64), gate=t(64), w_pre=t(64), x_out=t(4, 64), h=t(4, 64),
                            eps=1e-6), ("x", "y", "w_post", "gate", "w_pre", "x_out", "h")),
    "moe_block_norm_backward": (dict(x=t(4, 64), y=None, w_post=None, gate=None, w_pre=t(64), dx_out=None, dh=t(4, 64),
                                     dx=t(4, 64), dy=None, dw_post=None, dgate=None,
                                     dw_pre=t(64, dtype=torch.float32), eps=1e-6), ("x", "w_pre", "dh", "dx", "dw_pre")),
    "moe_swiglu": (dict(gu=t(4, 16), h=t(4, 8)), ("gu", "h")),
    "moe_swiglu_backward": (dict(gu=t(4, 16), dh=t(4, 8), dgu=t(4, 16)), ("gu", "dh", "dgu")),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_a_tensor_that_requires_a_gradient_is_refused(call, name, _device):
    a = dict(CALLS[call][0])
    with pytest.raises(_device):
        getattr(Q, call)(**a)
    a[name] = a[name].clone().requires_grad_()
    with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
        getattr(Q, call)(**a)
    with torch.no_grad(), pytest.raises(_device):
        getattr(Q, call)(**a)


def test_calls_within_an_autograd_function_pass(_device):
    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            with pytest.raises(_device):
                Q.moe_expert_gemm(x, w, i32(3), t(4, 8))
            return x.new_zeros((4, 8))

    Product.apply(t(4, 16).requires_grad_(), t(2, 8, 16).requires_grad_())
