"""Block norms at widths between those of the other tests and at the ends of
their ranges: gradients that do not depend on a tensor whose values are
infinite, NaN or near the largest."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, EPS16
from tests.test_gpu_block_norm import EPS, F, close, dev, formula, make, run_both

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("H", [136, 2304, 8200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_gradient_without_a_next_norm_does_not_depend_on_x(H, dtype, post, gate):
    """x_out = a x + gate r alone: no gradient holds x, whatever its values are."""
    T, a = 4, 1.5
    t = make(T, H, dtype, BF, F32, post, gate, False, seed=H)
    t["x"][0, :] = 3e38 * t["x"][0].sign()  # a x and sums with x overflow
    t["x"][1, 5], t["x"][1, H - 1], t["x"][2, 0] = float("inf"), -float("inf"), float("nan")
    _, _, grads = formula(t, a)
    c = {k: dev(v) for k, v in t.items()}
    dx, dy = torch.empty_like(c["x"]), torch.empty_like(c["y"])
    f = lambda w: None if w is None else torch.full(w.shape, float("nan"), device="cuda")  # noqa: E731
    dw_post, dgate = f(t["w_post"]), f(t["gate"])
    ws = torch.empty(Q.moe_block_norm_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    Q.moe_block_norm_backward(c["x"], c["y"], c["w_post"], c["gate"], None, c["dx_out"], None, dx, dy, dw_post, dgate,
                              None, EPS, a, ws)
    # dx is one product, rounded in fp32 and once more
    close(dx, grads["x"], EPS16[dtype] + F, 0.0, "dx")
    # the other bounds are those of test_gpu_block_norm.run_both
    big = max(grads["y"].abs().amax().item(), t["dx_out"].abs().amax().item())
    close(dy, grads["y"], EPS16[BF], 200 * F * big, "dy")
    for name, d in (("w_post", dw_post), ("gate", dgate)):
        if d is not None:
            n = H if name == "gate" and gate == "token" else T
            close(d, grads[name], 0.0, (n ** 0.5 * 200 + 8 * n ** 0.5 * min(n, 64) ** 0.5) * F * 8.0 * big, "d" + name)
    assert dx.to(D).isfinite().all()


@pytest.mark.parametrize("H", [136, 248, 256])
@pytest.mark.parametrize("T", [1, 5, 333])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_widths_of_eight_rows_a_workgroup(H, T, gate):
    run_both(T, H, BF, F32, F32, True, gate, True, 0.5, seed=T)


@pytest.mark.parametrize("H,gate", [(136, "channel"), (256, "token")])
def test_workgroups_that_walk_several_steps(H, gate):
    """More rows than 512 workgroups of eight take at once, the last step a partial one."""
    run_both(9003, H, HF, BF, HF, True, gate, True, seed=H)
