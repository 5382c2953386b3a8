"""Workspace queries of the activations' gradient and of the router's losses never fall where a size grows: one workspace
for a program's largest batch serves every smaller one.  Without a GPU."""
import pytest

import quantized_routed_expert_moe_amd as Q

ACT, LOSS = Q.moe_expert_act_backward_workspace_size, Q.moe_balance_loss_workspace_size
TOP = 1 << 24


def around(top):
    """1 .. 4500, and the places where the kernels' parts may double: 15 .. 130 (in steps) times a power of two."""
    at = set(range(1, min(top, 4500) + 1)) | {top - 1, top}
    for shift in range(0, 24):
        for m in (*range(15, 34), 63, 64, 65, 127, 128, 129, 1023, 1024, 1025, 1031, 2049):
            at |= {(m << shift) + d for d in (-1, 0, 1)}
    return sorted(a for a in at if 0 < a <= top)


def never_falls(size, values):
    last = 0
    for v in values:
        n = size(v)
        assert n >= last > -1, f"{v} needs {n} bytes, a smaller size {last}"
        last = n
    assert last > 0


@pytest.mark.parametrize("N", [8, 16, 32, 136, 256, 264, 1536, 2048, 7168, 1 << 20])
@pytest.mark.parametrize("S", [1, 7, 128, 1024])
def test_activation_gradient_over_rows(S, N):
    never_falls(lambda r: ACT(S, N, r), around(TOP))


@pytest.mark.parametrize("R", [1, 17, 1039, 1040, 32831, 32832, 1 << 20])
def test_activation_gradient_over_columns_and_slots(R):
    for S in (1, 64):
        never_falls(lambda n: ACT(S, 8 * n, R), range(1, 3000))
    for N in (8, 264, 2048):
        never_falls(lambda s: ACT(s, N, R), range(1, 1025))


@pytest.mark.parametrize("E", [1, 8, 64, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("G", [1, 8, 1024])
def test_router_losses_over_rows(E, G):
    never_falls(lambda t: LOSS(t, E, G), around(TOP))


@pytest.mark.parametrize("T", [0, 1, 64, 1039, 4111, 4112, 32831, 32832, TOP])
def test_router_losses_over_experts_and_sequences(T):
    for G in (1, 8, 1024):
        never_falls(lambda e: LOSS(T, e, G), range(1, 1025))
    for E in (16, 256, 257):
        never_falls(lambda g: LOSS(T, E, g), range(1, 1025))


def test_a_workspace_of_the_largest_batch_is_not_refused():
    """Past the size check of a smaller batch the next refusal is that of the address: nothing is enqueued."""
    fake = 1 << 20
    for small, large in ((1039, 1040), (32831, 32832), (32831, 43712)):
        for ws, want, needle in ((ACT(1, 2048, large), Q.MOE_ERR_INVALID_ARGUMENT, "workspace must"),
                                 (16, Q.MOE_ERR_WORKSPACE_TOO_SMALL, "needed")):
            st = Q.lib().moe_expert_act_backward(fake, fake * 2, Q.MOE_BF16, 1, 2048, None, small, None, 0, Q.MOE_ACT_GELU,
                                                 fake * 3, None, fake * 5, fake + 8, ws, None)
            assert st == want and needle in Q.lib().moe_last_error().decode(), (small, large)
    for E, small, large in ((256, 32831, 32832), (1000, 4111, 4112)):
        st = Q.lib().moe_balance_loss(fake, fake, small, E, 8, 0, fake, 8, fake, fake, fake, fake + 8, LOSS(large, E, 8), None)
        assert st == Q.MOE_ERR_INVALID_ARGUMENT and "workspace must" in Q.lib().moe_last_error().decode(), (small, large)
