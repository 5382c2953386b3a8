"""Weight gradients of slots with few or no rows: every count about a stage of
64 and a step of 16 rows, matrices whose rows end inside a cache line, both
tile sizes, parts of a split without rows."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.test_gpu_expert_gemm import run_wgrad

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("sizes", [[0, 0, 1], [15, 0, 16, 17], [31, 33, 47, 49, 0], [63, 64, 65, 66, 0, 127, 128]])
@pytest.mark.parametrize("N,K", [(8, 8), (128, 128), (136, 200), (264, 424)])
@pytest.mark.parametrize("dtype,out", [(BF, F32), (HF, HF)])
def test_few_rows(sizes, N, K, dtype, out):
    P = sum(sizes) + 3
    run_wgrad(sizes, N, K, dtype, out, k=2, P=P, dy_rows=PAIR, x_rows=TOKEN, seed=N)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF)])
@pytest.mark.parametrize("K", [1024, 1032])
def test_few_rows_beside_many(dtype, out, K):
    """The 256 x 256 tiles: enough of them, and enough rows on average."""
    sizes = [0, 1, 16, 17, 40, 64, 65, 0, 1800, 0, 1700, 3, 2000, 64, 0, 5, 600]
    run_wgrad(sizes, 1032, K, dtype, out, k=2, dy_rows=POS, x_rows=PAIR, seed=K)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("N,K", [(1032, 1024), (1000, 1032)])
def test_no_row_in_most_slots(N, K, out):
    """The zeros of a whole slot, and no other slot's, are written."""
    run_wgrad([0] * 13 + [2] + [0] * 8, N, K, BF, out, seed=1)
    sizes = [0, 2, 0, 0]
    off = torch.tensor([0, 0, 2, 2, 2], dtype=torch.int32, device="cuda")
    x, dy = torch.ones((5, K), dtype=BF, device="cuda"), torch.ones((5, N), dtype=BF, device="cuda")
    store = torch.full((6, N, K), 7.0, dtype=out, device="cuda")
    Q.moe_expert_gemm_wgrad(dy, x, off, store[1:5])
    assert (store[[0, 5]] == 7.0).all()
    assert all((store[1 + s] == n).all() for s, n in enumerate(sizes))


def test_parts_without_rows():
    """Three slots whose rows are split, one of them with a row, one with none."""
    sizes, N, K = [5000, 0, 1], 72, 200
    assert Q.moe_expert_gemm_wgrad_workspace_size(3, N, K, sum(sizes)) > 0
    run_wgrad(sizes, N, K, BF, F32, seed=5)


def test_nan_stays_in_its_slot():
    """Rows behind a slot's last, also of the same stage, add nothing to it: not a NaN either."""
    N, K = 136, 200
    dy, x = torch.ones((70, N), dtype=BF), torch.ones((70, K), dtype=BF)
    x[20:], dy[20:] = float("nan"), float("inf")
    off = torch.tensor([0, 3, 20, 70], dtype=torch.int32)
    dw = torch.empty((3, N, K), device="cuda")
    Q.moe_expert_gemm_wgrad(dy.cuda(), x.cuda(), off.cuda(), dw)
    assert (dw[0] == 3).all() and (dw[1] == 17).all() and dw[2].isnan().all()
