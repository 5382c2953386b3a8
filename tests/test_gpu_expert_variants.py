"""Variants of the expert products that the sizes of other tests do not
reach, against the formulas in 64 bits."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.test_gpu_expert_gemm import run_wgrad

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("sizes,N,K", [([5000], 128, 256), ([4000, 0, 1500, 37], 72, 200)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_weight_gradient_joined_parts(sizes, N, K, dtype, out):
    """Few matrices and many rows: parts of a slot's rows, joined in every output type."""
    assert Q.moe_expert_gemm_wgrad_workspace_size(len(sizes), N, K, sum(sizes)) > 0
    run_wgrad(sizes, N, K, dtype, out, k=2, dy_rows=PAIR, x_rows=TOKEN, seed=N)
