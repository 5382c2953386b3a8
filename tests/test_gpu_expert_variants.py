"""Variants of the expert products that the sizes of other tests do not
reach, against the formulas in 64 bits."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests import test_gpu_expert_w4 as w4
from tests.expert_util import D, batches
from tests.test_gpu_expert_gemm import run_product, run_wgrad, wgrad_ws

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("sizes,N,K", [([5000], 128, 256), ([4000, 0, 1500, 37], 72, 200)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_weight_gradient_joined_parts(sizes, N, K, dtype, out):
    """Few matrices and many rows: parts of a slot's rows, joined in every output type."""
    assert Q.moe_expert_gemm_wgrad_workspace_size(len(sizes), N, K, sum(sizes)) > 0
    run_wgrad(sizes, N, K, dtype, out, k=2, dy_rows=PAIR, x_rows=TOKEN, seed=N)


def uneven(slots, mean, seed):
    """Slot sizes about a mean, one slot empty and one with three times as many rows."""
    g = torch.Generator().manual_seed(seed)
    sizes = [int(v) for v in torch.randint(max(mean - 1, 0), mean + 2, (slots,), generator=g)]
    sizes[3], sizes[7] = 0, 3 * mean
    return sizes


@pytest.mark.parametrize("N", [248, 264])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("mean", [1, 3, 12, 30])
def test_4_bit_two_column_tiles(N, group, mean):
    """More than 512 tiles of 16 columns: a workgroup takes two, the last may have one (N = 264) or half a tile (248)."""
    sizes = uneven(40, mean, mean)
    assert -(-N // 16) * len(sizes) > 512
    w4.run(sizes, N, 384, group, BF if group == 64 else HF, F32, k=2, P=sum(sizes) + 5, x_rows=PAIR, y_rows=PAIR, seed=N)


def test_4_bit_two_column_tiles_of_long_rows():
    """As above with more groups than the table of scales holds."""
    w4.run(uneven(40, 2, 1), 264, 4224, 32, BF, BF, zeros=False, seed=2)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("N,K,mean", [(248, 264, 1), (264, 264, 2), (264, 520, 8), (248, 264, 11), (264, 1544, 2)])
def test_streamed_two_column_tiles(dtype, out, N, K, mean):
    sizes = uneven(40, mean, mean)
    run_product(sizes, N, K, dtype, out, k=2, P=sum(sizes) + sum(sizes) % 2, x_rows=TOKEN, y_rows=PAIR, seed=K)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("sizes", [[33], [48], [40, 0, 55, 1]])
@pytest.mark.parametrize("N,K", [(272, 200), (64, 1544)])
def test_streamed_swiglu_of_four_row_blocks(dtype, out, sizes, N, K):
    run_product(sizes, N, K, dtype, out, act=Q.MOE_ACT_SWIGLU, seed=K)


def test_gradients_against_differences_are_exact():
    """The loss sum(c y) moves by exactly what the gradients say.  It is
    linear in x and in w, and every input is a power of two of 2^-2..2^2: sums
    of at most 48 products of two inputs are multiples of 2^-4 below 2^10, and
    with c multiples of 2^-6 below 2^22 in 64 bits, so nothing rounds."""
    sizes, N, K = [3, 0, 9], 16, 48
    offsets, _ = batches(sizes, 12, 1, 0)
    g = torch.Generator().manual_seed(9)

    def pow2(shape):
        return (2.0 ** torch.randint(-2, 3, shape, generator=g)) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)

    x, w, c = (pow2(s).to(BF) for s in ((12, K), (3, N, K), (12, N)))
    off = offsets.cuda()

    def loss(xv, wv):
        y = torch.zeros((12, N), device="cuda")
        Q.moe_expert_gemm(xv.cuda(), wv.cuda(), off, y)
        return float((y.cpu().to(D) * c.to(D)).sum())

    gx, gw = torch.zeros((12, K), device="cuda"), torch.zeros((3, N, K), device="cuda")
    Q.moe_expert_gemm(c.cuda(), w.cuda(), off, gx, transpose=True)
    Q.moe_expert_gemm_wgrad(c.cuda(), x.cuda(), off, gw, ws=wgrad_ws(3, N, K, 12))
    base, gx, gw = loss(x, w), gx.cpu(), gw.cpu()
    moved = 0
    for i in range(12):
        for j in (0, 5, 17, 31, 32, 47):
            v = x.clone()
            v[i, j] *= 2
            assert loss(v, w) - base == float(gx[i, j]) * float(x[i, j])
            moved += float(gx[i, j]) != 0
    for s, i, j in [(s, i, j) for s in (0, 2) for i in (0, 3, 8, 15) for j in (0, 9, 31, 47)]:
        v = w.clone()
        v[s, i, j] *= 2
        assert loss(x, v) - base == float(gw[s, i, j]) * float(w[s, i, j])
        moved += float(gw[s, i, j]) != 0
    assert moved > 80, "the probes are of coordinates that move the loss"
    assert (gw[1] == 0).all()
