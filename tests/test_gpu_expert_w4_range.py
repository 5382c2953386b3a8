"""moe_expert_gemv_w4 with x at the ends of its type's range: the sums of
code x and zero x, which are taken apart, must neither overflow nor vanish
where scale (code - zero) x is a number of ordinary size."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, batches, check_sums, product, w4_magnitude, w4_matrix

pytestmark = pytest.mark.gpu

POS = Q.MOE_ROWS_POSITION
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def run(sizes, N, K, group, dtype, top, scale, act=0, zeros=True, seed=0):
    """x within a factor of two of 2^top, scales around `scale`, zeros over all bytes."""
    P = sum(sizes)
    offsets, _ = batches(sizes, P, 1, seed)
    g = torch.Generator().manual_seed(seed + 1)
    x = ((1.0 + 0.99 * torch.rand((P, K), generator=g, dtype=D)) * 2.0 ** top *
         (torch.randint(0, 2, (P, K), generator=g) * 2 - 1)).to(dtype)
    assert x.isfinite().all()
    q = torch.randint(0, 256, (len(sizes), N, K // 2), generator=g, dtype=torch.uint8)
    scales = (scale * (0.5 + torch.rand((len(sizes), N, K // group), generator=g, dtype=D))).to(F32)
    z = torch.randint(0, 256, scales.shape, generator=g, dtype=torch.uint8) if zeros else None
    want, _, mag = product(x, w4_matrix(q, scales, z, group), offsets, P, None, 1, POS, POS, False, act,
                           w4_magnitude(q, scales, z, group))
    y = torch.empty((P, want.shape[1]), device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), None if z is None else z.cuda(), group, offsets.cuda(), y,
                         act=act)
    check_sums(y.cpu(), want, mag, K, F32, bool(act))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows", [2, 14, 30, 60])
def test_largest_bf16_values(group, zeros, rows):
    run([rows, 0, 1], 48, 640, group, BF, 127, 2.0 ** -120, zeros=zeros, seed=rows)


def test_largest_bf16_values_swiglu():
    run([3, 20], 64, 384, 128, BF, 127, 2.0 ** -124, act=1)


@pytest.mark.parametrize("dtype,top", [(BF, -90), (HF, 15), (HF, -14)])
@pytest.mark.parametrize("rows", [2, 30])
def test_other_ends(dtype, top, rows):
    run([rows, 1], 48, 384, 64, dtype, top, 2.0 ** -(top + 5), seed=rows)
