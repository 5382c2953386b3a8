"""moe_expert_gemv_w4 against its formula in 64 bits: groups, zero points,
scale types, row counts from one to many a slot, odd sizes and row modes."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import batches, check_sums, product, w4_magnitude, w4_matrix

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def weights(S, N, K, group, dtype, zeros, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (S, N, K // 2), generator=g, dtype=torch.uint8)
    scales = (0.05 * torch.exp(0.5 * torch.randn((S, N, K // group), generator=g))).to(dtype)
    z = torch.randint(0, 16, (S, N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    return q, scales, z


def dev(t):
    return None if t is None else t.cuda()


def run(sizes, N, K, group, dtype=BF, out=BF, scale_dtype=None, zeros=True, k=1, P=None, x_rows=POS, y_rows=POS, act=0,
        seed=0):
    P = sum(sizes) if P is None else P
    offsets, perm = batches(sizes, P, k, seed)
    x = torch.randn((-(-P // k) if x_rows == TOKEN else P, K), generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    q, scales, z = weights(len(sizes), N, K, group, scale_dtype or dtype, zeros, seed + 2)
    want, written, mag = product(x, w4_matrix(q, scales, z, group), offsets, P, perm, k, x_rows, y_rows, False, act,
                                 w4_magnitude(q, scales, z, group))
    mark = -77.0
    y = torch.full((P, want.shape[1]), mark, dtype=out, device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), dev(z), group, offsets.cuda(), y, perm.cuda(), k, x_rows,
                         y_rows, act)
    got = y.cpu()
    assert (got[~written] == mark).all(), "a row that no slot owns was written"
    check_sums(got[written], want[written], mag[written], K, out, bool(act))
    return got


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,scale,out", [(BF, BF, BF), (BF, F32, F32), (HF, HF, HF), (HF, F32, F32)])
def test_groups_zeros_and_types(group, zeros, dtype, scale, out):
    run([1, 0, 3, 20], 144, 768, group, dtype, out, scale, zeros, seed=group)


@pytest.mark.parametrize("N,K,group", [(8, 32, 32), (16, 64, 64), (24, 128, 128), (40, 160, 32), (1000, 192, 64),
                                       (256, 4096, 128), (72, 7168, 64), (2056, 1120, 32)])
@pytest.mark.parametrize("rows", [1, 2, 7])
def test_sizes(N, K, group, rows):
    run([rows, 0, 1], N, K, group, seed=rows)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 33, 64, 65, 130, 300])
def test_row_counts(rows):
    run([rows, 0, 2, rows // 2], 80, 512, 128, HF, F32, seed=rows)


@pytest.mark.parametrize("x_rows,y_rows", [(POS, POS), (TOKEN, POS), (PAIR, POS), (POS, PAIR), (PAIR, PAIR), (TOKEN, PAIR)])
@pytest.mark.parametrize("tokens", [1, 30])
def test_row_modes(x_rows, y_rows, tokens):
    k = 8
    P = tokens * k
    run([P // 3, 0, P // 4, 1], 96, 256, 64, k=k, P=P, x_rows=x_rows, y_rows=y_rows, seed=tokens)


@pytest.mark.parametrize("sizes", [[1, 0, 2], [16], [5, 40]])
@pytest.mark.parametrize("N,K,group", [(16, 64, 32), (48, 192, 64), (1536, 256, 128)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
def test_swiglu(sizes, N, K, group, dtype, out):
    P = sum(sizes)
    offsets, perm = batches(sizes, P, 1, 0)
    x = torch.randn((P, K), generator=torch.Generator().manual_seed(1)).to(dtype)
    q, scales, z = weights(len(sizes), N, K, group, dtype, True, 2)
    scales = (scales.float() * 0.1).to(dtype)
    want, _, mag = product(x, w4_matrix(q, scales, z, group), offsets, P, perm, 1, POS, POS, False, 1,
                           w4_magnitude(q, scales, z, group))
    y = torch.empty((P, N // 2), dtype=out, device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), z.cuda(), group, offsets.cuda(), y, act=Q.MOE_ACT_SWIGLU)
    check_sums(y.cpu(), want, mag, K, out, True)


def test_many_slots_few_rows():
    g = torch.Generator().manual_seed(3)
    run([int(v) for v in (torch.rand(1024, generator=g) < 0.02)], 32, 96, 32, BF, F32, seed=11)


@pytest.mark.parametrize("rows", [1, 9, 50])
def test_dense_without_offsets(rows):
    N, K, group = 328, 384, 128
    x = torch.randn((rows, K), generator=torch.Generator().manual_seed(1)).to(HF)
    q, scales, _ = weights(1, N, K, group, HF, False, 2)
    want, _, mag = product(x, w4_matrix(q, scales, None, group), None, rows, None, 1, POS, POS, False, 0,
                           w4_magnitude(q, scales, None, group))
    y = torch.empty((rows, N), device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), None, group, None, y)
    check_sums(y.cpu(), want, mag, K, F32)


def test_codes_and_scales_are_exact():
    """One-hot rows read single weights: scale (code - zero) must come out as the formula's value rounded once."""
    N, K, group = 32, 256, 32
    q, scales, z = weights(1, N, K, group, F32, True, 5)
    x = torch.eye(K).to(BF)
    y = torch.empty((K, N), device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), z.cuda(), group, None, y)
    want = w4_matrix(q, scales, z, group)[0].t()
    assert ((y.cpu().double() - want).abs() <= 2.0 ** -24 * want.abs()).all()


def test_equal_calls_give_equal_bits():
    a = run([7, 3, 20], 272, 512, 64, BF, F32, seed=1)
    b = run([7, 3, 20], 272, 512, 64, BF, F32, seed=1)
    assert torch.equal(a, b)
