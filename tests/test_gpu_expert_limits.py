"""The expert products, block norms and SwiGLU over tensors of more than 4 GB
and 2^31 elements, and values at the ends of their ranges."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import batches, check_sums, product, w4_magnitude, w4_matrix, wgrad

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
POS = Q.MOE_ROWS_POSITION
TAIL = 300  # rows with values, behind the rows of zeros


def rand(shape, seed, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def long(rows, tail):
    t = torch.zeros((rows, tail.shape[1]), dtype=tail.dtype, device="cuda")
    t[-len(tail):] = tail.cuda()
    return t


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("N,K", [(32, 2048), (2048, 32)])
def test_product_rows_behind_4_gb(N, K, transpose):
    R = 1_150_000  # x (2048 wide) or y (2048 wide, fp32) is larger than 4 GB
    x, w = rand((TAIL, N if transpose else K), 1), rand((1, N, K), 2)
    want, _, mag = product(x, w, None, TAIL, None, 1, POS, POS, transpose, 0)
    y = torch.full((R, want.shape[1]), 7.0, device="cuda")
    Q.moe_expert_gemm(long(R, x), w.cuda(), None, y, transpose=transpose)
    assert (y[:-TAIL] == 0).all()
    check_sums(y[-TAIL:].cpu(), want, mag, N if transpose else K, F32)


def test_weight_gradient_rows_behind_4_gb():
    R, N, K = 1_150_000, 32, 2048
    dy, x = rand((TAIL, N), 1), rand((TAIL, K), 2)
    want, mag = wgrad(dy, x, None, 1, TAIL, None, 1, POS, POS)
    dw = torch.empty((1, N, K), device="cuda")
    ws = torch.empty(max(1, Q.moe_expert_gemm_wgrad_workspace_size(1, N, K, R)), dtype=torch.uint8, device="cuda")
    Q.moe_expert_gemm_wgrad(long(R, dy), long(R, x), None, dw, ws=ws)
    check_sums(dw.cpu(), want, mag, TAIL, F32)


@pytest.mark.parametrize("rows,transpose", [(2, False), (200, False), (200, True)])
def test_matrices_behind_4_gb(rows, transpose):
    S, N, K, stride = 3, 72, 512, 1_150_000_000  # elements from matrix to matrix: 2.3 GB
    w, x = rand((S, N, K), 1), rand((S * rows, N if transpose else K), 2)
    pool = torch.zeros(2 * stride + N * K, dtype=BF, device="cuda")
    apart = pool.as_strided((S, N, K), (stride, K, 1))
    apart.copy_(w)
    offsets = torch.arange(S + 1, dtype=torch.int32) * rows
    want, _, mag = product(x, w, offsets, S * rows, None, 1, POS, POS, transpose, 0)
    y = torch.empty((S * rows, want.shape[1]), device="cuda")
    Q.moe_expert_gemm(x.cuda(), apart, offsets.cuda(), y, transpose=transpose)
    check_sums(y.cpu(), want, mag, N if transpose else K, F32)


def test_4_bit_rows_behind_4_gb():
    R, N, K, group = 1_150_000, 32, 2048, 128
    x, q = rand((TAIL, K), 1), torch.randint(0, 256, (1, N, K // 2), generator=torch.Generator().manual_seed(2), dtype=torch.uint8)
    scales = rand((1, N, K // group), 3).abs()
    want, _, mag = product(x, w4_matrix(q, scales, None, group), None, TAIL, None, 1, POS, POS, False, 0,
                           w4_magnitude(q, scales, None, group))
    y = torch.full((R, N), 7.0, device="cuda")
    Q.moe_expert_gemv_w4(long(R, x), q.cuda(), scales.cuda(), None, group, None, y)
    assert (y[:-TAIL] == 0).all()
    check_sums(y[-TAIL:].cpu(), want, mag, K, F32)


@pytest.mark.parametrize("group", [32, 128])
def test_4_bit_zeros_of_a_whole_byte(group):
    """zeros are bytes: 0 and 16..255 too, far from the codes."""
    sizes, N, K = [3, 20], 48, 256
    offsets, _ = batches(sizes, 23, 1, 0)
    g = torch.Generator().manual_seed(4)
    x, q = rand((23, K), 1), torch.randint(0, 256, (2, N, K // 2), generator=g, dtype=torch.uint8)
    scales, zeros = rand((2, N, K // group), 3), torch.randint(0, 256, (2, N, K // group), generator=g, dtype=torch.uint8)
    zeros.view(-1)[:4] = torch.tensor([0, 255, 16, 128], dtype=torch.uint8)
    # scales of both signs: w4_magnitude is scale (code + zero), what the terms amount to is its absolute value
    want, _, mag = product(x, w4_matrix(q, scales, zeros, group), offsets, 23, None, 1, POS, POS, False, 0,
                           w4_magnitude(q, scales, zeros, group).abs())
    y = torch.empty((23, N), device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), zeros.cuda(), group, offsets.cuda(), y)
    check_sums(y.cpu(), want, mag, K, F32)


@pytest.mark.parametrize("K,group", [(4128, 32), (8256, 64), (16512, 128)])
@pytest.mark.parametrize("rows", [2, 12, 28, 70])
def test_4_bit_rows_of_many_groups(K, group, rows):
    """More groups than a workgroup holds at a time (64), and a short rest; all counts of rows a pass."""
    N = 40
    x, q = rand((rows, K), 1), torch.randint(0, 256, (1, N, K // 2), generator=torch.Generator().manual_seed(2), dtype=torch.uint8)
    scales = rand((1, N, K // group), 3).abs()
    zeros = torch.randint(0, 16, (1, N, K // group), generator=torch.Generator().manual_seed(4), dtype=torch.uint8)
    want, _, mag = product(x, w4_matrix(q, scales, zeros, group), None, rows, None, 1, POS, POS, False, 0,
                           w4_magnitude(q, scales, zeros, group))
    y = torch.empty((rows, N), device="cuda")
    Q.moe_expert_gemv_w4(x.cuda(), q.cuda(), scales.cuda(), zeros.cuda(), group, None, y)
    check_sums(y.cpu(), want, mag, K, F32)


@pytest.mark.parametrize("k", [1, 3, 7, 64])
def test_token_rows_at_the_end_of_the_range(k):
    """Pairs up to 2^24 - 1 find their token (pair / k) exactly."""
    R, N, K = 1 << 24, 8, 8
    tokens = -(-R // k)
    x = torch.arange(tokens, device="cuda").remainder(251).to(BF).unsqueeze(1).repeat(1, K)
    w = torch.eye(8, dtype=BF).unsqueeze(0).cuda()
    perm = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = torch.empty((R, N), dtype=BF, device="cuda")
    Q.moe_expert_gemm(x, w, None, y, perm, k, Q.MOE_ROWS_TOKEN, POS)
    assert torch.equal(y, x[(perm.long() // k)])


@pytest.mark.parametrize("rows", [7, 45])
def test_4_bit_nan_and_infinity_stay_in_their_rows(rows):
    """A row with an infinity or a NaN gives no finite value; the rows beside it do not change."""
    N, K, group = 64, 320, 64
    x, q = rand((rows, K), 1), torch.randint(0, 256, (1, N, K // 2), generator=torch.Generator().manual_seed(2), dtype=torch.uint8)
    scales = rand((1, N, K // group), 3).abs() + 0.5
    bad = x.clone()
    bad[2, 7], bad[5, K - 1] = float("nan"), float("inf")
    y0, y1 = (torch.zeros((rows, N), dtype=BF, device="cuda") for _ in range(2))
    for v, y in ((x, y0), (bad, y1)):
        Q.moe_expert_gemv_w4(v.cuda(), q.cuda(), scales.cuda(), None, group, None, y)
    keep = [i for i in range(rows) if i not in (2, 5)]
    assert torch.equal(y0[keep], y1[keep])
    assert not y1[[2, 5]].isfinite().any()


def test_block_norm_rows_behind_4_gb():
    T, H = 270_000, 8192  # 2^31 elements and more
    x, y, dxo, dh = (rand((TAIL, H), s) for s in range(4))
    w = rand((H,), 5, F32).cuda()
    a = [t.cuda() for t in (x, y, dxo, dh)]
    small = [torch.empty_like(a[0]) for _ in range(4)]
    grads = [torch.empty(H, device="cuda") for _ in range(3)]

    def both(x, y, dxo, dh, x_out, h, dx, dy):
        Q.moe_block_norm(x, y, w, w, w, x_out, h, 1e-6, 0.5)
        ws = torch.empty(Q.moe_block_norm_backward_workspace_size(*x.shape), dtype=torch.uint8, device="cuda")
        Q.moe_block_norm_backward(x, y, w, w, w, dxo, dh, dx, dy, *grads, 1e-6, 0.5, ws)

    both(*a, *small)
    large = [long(T, t) for t in (x, y, dxo, dh)]
    out = [torch.empty_like(large[0]) for _ in range(4)]
    both(*large, *out)
    for got, want in zip(out, small):
        assert torch.equal(got[-TAIL:], want)
        assert (got[:-TAIL] == 0).all()


def test_swiglu_rows_behind_4_gb():
    R, I = 270_000, 4096
    gu, dh = rand((TAIL, 2 * I), 1), rand((TAIL, I), 2)
    h, d = torch.empty((TAIL, I), dtype=BF, device="cuda"), torch.empty((TAIL, 2 * I), dtype=BF, device="cuda")
    Q.moe_swiglu(gu.cuda(), h)
    Q.moe_swiglu_backward(gu.cuda(), dh.cuda(), d)
    lgu, ldh = long(R, gu), long(R, dh)
    lh = torch.empty((R, I), dtype=BF, device="cuda")
    Q.moe_swiglu(lgu, lh)
    assert torch.equal(lh[-TAIL:], h) and (lh[:-TAIL] == 0).all()
    Q.moe_swiglu_backward(lgu, ldh, lgu)  # in place
    assert torch.equal(lgu[-TAIL:], d) and (lgu[:-TAIL] == 0).all()
