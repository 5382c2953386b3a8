"""moe_expert_gemm and moe_expert_gemm_wgrad against their formulas in 64
bits: types, row modes, ragged and empty slots, odd sizes, rows that no slot
owns, and the gradients against differences."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, batches, check_sums, product, wgrad

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _count(mode, P, k):
    return -(-P // k) if mode == TOKEN else P


def run_product(sizes, N, K, dtype, out, k=1, P=None, x_rows=POS, y_rows=POS, transpose=False, act=0, seed=0, pad=0):
    """One product on the device against the formula; rows of no slot must keep their value."""
    P = sum(sizes) if P is None else P
    offsets, perm = batches(sizes, P, k, seed)
    x = _rand((_count(x_rows, P, k), N if transpose else K), dtype, seed + 1)
    store = _rand((len(sizes), N * K + pad), dtype, seed + 2, K ** -0.5)
    w = store[:, :N * K].unflatten(1, (N, K))
    want, written, mag = product(x, w, offsets, P, perm, k, x_rows, y_rows, transpose, act)
    mark = -77.0
    y = torch.full((P, want.shape[1]), mark, dtype=out, device="cuda")
    Q.moe_expert_gemm(x.cuda(), store.cuda()[:, :N * K].unflatten(1, (N, K)), offsets.cuda(), y, perm.cuda(), k, x_rows,
                      y_rows, transpose, act)
    got = y.cpu()
    assert (got[~written] == mark).all(), "a row that no slot owns was written"
    check_sums(got[written], want[written], mag[written], N if transpose else K, out, bool(act))
    return got


@pytest.mark.parametrize("sizes", [[1], [0, 1, 0], [2, 0, 0, 3, 1], [17, 1, 0, 33], [64, 65, 0, 130, 7], [300, 0, 257, 1]])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_product_of_ragged_slots(sizes, dtype, out):
    run_product(sizes, 272, 200, dtype, out, seed=len(sizes))


@pytest.mark.parametrize("N,K", [(8, 8), (16, 2048), (2048, 8), (136, 72), (264, 520), (1000, 1032)])
@pytest.mark.parametrize("rows", [1, 5, 90, 400])
@pytest.mark.parametrize("transpose", [False, True])
def test_product_odd_sizes(N, K, rows, transpose):
    run_product([rows, 0, rows // 2 + 1], N, K, BF, BF, transpose=transpose, seed=rows)


@pytest.mark.parametrize("x_rows,y_rows", [(POS, POS), (TOKEN, POS), (PAIR, POS), (POS, PAIR), (PAIR, PAIR), (TOKEN, PAIR)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("tokens", [3, 150])
def test_product_row_modes(x_rows, y_rows, transpose, tokens):
    k = 4
    P = tokens * k
    sizes = [P // 3, 0, P // 4, 1]  # some pairs belong to no slot
    run_product(sizes, 192, 264, HF, HF, k=k, P=P, x_rows=x_rows, y_rows=y_rows, transpose=transpose, seed=tokens)


@pytest.mark.parametrize("sizes", [[1, 0, 2], [20, 5], [140, 0, 300]])
@pytest.mark.parametrize("N,K", [(16, 64), (48, 200), (1536, 256), (272, 136)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
def test_product_swiglu(sizes, N, K, dtype, out):
    run_product(sizes, N, K, dtype, out, act=Q.MOE_ACT_SWIGLU, seed=N)


LARGE = [300, 0, 257, 1, 64, 65, 33, 128, 129, 200, 255, 256, 31, 32, 320, 97] * 2  # every count of 32-row blocks


@pytest.mark.parametrize("inner", [8, 64, 72, 128, 136, 192, 200, 256, 264, 328, 392, 584])
@pytest.mark.parametrize("transpose", [False, True])
def test_product_large_tiles(inner, transpose):
    """Enough tiles for the 256 x 256 kernels, every count of contraction stages and rests."""
    N, K = (inner, 2824) if transpose else (2824, inner)
    run_product(LARGE, N, K, BF, BF, transpose=transpose, seed=inner)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("mode", ["forward", "transpose", "swiglu"])
def test_product_large_tiles_types(dtype, out, mode):
    N, K = (328, 2824) if mode == "transpose" else (2832, 328)
    k, P = 2, sum(LARGE) + 100
    run_product(LARGE, N, K, dtype, out, k=k, P=P, x_rows=PAIR if mode == "transpose" else TOKEN,
                y_rows=POS if mode == "swiglu" else PAIR, transpose=mode == "transpose", act=int(mode == "swiglu"), seed=3)


def test_product_larger_weight_stride():
    run_product([3, 40], 72, 80, BF, BF, pad=64, seed=5)
    run_product([200, 140], 72, 80, BF, BF, pad=64, seed=6)


def test_product_many_slots_few_rows():
    g = torch.Generator().manual_seed(3)
    sizes = [int(v) for v in (torch.rand(1024, generator=g) < 0.02)]
    run_product(sizes, 64, 96, BF, F32, seed=11)
    run_product(sizes, 64, 96, BF, F32, transpose=True, seed=12)


@pytest.mark.parametrize("rows", [1, 16, 33, 512])
@pytest.mark.parametrize("transpose", [False, True])
def test_dense_product_without_offsets(rows, transpose):
    N, K = 320, 136
    x, w = _rand((rows, N if transpose else K), BF, 1), _rand((1, N, K), BF, 2, K ** -0.5)
    want, _, mag = product(x, w, None, rows, None, 1, POS, POS, transpose, 0)
    y = torch.empty((rows, want.shape[1]), dtype=F32, device="cuda")
    Q.moe_expert_gemm(x.cuda(), w.cuda(), None, y, transpose=transpose)
    check_sums(y.cpu(), want, mag, N if transpose else K, F32)


def test_no_rows_at_all():
    w = _rand((2, 16, 16), BF, 0).cuda()
    y = torch.full((4, 16), 5.0, dtype=BF, device="cuda")
    x = _rand((4, 16), BF, 1).cuda()
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    Q.moe_expert_gemm(x, w, zero, y)
    assert (y == 5.0).all()
    Q.moe_expert_gemm(x[:0], w, zero, y[:0])
    dw = torch.full((2, 16, 16), 5.0, device="cuda")
    Q.moe_expert_gemm_wgrad(x, x, zero, dw, ws=wgrad_ws(2, 16, 16, 4))
    assert (dw == 0).all()
    dw.fill_(5.0)
    Q.moe_expert_gemm_wgrad(x[:0], x[:0], zero, dw, ws=wgrad_ws(2, 16, 16, 0))
    assert (dw == 0).all()


def test_nan_and_infinity_stay_in_their_rows():
    """A row with NaN or infinity changes its own outputs only, also beside it in a tile."""
    sizes, N, K = [5, 40], 64, 96
    offsets, perm = batches(sizes, 45, 1, 0)
    x, w = _rand((45, K), BF, 1), _rand((2, N, K), BF, 2)
    bad = x.clone()
    bad[2, 7], bad[30, 95], bad[31, 0] = float("nan"), float("inf"), float("nan")
    y0, y1 = (torch.zeros((45, N), dtype=BF, device="cuda") for _ in range(2))
    for v, y in ((x, y0), (bad, y1)):
        Q.moe_expert_gemm(v.cuda(), w.cuda(), offsets.cuda(), y)
    keep = [i for i in range(45) if i not in (2, 30, 31)]
    assert torch.equal(y0[keep], y1[keep])
    assert y1[[2, 31]].isnan().all() and not y1[30].isfinite().any()


def wgrad_ws(S, N, K, R):
    return torch.empty(max(1, Q.moe_expert_gemm_wgrad_workspace_size(S, N, K, R)), dtype=torch.uint8, device="cuda")


def run_wgrad(sizes, N, K, dtype, out, k=1, P=None, dy_rows=POS, x_rows=POS, seed=0):
    P = sum(sizes) if P is None else P
    offsets, perm = batches(sizes, P, k, seed)
    dy, x = _rand((_count(dy_rows, P, k), N), dtype, seed + 1), _rand((_count(x_rows, P, k), K), dtype, seed + 2)
    want, mag = wgrad(dy, x, offsets, len(sizes), P, perm, k, dy_rows, x_rows)
    dw = torch.full((len(sizes), N, K), float("nan"), dtype=out, device="cuda")
    Q.moe_expert_gemm_wgrad(dy.cuda(), x.cuda(), offsets.cuda(), dw, perm.cuda(), k, dy_rows, x_rows,
                            wgrad_ws(len(sizes), N, K, P))
    check_sums(dw.cpu(), want, mag, max(sizes + [1]), out)
    return dw


@pytest.mark.parametrize("sizes", [[1], [0, 1, 0], [2, 0, 0, 3, 1], [31, 32, 33, 0], [63, 64, 65, 130], [300, 0, 1000, 1]])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_weight_gradient_of_ragged_slots(sizes, dtype, out):
    run_wgrad(sizes, 136, 200, dtype, out, seed=len(sizes))


@pytest.mark.parametrize("N,K", [(8, 8), (16, 1032), (1000, 8), (264, 520)])
@pytest.mark.parametrize("rows", [1, 70, 2049])
def test_weight_gradient_odd_sizes(N, K, rows):
    run_wgrad([rows, 0, rows // 3 + 1], N, K, BF, F32, seed=rows)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (HF, HF)])
@pytest.mark.parametrize("dy_rows,x_rows", [(POS, POS), (PAIR, TOKEN)])
def test_weight_gradient_large_tiles(dtype, out, dy_rows, x_rows):
    """Enough tiles for the 256 x 256 kernels, every count of row stages, slots beyond the window of source rows."""
    sizes = [0, 1, 63, 64, 65, 128, 129, 192, 193, 256, 257, 320, 321, 1100, 2500, 1024, 1025]
    run_wgrad(sizes, 1032, 1048, dtype, out, k=2, P=sum(sizes) + 64, dy_rows=dy_rows, x_rows=x_rows, seed=2)


@pytest.mark.parametrize("dy_rows", [POS, PAIR, TOKEN])
@pytest.mark.parametrize("x_rows", [POS, PAIR, TOKEN])
def test_weight_gradient_row_modes(dy_rows, x_rows):
    k = 4
    P = 75 * k
    run_wgrad([P // 3, 0, P // 4, 1], 72, 136, HF, F32, k=k, P=P, dy_rows=dy_rows, x_rows=x_rows, seed=4)


def test_weight_gradient_one_dense_matrix():
    """One matrix and many rows: the rows are split between workgroups."""
    run_wgrad([5000], 128, 256, BF, F32, seed=8)
    N, K, R = 64, 48, 777
    dy, x = _rand((R, N), BF, 1), _rand((R, K), BF, 2)
    want, mag = wgrad(dy, x, None, 1, R, None, 1, POS, POS)
    dw = torch.empty((1, N, K), device="cuda")
    Q.moe_expert_gemm_wgrad(dy.cuda(), x.cuda(), None, dw, ws=wgrad_ws(1, N, K, R))
    check_sums(dw.cpu(), want, mag, R, F32)


def test_equal_calls_give_equal_bits():
    a = run_product([70, 3, 200], 272, 520, BF, F32, seed=1)
    b = run_product([70, 3, 200], 272, 520, BF, F32, seed=1)
    assert torch.equal(a, b)
    a = run_wgrad([900, 3, 200], 136, 264, BF, F32, seed=1)
    b = run_wgrad([900, 3, 200], 136, 264, BF, F32, seed=1)
    assert torch.equal(a, b)


def test_gradients_against_differences():
    """The loss sum(c * y) moves by the gradients' prediction: in x through
    the transposed product, in w through the weight gradient.  The product is
    linear in each, so a step of any size has no curvature error; powers of
    two keep every input and step exact in bf16, and fp32 sums of 48 terms
    leave 2 * 48 * 2^-24 of the absolute sum on each side."""
    sizes, N, K = [3, 9], 16, 48
    offsets, perm = batches(sizes, 12, 1, 0)
    g = torch.Generator().manual_seed(9)

    def pow2(shape):
        return (2.0 ** torch.randint(-2, 3, shape, generator=g)) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)

    x, w, c, dx, dw = (pow2(s).to(BF) for s in ((12, K), (2, N, K), (12, N), (12, K), (2, N, K)))
    off = offsets.cuda()

    def loss(xv, wv):
        y = torch.zeros((12, N), device="cuda")
        Q.moe_expert_gemm(xv.to(BF).cuda(), wv.to(BF).cuda(), off, y)
        return (y.cpu().to(D) * c.to(D)).sum()

    gx = torch.zeros((12, K), device="cuda")
    Q.moe_expert_gemm(c.cuda(), w.cuda(), off, gx, transpose=True)
    gw = torch.zeros((2, N, K), device="cuda")
    Q.moe_expert_gemm_wgrad(c.cuda(), x.cuda(), off, gw, ws=wgrad_ws(2, N, K, 12))
    size = 4.0 ** 3 * 12 * N * K * 2  # bound of the sums of absolute terms
    tol = 4 * 48 * 2.0 ** -24 * size
    # the directions are single coordinates, so x + step stays exact
    for i, j in ((0, 0), (5, 47), (11, 20)):
        step = torch.zeros((12, K))
        step[i, j] = x[i, j].float()  # doubles one element
        assert abs(float(loss(x.float() + step, w.float()) - loss(x.float(), w.float())) - float((gx.cpu() * step).sum())) <= tol
    for s, i, j in ((0, 0, 0), (1, 15, 47), (1, 3, 9)):
        step = torch.zeros((2, N, K))
        step[s, i, j] = w[s, i, j].float()
        assert abs(float(loss(x.float(), w.float() + step) - loss(x.float(), w.float())) - float((gw.cpu() * step).sum())) <= tol
