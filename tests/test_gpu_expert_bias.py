"""moe_expert_gemm_bias and moe_expert_act_backward against their formulas in 64 bits: activations, types, row modes,
ragged and empty slots, both kinds of product kernels, in-place forms, and the gradients against differences."""
import math

import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, batches, rows_of
from tests.train_util import ACTS, F, act, act_grad, bias_product, rand, store_bound, sum_terms, within

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SWI = Q.MOE_ACT_SWIGLU
MARK = -77.0


def run_product(sizes, N, K, dtype, out, kind, bias=F32, res=None, keep=True, k=1, P=None, x_rows=POS, y_rows=POS, seed=0,
                inplace=False, dense=False):
    P = sum(sizes) if P is None else P
    offsets, perm = batches(sizes, P, k, seed)
    S = len(sizes)
    if dense:
        offsets = None
    width = N // 2 if kind == SWI else N
    x = rand((-(-P // k) if x_rows == TOKEN else P, K), dtype, seed + 1)
    w = rand((S, N, K), dtype, seed + 2, K ** -0.5)
    b = None if bias is None else rand((S, N), bias, seed + 3)
    r = None if res is None else rand((P, width), res, seed + 4)
    y, z, written, by, bz = bias_product(x, w, b, r, offsets, P, perm, k, x_rows, y_rows, kind, out)
    dev = lambda t: None if t is None else t.cuda()
    rd = dev(r)
    got = rd if inplace else torch.full((P, width), MARK, dtype=out, device="cuda")
    gz = torch.full((P, N), MARK, dtype=dtype, device="cuda") if keep else None
    Q.moe_expert_gemm_bias(x.cuda(), w.cuda(), dev(b), rd, dev(offsets), got, perm.cuda(), k, x_rows, y_rows, kind, z=gz)
    got = got.cpu()
    if not inplace:
        assert (got[~written] == MARK).all(), "a row of y that no slot owns was written"
    within(got[written], y[written], by[written] + store_bound(y[written], out), "y")
    if keep:
        gz = gz.cpu()
        assert (gz[~written] == MARK).all(), "a row of z that no slot owns was written"
        within(gz[written], z[written], bz[written] + store_bound(z[written], dtype), "z")


FEW, RAGGED = [2, 0, 3, 1], [64, 65, 0, 130, 7, 300]
LARGE = [300, 0, 257, 1, 64, 65, 33, 128, 129, 200, 255, 256, 31, 32, 320, 97] * 2


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("sizes", [FEW, RAGGED])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_activations_and_types(kind, sizes, dtype, out):
    run_product(sizes, 272, 200, dtype, out, kind, bias=F32, res=out, seed=kind)


@pytest.mark.parametrize("bias", [None, BF, F32])
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("kind", [Q.MOE_ACT_NONE, SWI, Q.MOE_ACT_GELU])
@pytest.mark.parametrize("sizes,keep", [(FEW, True), (FEW, False), (RAGGED, True), (RAGGED, False)])
def test_optional_operands(bias, res, kind, sizes, keep):
    run_product(sizes, 144, 136, BF, BF, kind, bias=bias, res=res, keep=keep, seed=3)


@pytest.mark.parametrize("N,K", [(16, 8), (16, 2048), (2048, 8), (144, 72), (528, 520), (1008, 1032)])
@pytest.mark.parametrize("rows", [1, 5, 90, 400])
@pytest.mark.parametrize("kind", [SWI, Q.MOE_ACT_GELU_TANH])
def test_odd_sizes(N, K, rows, kind):
    run_product([rows, 0, rows // 2 + 1], N, K, BF, BF, kind, res=F32, seed=rows)


@pytest.mark.parametrize("x_rows,y_rows", [(POS, POS), (TOKEN, POS), (PAIR, POS), (POS, PAIR), (PAIR, PAIR), (TOKEN, PAIR)])
@pytest.mark.parametrize("tokens", [3, 150])
@pytest.mark.parametrize("kind", [SWI, Q.MOE_ACT_SILU])
def test_row_modes(x_rows, y_rows, tokens, kind):
    P = tokens * 4
    run_product([P // 3, 0, P // 4, 1], 192, 264, HF, HF, kind, res=HF, k=4, P=P, x_rows=x_rows, y_rows=y_rows, seed=tokens)


@pytest.mark.parametrize("inner", [8, 72, 256, 584])
@pytest.mark.parametrize("kind", ACTS)
def test_large_tiles(inner, kind):
    """Enough tiles for the 256 x 256 kernels."""
    run_product(LARGE, 2832, inner, BF, BF, kind, res=BF, P=sum(LARGE) + 100, k=2, x_rows=TOKEN, y_rows=PAIR, seed=inner)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("kind", [Q.MOE_ACT_NONE, SWI])
def test_large_tiles_types(dtype, out, kind):
    run_product(LARGE, 2832, 328, dtype, out, kind, bias=dtype, res=out, keep=kind == SWI, seed=5)


@pytest.mark.parametrize("rows", [1, 16, 33, 512, 1001])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("kind", [Q.MOE_ACT_NONE, SWI])
def test_dense_adds_to_its_residual(rows, out, kind):
    run_product([rows], 320, 136, BF, out, kind, res=out, inplace=True, dense=True, seed=rows)


def test_many_slots_few_rows():
    g = torch.Generator().manual_seed(3)
    run_product([int(v) for v in (torch.rand(1024, generator=g) < 0.02)], 64, 96, BF, F32, SWI, seed=11)


def test_without_epilogue_equals_the_plain_product():
    """No bias, no residual, no activation: the sums are moe_expert_gemm's, bit for bit."""
    for sizes in (FEW, RAGGED):
        offsets, _ = batches(sizes, sum(sizes), 1, 0)
        x, w, off = rand((sum(sizes), 200), BF, 1).cuda(), rand((len(sizes), 272, 200), BF, 2, 0.07).cuda(), offsets.cuda()
        for kind in (Q.MOE_ACT_NONE, SWI):
            a = torch.zeros((sum(sizes), 136 if kind else 272), dtype=F32, device="cuda")
            b = torch.zeros_like(a)
            Q.moe_expert_gemm(x, w, off, a, act=kind)
            Q.moe_expert_gemm_bias(x, w, None, None, off, b, act=kind)
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ACTS)
def test_infinite_and_nan_sums(kind):
    """Values far outside: an activation of +-inf and NaN sums is the formula's."""
    x = torch.zeros((6, 16), dtype=BF)
    x[:, 0] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1.0])
    w = torch.zeros((1, 32, 16), dtype=BF)
    w[:, :, 0] = 1
    z = x[:, :1].to(D).expand(6, 32).contiguous()
    want = act(z.float(), kind).to(D)  # overflows where fp32 does
    y = torch.empty((6, want.shape[1]), dtype=F32, device="cuda")
    Q.moe_expert_gemm_bias(x.cuda(), w.cuda(), None, None, None, y, act=kind)
    got = y.cpu().to(D)
    finite = torch.isfinite(want) & torch.isfinite(z[:, :want.shape[1]])
    assert torch.isnan(got[2]).all()
    assert torch.allclose(got[finite], want[finite], rtol=1e-6)
    assert (got[0] == float("inf")).all()


def test_more_than_4_gb_of_rows():
    """Rows and sums behind 2^32 bytes, through both product kernels and the gradient."""
    R, N, K = (1 << 20) + 77, 2816, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((R, K), generator=g, device="cuda", dtype=BF)
    w, b = rand((1, N, K), BF, 2, 0.25).cuda(), rand((1, N), F32, 3).cuda()
    y = torch.empty((R, N // 2), dtype=BF, device="cuda")
    z = torch.empty((R, N), dtype=BF, device="cuda")
    Q.moe_expert_gemm_bias(x, w, b, None, None, y, act=SWI, z=z)
    for rows in (slice(0, 100), slice(R - 200, R)):
        v = x[rows].double() @ w[0].double().t() + b[0].double()
        within(z[rows], v.cpu(), 40 * F * (1 + v.abs().cpu()) + store_bound(v.cpu(), BF), "z")
        o = act(v, SWI).cpu()
        within(y[rows], o, 40 * F * (1 + v.abs().cpu()).max() ** 2 + store_bound(o, BF), "y")
    last = torch.full((R,), R - 1, dtype=torch.int32, device="cuda")  # few rows, the last ones of the buffers
    last[:3] = torch.tensor([R - 1, R - 2, 5], dtype=torch.int32)
    off = torch.tensor([0] + [3] * 600, dtype=torch.int32, device="cuda")
    few_w = w.expand(600, N, K)
    y2 = torch.empty_like(y)
    Q.moe_expert_gemm_bias(x, few_w.contiguous(), None, y, off, y2, last, 1, PAIR, PAIR, SWI)
    for r in (R - 1, R - 2, 5):
        o = act(x[r:r + 1].double() @ w[0].double().t(), SWI) + y[r:r + 1].double()
        within(y2[r:r + 1], o.cpu(), 40 * F * (1 + o.abs().cpu()) * 8 + store_bound(o.cpu(), BF), "row")
    del y2, few_w
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(1, N, R), dtype=torch.uint8, device="cuda")
    db = torch.empty((1, N), device="cuda")
    end = z[R - 50:].clone()
    Q.moe_expert_act_backward(y, z, None, z, db, act=SWI, ws=ws)
    want = act_grad(end.cpu().to(D), y[R - 50:].cpu().to(D), SWI)
    within(z[R - 50:], want, 16 * F * (1 + end.cpu().to(D).abs().max()) ** 3 + store_bound(want, BF), "dz")
    # the stored dz has one rounding to bf16 each; their sum is the fp32 sum's up to those
    total, size = z.double().sum(0), z.double().abs().sum(0)
    assert ((db[0] - total).abs() <= (2.0 ** -8 + sum_terms(R)) * size).all()


# --------------------------------------------------------------- gradients

def run_grad(sizes, N, dtype, kind, rows=POS, k=1, P=None, h=True, bias=True, seed=0, inplace=None, dense=False, scale=1.5):
    P = sum(sizes) if P is None else P
    S = len(sizes)
    offsets, perm = batches(sizes, P, k, seed)
    I = N // 2 if kind == SWI else N
    none = kind == Q.MOE_ACT_NONE
    z, dy = rand((P, N), dtype, seed + 1, scale), rand((P, I), dtype, seed + 2)
    dzw, hw = torch.full((P, N), MARK, dtype=D), torch.full((P, I), MARK, dtype=D)
    bdz, bh = torch.zeros((P, N), dtype=D), torch.zeros((P, I), dtype=D)
    db, bdb = torch.zeros((S, N), dtype=D), torch.zeros((S, N), dtype=D)
    written = torch.zeros(P, dtype=torch.bool)
    for s in range(S):
        a, b = (0, P) if dense else (int(offsets[s]), int(offsets[s + 1]))
        i = rows_of(rows, perm, k, a, b)
        zs, ds = z[i].to(D), dy[i].to(D)
        v, o = act_grad(zs, ds, kind), act(zs, kind)
        # the derivative is below 1.2 in magnitude, off by a few roundings of 1 (SwiGLU: of u and g too)
        if kind == SWI:
            g, u = zs.chunk(2, 1)
            e = torch.cat((16 * F * (ds * u).abs(), 8 * F * (ds * g).abs()), 1)
            eh = 8 * F * o.abs()
        elif none or kind == Q.MOE_ACT_RELU:
            e, eh = torch.zeros_like(v), torch.zeros_like(o)
        else:
            e, eh = 16 * F * ds.abs(), 8 * F * zs.abs()
        dzw[i], hw[i], bdz[i], bh[i] = v, o, e, eh
        if b > a:
            db[s] = v.sum(0)
            bdb[s] = e.sum(0) + sum_terms(b - a) * v.abs().sum(0)
        written[i] = True
    zd, dyd = z.cuda(), dy.cuda()
    dz = None if none else zd if inplace == "z" else dyd if inplace == "dy" else torch.full((P, N), MARK, dtype=dtype, device="cuda")
    hd = torch.full((P, I), MARK, dtype=dtype, device="cuda") if h and not none else None
    dbd = torch.full((S, N), MARK, dtype=F32, device="cuda") if bias or none else None
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(S, N, P), dtype=torch.uint8, device="cuda")
    Q.moe_expert_act_backward(dyd, None if none else zd, None if dense else offsets.cuda(), dz, dbd, perm.cuda(), rows, kind,
                              h=hd, ws=ws)
    if not none:
        got = dz.cpu()
        if inplace is None:
            assert (got[~written] == MARK).all()
        within(got[written], dzw[written], (bdz + store_bound(dzw, dtype))[written], "dz")
    if hd is not None:
        got = hd.cpu()
        assert (got[~written] == MARK).all()
        within(got[written], hw[written], (bh + store_bound(hw, dtype))[written], "h")
    if dbd is not None:
        within(dbd.cpu(), db, bdb + F * db.abs(), "dbias")


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("sizes", [[1], [0, 1, 0], FEW, RAGGED, [0, 0]])
def test_gradients(kind, dtype, sizes):
    run_grad(sizes, 272, dtype, kind, seed=len(sizes), P=sum(sizes) + 3)


@pytest.mark.parametrize("N", [16, 48, 144, 512, 528, 2064])
@pytest.mark.parametrize("rows", [1, 15, 17, 700])
@pytest.mark.parametrize("kind", [Q.MOE_ACT_NONE, SWI, Q.MOE_ACT_GELU])
def test_gradient_sizes(N, rows, kind):
    run_grad([rows, 0, 3], N, BF, kind, seed=N)
    run_grad([rows], N, HF, kind, seed=N, dense=True)


@pytest.mark.parametrize("kind", [SWI, Q.MOE_ACT_GELU_TANH])
@pytest.mark.parametrize("h,bias", [(True, False), (False, True), (False, False)])
def test_gradient_optional_outputs(kind, h, bias):
    run_grad(RAGGED, 160, BF, kind, h=h, bias=bias, rows=PAIR, k=4, P=sum(RAGGED) + 6)


@pytest.mark.parametrize("kind,inplace", [(SWI, "z"), (Q.MOE_ACT_SILU, "z"), (Q.MOE_ACT_GELU, "dy"), (Q.MOE_ACT_RELU, "dy")])
def test_gradient_in_place(kind, inplace):
    run_grad(RAGGED, 160, BF, kind, inplace=inplace)


def test_gradient_of_many_rows_and_slots():
    g = torch.Generator().manual_seed(5)
    run_grad([int(v) for v in torch.randint(0, 60, (1024,), generator=g)], 32, BF, SWI, seed=9)
    run_grad([40000, 0, 5], 256, BF, SWI, seed=10, h=False)


@pytest.mark.parametrize("N", [8, 16, 24, 40, 64, 128, 136, 256, 264])
@pytest.mark.parametrize("rows", [3, 600, 5000, 40000])
def test_bias_gradient_of_narrow_rows(N, rows):
    run_grad([rows], N, BF, Q.MOE_ACT_NONE, seed=N, dense=True)
    run_grad([rows, 0, 7], N, F32, Q.MOE_ACT_RELU, seed=N, rows=PAIR, P=rows + 9, h=False)


@pytest.mark.parametrize("kind", ACTS[1:])
def test_gradient_far_out(kind):
    """Activations of values from 2^-100 to 2^100, both signs."""
    e = torch.arange(-100, 101, dtype=D)
    z = torch.cat((2.0 ** e, -(2.0 ** e), torch.linspace(-30, 30, 622, dtype=D))).float()
    n = z.numel() // 8 * 8
    z = z[:n].reshape(-1, 8)
    zz = torch.cat((z, torch.ones_like(z)), 1) if kind == SWI else z
    dy = torch.ones_like(z)
    dz, h = torch.empty_like(zz, device="cuda"), torch.empty_like(z, device="cuda")
    Q.moe_expert_act_backward(dy.cuda(), zz.cuda(), None, dz, None, act=kind, h=h)
    zd, wd = zz.to(D), act_grad(zz.to(D), dy.to(D), kind)
    own = 16 * F * (1 + (zd[:, :8].abs() if kind == SWI else 0 * zd))
    bound = torch.cat((16 * F + 0 * own, own), 1) if kind == SWI else own
    within(dz, wd, bound, "dz")
    within(h, act(zd, kind), 8 * F * zd[:, :8].abs(), "h")

INF = math.inf


def limits(kind, z, d):
    """act and d act' at infinite z as their limits (SwiGLU: z = (g, u)): a factor of 0 stays 0.  A sigmoid below fp32's
    range (of less than -104) is one."""
    times = lambda a, v: 0.0 if a == 0 and math.isinf(v) else a * v
    if kind == SWI:
        g, u = z
        s = 0.0 if g < -104 else 1.0 if g == INF else 1 / (1 + math.exp(-g))
        gs = 0.0 if g == -INF else g * s
        slope = s if math.isinf(g) else s * (1 + g * (1 - s))
        h = times(u, gs) if math.isinf(gs) else times(gs, u)
        return h, (times(d * slope, u), times(d, gs))
    return (INF, (d,)) if z > 0 else (0.0, (0.0 * d,))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("kind", ACTS[1:])
def test_gradient_of_infinite_sums(kind, dtype):
    """z beyond its type's range is stored as infinite: gradients are the limits there, not NaN; NaN stays NaN."""
    if kind == SWI:
        cases = [(g, u, d) for g in (INF, -INF, 0.0, 1.5, -2.0, -200.0) for u in (INF, -INF, 0.0, 2.0, -3.0)
                 for d in (0.0, 1.0, -0.5) if math.isinf(g) or math.isinf(u)]
    else:
        cases = [(z, d) for z in (INF, -INF) for d in (0.0, 1.0, -0.5)]
    n = -(-len(cases) // 8) * 8
    cases = (cases * 8)[:n]
    want = [limits(kind, c[:2] if kind == SWI else c[0], c[-1]) for c in cases]
    z = torch.tensor([c[0] for c in cases] + ([c[1] for c in cases] if kind == SWI else []), dtype=dtype)[None]
    dy = torch.tensor([c[-1] for c in cases], dtype=dtype)[None]
    dz, h = torch.empty_like(z, device="cuda"), torch.empty_like(dy, device="cuda")
    db = torch.empty((1, z.shape[1]), device="cuda")
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(1, z.shape[1], 1), dtype=torch.uint8, device="cuda")
    Q.moe_expert_act_backward(dy.cuda(), z.cuda(), None, dz, db, act=kind, h=h, ws=ws)
    wd = torch.tensor([w[1][i] for i in range(2 if kind == SWI else 1) for w in want], dtype=D)[None]
    wh = torch.tensor([w[0] for w in want], dtype=D)[None]
    # finite ones: the sigmoid's and four products' roundings of values below 10
    within(dz, wd, 100 * F + store_bound(wd.nan_to_num(posinf=0, neginf=0), dtype), "dz")
    within(db, wd, torch.full_like(wd, 100 * F), "dbias")
    within(h, wh, 100 * F + store_bound(wh.nan_to_num(posinf=0, neginf=0), dtype), "h")
    z = torch.full_like(z, math.nan)
    Q.moe_expert_act_backward(dy.cuda(), z.cuda(), None, dz, None, act=kind, h=h)
    if kind != Q.MOE_ACT_RELU:
        assert torch.isnan(dz).all()
    assert torch.isnan(h).all()


@pytest.mark.parametrize("kind", ACTS[1:])
def test_gradient_where_fp16_sums_overflow(kind):
    """The product's own fp16 z is infinite where the sums pass 65504; y in fp32 is finite, and so is what the gradient
    makes of it where it has a limit.  The elements beside the infinite ones keep their bits."""
    N, K, R = 32, 16, 24
    x, w = torch.full((R, K), 200.0, dtype=HF), rand((1, N, K), HF, 1)
    w[:, 3], w[:, 7], w[:, 20] = 30.0, -30.0, 25.0  # sums of +-96000 and 80000
    I = N // 2 if kind == SWI else N
    y, z = torch.empty((R, I), device="cuda"), torch.empty((R, N), dtype=HF, device="cuda")
    Q.moe_expert_gemm_bias(x.cuda(), w.cuda(), None, None, None, y, act=kind, z=z)
    assert torch.isfinite(y).all() and (z[:, 3] == INF).all() and (z[:, 7] == -INF).all() and (z[:, 20] == INF).all()
    dy = rand((R, I), HF, 2).abs()  # of one sign: so are the infinite terms of a bias's gradient
    dy[::3] = 0
    dz, h, db = torch.empty_like(z), torch.empty((R, I), dtype=HF, device="cuda"), torch.empty((1, N), device="cuda")
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(1, N, R), dtype=torch.uint8, device="cuda")
    Q.moe_expert_act_backward(dy.cuda(), z, None, dz, db, act=kind, h=h, ws=ws)
    assert not torch.isnan(dz).any() and not torch.isnan(h).any() and not torch.isnan(db).any()
    assert (dz[::3] == 0).all()
    others = z.clone()
    others[torch.isinf(z)] = 1.0
    dz2, h2 = torch.empty_like(z), torch.empty_like(h)
    Q.moe_expert_act_backward(dy.cuda(), others, None, dz2, None, act=kind, h=h2)
    far = torch.isinf(z)
    if kind == SWI:
        far = (far[:, :I] | far[:, I:]).repeat(1, 2)
    assert torch.equal(dz[~far], dz2[~far]) and torch.equal(h[~far[:, :I]], h2[~far[:, :I]])


@pytest.mark.parametrize("kind", ACTS[1:])
def test_gradient_against_differences(kind):
    """dz . v against the 64-bit activation's central difference along v, and the bias gradient the same way."""
    sizes, N = [9, 0, 23], 48
    offsets, perm = batches(sizes, 32, 1, 1)
    I = N // 2 if kind == SWI else N
    z, dy, v = rand((32, N), F32, 1), rand((32, I), F32, 2), rand((32, N), F32, 3)
    if kind == Q.MOE_ACT_RELU:
        z = z + 0.01 * z.sign()  # no step across the kink
    vb = rand((3, N), F32, 4)
    dz, db = torch.empty_like(z, device="cuda"), torch.empty((3, N), device="cuda")
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(3, N, 32), dtype=torch.uint8, device="cuda")
    Q.moe_expert_act_backward(dy.cuda(), z.cuda(), offsets.cuda(), dz, db, act=kind, ws=ws)
    step = 1e-4
    spread = torch.repeat_interleave(vb, torch.tensor(sizes), 0)
    for direction, slope in ((v, (dz.cpu().to(D) * v.to(D)).sum()), (spread, (db.cpu().to(D) * vb.to(D)).sum())):
        f = [(act(z.to(D) + s * direction.to(D), kind) * dy.to(D)).sum() for s in (step, -step)]
        # differences: third derivatives below 3, 32 N terms of |v|^3 |dy| <= 30 at most on average 2
        assert abs((f[0] - f[1]) / (2 * step) - slope) < 32 * N * 2 * 3 * step ** 2 + 32 * N * 16 * F * 4


def test_captured_product_and_gradient_follow_new_batches():
    """Replays read offsets and values anew; workspaces of two graphs are their own."""
    N, K, S, R = 96, 64, 3, 40
    w, b = rand((S, N, K), BF, 1, 0.1).cuda(), rand((S, N), F32, 2).cuda()
    x, offsets = rand((R, K), BF, 3).cuda(), torch.tensor([0, 10, 10, 40], dtype=torch.int32, device="cuda")
    y, z = torch.zeros((R, N // 2), dtype=BF, device="cuda"), torch.zeros((R, N), dtype=BF, device="cuda")
    dy, dz, db = rand((R, N // 2), BF, 4).cuda(), torch.zeros((R, N), dtype=BF, device="cuda"), torch.zeros((S, N), device="cuda")
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(S, N, R), dtype=torch.uint8, device="cuda")

    def step():
        Q.moe_expert_gemm_bias(x, w, b, None, offsets, y, act=SWI, z=z)
        Q.moe_expert_act_backward(dy, z, offsets, dz, db, act=SWI, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, cut in enumerate([[0, 0, 40, 40], [0, 40, 40, 40], [0, 5, 9, 20]]):
        offsets.copy_(torch.tensor(cut, dtype=torch.int32))
        x.copy_(rand((R, K), BF, 10 + i))
        for t in (y, z, dz, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, z, dz, db)]
        for t in (y, z, dz, db):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, z, dz, db)))


def test_binding_refuses():
    x, w = rand((4, 16), BF, 0).cuda(), rand((2, 32, 16), BF, 1).cuda()
    off, y = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"), torch.zeros((4, 32), dtype=BF, device="cuda")
    good = dict(x=x, w=w, bias=torch.zeros((2, 32), device="cuda"), residual=None, slot_offsets=off, y=y)
    Q.moe_expert_gemm_bias(**good)
    for kw, error in ((dict(bias=torch.zeros(32, device="cuda")), ValueError), (dict(bias=torch.zeros((2, 32))), TypeError),
                      (dict(residual=y[:3]), ValueError), (dict(residual=y.double()), TypeError),
                      (dict(z=torch.zeros((4, 32), device="cuda")), TypeError), (dict(y=y[:, :16]), ValueError),
                      (dict(x=x[::2]), ValueError), (dict(bias=torch.zeros((2, 32), device="cuda", requires_grad=True)), ValueError),
                      (dict(z=y), Q.QmoeError)):
        with pytest.raises(error):
            Q.moe_expert_gemm_bias(**{**good, **kw})
    dz, db = torch.zeros_like(y), torch.zeros((2, 32), device="cuda")
    ws = torch.empty(Q.moe_expert_act_backward_workspace_size(2, 32, 4), dtype=torch.uint8, device="cuda")
    good = dict(dy=y, z=y.clone(), slot_offsets=off, dz=dz, dbias=db, act=Q.MOE_ACT_GELU, ws=ws)
    Q.moe_expert_act_backward(**good)
    for kw, error in ((dict(z=y[:, :16].contiguous()), ValueError), (dict(dz=dz.float()), TypeError),
                      (dict(dbias=db.bfloat16()), ValueError), (dict(dbias=db[:1]), ValueError), (dict(ws=ws[:16]), Q.QmoeError),
                      (dict(rows=TOKEN), ValueError), (dict(slot_offsets=off.long()), ValueError)):
        with pytest.raises(error):
            Q.moe_expert_act_backward(**{**good, **kw})
