"""moe_block_norm and its gradient against their formulas in 64 bits, every
type and optional part, and the gradients against differences; moe_swiglu
and its gradient likewise."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, EPS16

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
F = 2.0 ** -24
EPS = 1e-6


def make(T, H, dtype, y_dtype, w_dtype, post, gate, pre, seed=0):
    g = torch.Generator().manual_seed(seed)

    def n(shape, t, scale=1.0, base=0.0):
        return (base + scale * torch.randn(shape, generator=g)).to(t)

    t = dict(x=n((T, H), dtype), y=None if y_dtype is None else n((T, H), y_dtype, 0.7),
             w_post=n((H,), w_dtype, 0.2, 1.0) if post else None,
             gate={None: None, "channel": n((H,), w_dtype, 0.3, 0.5), "token": n((T, 1), w_dtype, 0.3, 0.5)}[gate],
             w_pre=n((H,), w_dtype, 0.2, 1.0) if pre else None)
    t["dx_out"], t["dh"] = n((T, H), dtype), n((T, H), dtype) if pre else None
    return t


def formula(t, a, eps=EPS):
    """Every output in 64 bits with autograd's gradients of the plain expressions."""
    v = {k: None if t[k] is None else t[k].to(D).requires_grad_() for k in ("x", "y", "w_post", "gate", "w_pre")}
    xo = a * v["x"]
    if v["y"] is not None:
        r = v["y"]
        if v["w_post"] is not None:
            r = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * v["w_post"]
        xo = xo + (r if v["gate"] is None else v["gate"] * r)
    h = None if v["w_pre"] is None else xo / torch.sqrt((xo * xo).mean(1, keepdim=True) + eps) * v["w_pre"]
    loss = (xo * t["dx_out"].to(D)).sum() if t["dx_out"] is not None else 0.0
    if h is not None:
        loss = loss + (h * t["dh"].to(D)).sum()
    names = [k for k in v if v[k] is not None]
    grads = dict(zip(names, torch.autograd.grad(loss, [v[k] for k in names])))
    return xo.detach(), None if h is None else h.detach(), grads


def close(got, want, rel, scale, name):
    """|got - want| <= rel |want| + scale: rel holds the roundings relative to the value (half a step of the output's
    type), scale those of the sums behind it."""
    err = (got.cpu().to(D) - want).abs()
    bound = rel * want.abs() * (1 + 2.0 ** -6) + scale
    assert (err <= bound).all(), f"{name}: {float((err / (bound + 1e-300)).max()):.3f} x the bound"


def dev(t):
    return None if t is None else t.cuda()


def run_both(T, H, dtype, y_dtype, w_dtype, post, gate, pre, a=1.0, seed=0):
    t = make(T, H, dtype, y_dtype, w_dtype, post, gate, pre, seed)
    xo, h, grads = formula(t, a)
    c = {k: dev(v) for k, v in t.items()}
    x_out, ho = torch.empty_like(c["x"]), torch.empty_like(c["x"]) if pre else None
    Q.moe_block_norm(c["x"], c["y"], c["w_post"], c["gate"], c["w_pre"], x_out, ho, EPS, a)
    # Forward: a row's mean square is a sum of H squares (relative error at
    # most (8 + log2 H) 2^-24 in the tree the kernel adds it in), its
    # reciprocal root and the products that follow add under 10 roundings of
    # values of at most the row's largest; 2^-24 * 40 of that covers them.
    # fp16 stores add half its smallest step.
    tiny = 2.0 ** -25 if HF in (dtype, y_dtype) else 0.0
    big = xo.abs().amax().item()
    close(x_out, xo, EPS16[dtype], 40 * F * big + tiny, "x_out")
    if pre:
        close(ho, h, EPS16[dtype], 40 * F * h.abs().amax().item() + tiny, "h")
    f = lambda w: None if w is None else torch.full(w.shape, float("nan"), device="cuda")  # noqa: E731
    dx, dy = torch.empty_like(c["x"]), None if y_dtype is None else torch.empty_like(c["y"])
    dw_post, dgate, dw_pre = f(t["w_post"]), f(t["gate"]), f(t["w_pre"])
    ws = torch.empty(max(1, Q.moe_block_norm_backward_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    Q.moe_block_norm_backward(c["x"], c["y"], c["w_post"], c["gate"], c["w_pre"], c["dx_out"], c["dh"], dx, dy,
                              dw_post, dgate, dw_pre, EPS, a, ws)
    # Gradients: dxo is a difference of terms as large as i2 |dh| w_pre; i1 and
    # i2 are at most a few here, so 200 2^-24 of the largest gradient's scale
    # covers the row sums behind m and mp.
    gx = max(grads["x"].abs().amax().item(), t["dx_out"].abs().amax().item() * abs(a))
    close(dx, grads["x"], EPS16[dtype], 200 * F * gx + tiny, "dx")
    if y_dtype is not None:
        gy = max(grads["y"].abs().amax().item(), gx / abs(a))
        close(dy, grads["y"], EPS16[y_dtype], 200 * F * gy + tiny, "dy")
    # Channel sums over T rows: at most T + 64 additions of terms bounded by
    # the largest term, each term with the 200 roundings above.
    for name, d in (("w_post", dw_post), ("gate", dgate), ("w_pre", dw_pre)):
        if d is not None:
            n = H if name == "gate" and gate == "token" else T
            term = 8.0 * max(gx / abs(a), t["dh"].abs().amax().item() if pre else 0.0)
            close(d, grads[name], 0.0, (n ** 0.5 * 200 + 8 * n ** 0.5 * min(n, 64) ** 0.5) * F * term, "d" + name)


@pytest.mark.parametrize("H", [8, 72, 512, 520, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("T", [1, 5, 333])
def test_widths_and_rows(H, T):
    run_both(T, H, BF, F32, F32, True, "channel", True, 0.5, seed=T)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("y_dtype", [BF, HF, F32])
@pytest.mark.parametrize("w_dtype", [BF, HF, F32])
def test_types(dtype, y_dtype, w_dtype):
    run_both(37, 264, dtype, y_dtype, w_dtype, True, "token", True, 1.25)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("H", [128, 2304])
def test_optional_parts(post, gate, pre, H):
    run_both(19, H, BF, BF, F32, post, gate, pre, 0.75, seed=H)


@pytest.mark.parametrize("H", [128, 2304])
def test_norm_before_a_block_alone(H):
    run_both(70, H, BF, None, BF, False, None, True, 1.0)
    # h alone, x_out not wanted
    t = make(70, H, BF, None, F32, False, None, True, 3)
    _, h, _ = formula(t, 1.0)
    out = torch.empty((70, H), dtype=BF, device="cuda")
    Q.moe_block_norm(t["x"].cuda(), None, None, None, t["w_pre"].cuda(), None, out, EPS)
    close(out, h, EPS16[BF], 40 * F * h.abs().amax().item(), "h")


def test_many_rows():
    run_both(5000, 64, BF, BF, F32, True, "channel", True)
    run_both(3001, 1032, HF, HF, HF, True, "token", True)


def test_in_place_equals_out_of_place():
    t = {k: dev(v) for k, v in make(130, 1032, BF, BF, F32, True, "channel", True).items()}
    a, b = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    Q.moe_block_norm(t["x"], t["y"], t["w_post"], t["gate"], t["w_pre"], a, b, EPS)
    x, b2 = t["x"].clone(), torch.empty_like(b)
    Q.moe_block_norm(x, t["y"], t["w_post"], t["gate"], t["w_pre"], x, b2, EPS)
    assert torch.equal(x, a) and torch.equal(b, b2)
    ws = torch.empty(Q.moe_block_norm_backward_workspace_size(130, 1032), dtype=torch.uint8, device="cuda")
    v = [torch.empty(1032, device="cuda") for _ in range(6)]
    dx, dy = torch.empty_like(a), torch.empty_like(a)
    Q.moe_block_norm_backward(t["x"], t["y"], t["w_post"], t["gate"], t["w_pre"], t["dx_out"], t["dh"], dx, dy, v[0],
                              v[1], v[2], EPS, 1.0, ws)
    dx2, dy2 = t["dx_out"].clone(), t["dh"].clone()
    Q.moe_block_norm_backward(t["x"], t["y"], t["w_post"], t["gate"], t["w_pre"], dx2, dy2, dx2, dy2, v[3], v[4], v[5],
                              EPS, 1.0, ws)
    assert torch.equal(dx, dx2) and torch.equal(dy, dy2)
    assert all(torch.equal(p, q) for p, q in zip(v[:3], v[3:]))


def test_zero_rows_and_no_rows():
    """A row of zeros is normed by sqrt(eps); no rows: nothing but zero channel gradients is written."""
    H = 264
    z = torch.zeros((3, H), dtype=BF, device="cuda")
    w = torch.full((H,), 2.0, device="cuda")
    x_out, h = torch.full_like(z, 7), torch.full_like(z, 7)
    Q.moe_block_norm(z, z, w, None, w, x_out, h, EPS)
    assert (x_out == 0).all() and (h == 0).all()
    Q.moe_block_norm(z[:0], z[:0], w, None, w, x_out[:0], h[:0], EPS)
    dw = [torch.full((H,), 7.0, device="cuda") for _ in range(2)]
    Q.moe_block_norm_backward(z[:0], z[:0], w, None, w, z[:0], z[:0], z[:0], z[:0], dw[0], None, dw[1], EPS)
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


def test_token_gate_of_zero():
    """The gate's gradient does not divide by the gate."""
    t = make(9, 264, F32, F32, F32, True, "token", True, 4)
    t["gate"][3] = 0.0
    _, _, grads = formula(t, 1.0)
    c = {k: dev(v) for k, v in t.items()}
    dx, dy = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    v = [torch.empty(264, device="cuda"), torch.empty((9, 1), device="cuda"), torch.empty(264, device="cuda")]
    ws = torch.empty(Q.moe_block_norm_backward_workspace_size(9, 264), dtype=torch.uint8, device="cuda")
    Q.moe_block_norm_backward(c["x"], c["y"], c["w_post"], c["gate"], c["w_pre"], c["dx_out"], c["dh"], dx, dy, v[0],
                              v[1], v[2], EPS, 1.0, ws)
    assert (dy[3] == 0).all()
    close(v[1], grads["gate"], 0.0, 264 ** 0.5 * 200 * F * 8 * 5.0, "dgate")


def test_gradients_against_differences():
    """Central differences of the fp32 forward call's loss in a random
    direction.  The loss sums 2 T H terms of order one in 64 bits, each output
    with a relative error of at most 40 2^-24 (a random walk over the terms),
    and the step e leaves a curvature error of order e^2: with e = 2^-6 and
    T H = 2112 values the sum's error over 2 e is below 40 * 2^-24 * 8 *
    sqrt(4224) / 2^-5 = 0.04, the third derivative's below 2^-12 / 6 times
    the direction's cubed size per value, under 0.1 on a slope of tens."""
    T, H, e = 8, 264, 2.0 ** -6
    t = make(T, H, F32, F32, F32, True, "channel", True, 6)
    c = {k: dev(v) for k, v in t.items()}
    names = ("x", "y", "w_post", "gate", "w_pre")
    dx, dy = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    v = [torch.empty(H, device="cuda") for _ in range(3)]
    ws = torch.empty(Q.moe_block_norm_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    Q.moe_block_norm_backward(*(c[n] for n in names), c["dx_out"], c["dh"], dx, dy, *v, EPS, 1.0, ws)
    got = dict(zip(names, (dx, dy, *v)))

    def loss(p):
        xo, h = torch.empty_like(p["x"]), torch.empty_like(p["x"])
        Q.moe_block_norm(*(p[n] for n in names), xo, h, EPS)
        return float((xo.double() * c["dx_out"].double()).sum() + (h.double() * c["dh"].double()).sum())

    g = torch.Generator().manual_seed(1)
    for n in names:
        d = torch.randn(c[n].shape, generator=g).cuda()
        up, down = (dict(c, **{n: c[n] + s * e * d}) for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * e)
        want = float((got[n].double() * d.double()).sum())
        size = float((got[n].double() * d.double()).abs().sum())
        assert abs(slope - want) <= 0.2 + 2.0 ** -10 * size, (n, slope, want)


# -------------------------------------------------------------------- SwiGLU

def swiglu_formula(gu, dh):
    v = gu.to(D).requires_grad_()
    I = gu.shape[1] // 2
    h = torch.sigmoid(v[:, :I]) * v[:, :I] * v[:, I:]
    return h.detach(), torch.autograd.grad((h * dh.to(D)).sum(), v)[0]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,I", [(1, 8), (3, 1400), (257, 64), (1000, 768)])
def test_swiglu(dtype, R, I):
    g = torch.Generator().manual_seed(R)
    gu, dh = (2 * torch.randn((R, 2 * I), generator=g)).to(dtype), torch.randn((R, I), generator=g).to(dtype)
    want, dwant = swiglu_formula(gu, dh)
    h, h2 = (torch.empty((R, I), dtype=dtype, device="cuda") for _ in range(2))
    Q.moe_swiglu(gu.cuda(), h)
    d = torch.empty((R, 2 * I), dtype=dtype, device="cuda")
    Q.moe_swiglu_backward(gu.cuda(), dh.cuda(), d, h2)
    assert torch.equal(h, h2)
    # under 10 roundings of 2^-24 in the sigmoid and the products; the
    # gradient's factor 1 + g (1 - s) is a sum of terms of at most 1 + |g|
    tiny = 2.0 ** -25 if dtype == HF else 1e-38
    close(h, want, EPS16[dtype] + 16 * F, tiny, "h")
    s = torch.sigmoid(gu[:, :I].to(D))
    size = torch.cat((dh.to(D) * gu[:, I:].to(D) * s * (1 + gu[:, :I].to(D).abs()), dwant[:, I:]), 1).abs()
    close(d, dwant, EPS16[dtype], 20 * F * size + tiny, "dgu")
    same = gu.cuda()
    Q.moe_swiglu_backward(same, dh.cuda(), same)
    assert torch.equal(same, d)


def test_swiglu_extreme_values():
    """silu of +-infinity and of values whose exponential overflows: the formula's limits, as torch computes them."""
    g = torch.tensor([0.0, -0.0, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38])
    gu = torch.cat((g, torch.ones(8))).reshape(1, 16).cuda()
    h = torch.empty((1, 8), device="cuda")
    Q.moe_swiglu(gu, h)
    want = g.double() * torch.sigmoid(g.double())
    assert ((h.cpu()[0].double() - want).abs() <= 16 * F * want.abs() + 1e-36).all()
    gu[0, 0], gu[0, 1] = float("inf"), float("nan")
    Q.moe_swiglu(gu, h)
    assert h[0, 0] == float("inf") and h[0, 1].isnan() and h[0, 2:].isfinite().all()


def test_swiglu_rows_of_no_slot():
    gu = torch.randn((20, 64), device="cuda").to(BF)
    off = torch.tensor([0, 5, 5, 13], dtype=torch.int32, device="cuda")
    h, full = torch.full((20, 32), -77.0, dtype=BF, device="cuda"), torch.empty((20, 32), dtype=BF, device="cuda")
    Q.moe_swiglu(gu, h, off)
    Q.moe_swiglu(gu, full)
    assert torch.equal(h[:13], full[:13]) and (h[13:] == -77.0).all()
    d, dfull = torch.full_like(gu, -77.0), torch.empty_like(gu)
    Q.moe_swiglu_backward(gu, full, d, h, off)
    Q.moe_swiglu_backward(gu, full, dfull)
    assert torch.equal(d[:13], dfull[:13]) and (d[13:] == -77.0).all() and (h[13:] == -77.0).all()
    Q.moe_swiglu(gu[:0], h[:0])
