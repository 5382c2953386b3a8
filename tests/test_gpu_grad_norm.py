"""moe_grad_norm and moe_grad_clip against their formulas in 64 bits: types, odd sizes and places, long lists, in place and
into other buffers, values at the ends of the range, infinities and NaN."""
import math

import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, EPS16
from tests.train_util import F, rand, store_bound, within

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def norm(grads, kind=Q.MOE_NORM_L2, scale=1.0):
    total = torch.full((1,), -7.0, device="cuda")
    ws = torch.empty(Q.moe_grad_norm_workspace_size(len(grads)), dtype=torch.uint8, device="cuda")
    Q.moe_grad_norm(grads, total, kind, scale, ws=ws)
    return total


def exact(grads, kind=Q.MOE_NORM_L2, scale=1.0):
    g = [t.cpu().to(D).reshape(-1) for t in grads]
    if kind == Q.MOE_NORM_MAX:
        return abs(scale) * max([float(t.abs().max()) for t in g if t.numel()], default=0.0)
    return abs(scale) * math.sqrt(sum(float((t * t).sum()) for t in g))


def check(sizes, types, outs=None, max_norm=1.0, scale=1.0, eps=1e-6, seed=0, mean=1.0):
    grads = [rand((n,), t, seed + i, mean) for i, (n, t) in enumerate(zip(sizes, types))]
    dev = [g.cuda() for g in grads]
    want = exact(grads, scale=scale)
    total = norm(dev, scale=scale)
    # the sum is in 64 bits: one rounding of the root
    assert abs(float(total) - want) <= F * want * (1 + 2.0 ** -20)
    out = None if outs is None else [torch.full((n,), -7.0, dtype=t, device="cuda") for n, t in zip(sizes, outs)]
    Q.moe_grad_clip(dev, total, max_norm, eps, scale, out)
    factor = scale * min(1.0, max_norm / (want + eps))
    for g, o, d in zip(grads, dev if out is None else out, dev):
        w = g.to(D) * factor
        # the norm's rounding, the factor's, the product's, the store's
        within(o, w, 3 * F * w.abs() * (1 + 2.0 ** -20) + (store_bound(w, o.dtype) if o.dtype != F32 else 0), "clipped")
        if out is not None:
            assert torch.equal(d.cpu(), g)  # the gradient itself stays


@pytest.mark.parametrize("kind", [BF, HF, F32])
@pytest.mark.parametrize("out", [None, BF, HF, F32])
@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
def test_types(kind, out, max_norm):
    sizes = [1, 7, 8, 9, 4095, 4096, 4097, 100003]
    check(sizes, [kind] * 8, None if out is None else [out] * 8, max_norm=max_norm)


@pytest.mark.parametrize("scale", [1.0, 0.125, -2.0])
def test_mixed_types_and_scales(scale):
    sizes = [3000, 1, 0, 555, 70000, 16, 31]
    types = [BF, F32, F32, HF, F32, BF, HF]
    check(sizes, types, None, 2.0, scale)
    check(sizes, types, [F32, BF, F32, F32, HF, BF, F32], 2.0, scale)


@pytest.mark.parametrize("n", [1, 159, 160, 161, 239, 240, 241, 500])
def test_long_lists(n):
    sizes = [(i * 37) % 300 for i in range(n)]
    sizes[-1] = 5
    check(sizes, [(BF, HF, F32)[i % 3] for i in range(n)], None, 1.5)


@pytest.mark.parametrize("n", [161, 241, 317, 4100])
@pytest.mark.parametrize("out", [None, BF])
def test_long_lists_by_their_table(n, out):
    """A kept list of more tensors than a launch's arguments hold: one launch, the results of the plain list."""
    sizes = [0 if i % 50 == 7 else 1 + (i * 37) % 300 for i in range(n)]
    sizes[n // 2] = 70001
    types = [(BF, HF, F32)[i % 3] for i in range(n)]
    grads = [rand((s,), t, i).cuda() for i, (s, t) in enumerate(zip(sizes, types))]
    plain = [g.clone() for g in grads]
    lst, want = Q.moe_tensor_list(grads), exact(grads)
    assert lst.table is not None
    for kind, w in ((Q.MOE_NORM_L2, want), (Q.MOE_NORM_MAX, exact(grads, Q.MOE_NORM_MAX))):
        assert abs(float(norm(lst, kind)) - w) <= F * w * 1.001
    total = norm(lst)
    make = lambda: None if out is None else [torch.full((s,), -7.0, dtype=out, device="cuda") for s in sizes]
    a, b = make(), make()
    Q.moe_grad_clip(plain, total, 3.0, outs=a)
    kept = None if b is None else Q.moe_tensor_list(b)
    Q.moe_grad_clip(lst, total, 3.0, outs=kept)
    for p, q in zip(a or plain, b or grads):
        assert torch.equal(p, q)
    s = torch.cuda.Stream()  # another stream than the table's: the arguments carry the list
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert lst.table_on(torch.cuda.current_stream().cuda_stream) == 0
        again = norm(lst)
    s.synchronize()
    w = exact(grads)
    assert abs(float(again) - w) <= F * w * 1.001


def test_long_list_captured_outlives_its_table():
    grads = [rand((100 + i,), F32, i).cuda() for i in range(300)]
    total, ws = torch.zeros(1, device="cuda"), torch.empty(Q.moe_grad_norm_workspace_size(300), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(g) for g in grads]
    lst, out = Q.moe_tensor_list(grads), Q.moe_tensor_list(outs)
    Q.moe_grad_norm(lst, total, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.moe_grad_norm(lst, total, ws=ws)
        Q.moe_grad_clip(lst, total, 2.0, outs=out)
        inside = Q.moe_tensor_list(grads)  # no copy while capturing
        assert inside.table is None
        Q.moe_grad_norm(inside, total, ws=ws)
    del lst, out, inside
    fill = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")  # what the tables' memory may hold by now
    for seed in range(3):
        for g in grads:
            g.copy_(rand(g.shape, F32, seed * 1000 + g.numel()))
        graph.replay()
        torch.cuda.synchronize()
        want = exact(grads)
        assert abs(float(total) - want) <= F * want * 1.001
        for g, o in zip(grads, outs):
            w = g.cpu().to(D) * min(1.0, 2.0 / (want + 1e-6))
            within(o, w, 3 * F * w.abs() * 1.001, "clipped")
    assert int(fill[0]) == 255


def test_long_list_captured_does_not_read_its_table():
    """The tables' own bytes are cleared before the replays: entries of nothing, with which a norm would be 0 and outputs
    would stay."""
    grads = [rand((100 + i,), F32, i).cuda() for i in range(300)]
    total, ws = torch.zeros(1, device="cuda"), torch.empty(Q.moe_grad_norm_workspace_size(300), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(g) for g in grads]
    lst, out = Q.moe_tensor_list(grads), Q.moe_tensor_list(outs)
    Q.moe_grad_norm(lst, total, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.moe_grad_norm(lst, total, ws=ws)
        Q.moe_grad_clip(lst, total, 2.0, outs=out)
    for t in (lst.table, out.table):
        t.zero_()
    torch.cuda.synchronize()
    for seed in range(3):
        for g, o in zip(grads, outs):
            g.copy_(rand(g.shape, F32, seed * 1000 + g.numel()))
            o.fill_(-7.0)
        total.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = exact(grads)
        assert abs(float(total) - want) <= F * want * 1.001
        for g, o in zip(grads, outs):
            w = g.cpu().to(D) * min(1.0, 2.0 / (want + 1e-6))
            within(o, w, 3 * F * w.abs() * 1.001, "clipped")


def test_empty_lists_and_tensors():
    assert float(norm([])) == 0.0
    empty = [torch.empty(0, dtype=BF, device="cuda"), torch.empty((0, 5), device="cuda")]
    assert float(norm(empty)) == 0.0
    Q.moe_grad_clip(empty, torch.ones(1, device="cuda"), 1.0)


@pytest.mark.parametrize("kind", [BF, HF, F32])
@pytest.mark.parametrize("out", [BF, HF, F32])
def test_odd_places_of_one_buffer(kind, out):
    """Views behind one another, none of them at a 16-byte boundary; what lies between and around stays."""
    sizes = [5, 1, 12, 4099, 3, 2, 20001, 8, 6]
    flat, to = rand((sum(sizes) + 4,), kind, 1).cuda(), torch.full((sum(sizes) + 9,), -7.0, dtype=out, device="cuda")
    keep = flat.clone()
    grads, outs, at = [], [], 0
    for n in sizes:
        grads.append(flat[at + 3:at + 3 + n])
        outs.append(to[at + 5:at + 5 + n])
        at += n
    total = norm(grads)
    want = exact(grads)
    assert abs(float(total) - want) <= F * want * (1 + 2.0 ** -20)
    Q.moe_grad_clip(grads, total, 3.0, 0.0, outs=outs)
    w = keep[3:3 + sum(sizes)].cpu().to(D) * (3.0 / want)
    within(to[5:5 + sum(sizes)], w, 3 * F * w.abs() * 1.001 + (store_bound(w, out) if out != F32 else 0), "clipped")
    assert (to[:5] == -7).all() and (to[5 + sum(sizes):] == -7).all() and torch.equal(flat, keep)
    Q.moe_grad_clip(grads, total, 3.0, 0.0)
    within(flat[3:3 + sum(sizes)], w, 3 * F * w.abs() * 1.001 + (store_bound(w, kind) if kind != F32 else 0), "in place")
    assert torch.equal(flat[:3], keep[:3]) and torch.equal(flat[-1:], keep[-1:])


def test_any_shape_and_a_list_that_is_kept():
    grads = [rand((3, 5, 7), F32, 1).cuda(), rand((64, 40), BF, 2).cuda(), rand((), F32, 3).cuda()]
    first = [g.clone() for g in grads]
    lst = Q.moe_tensor_list(grads)
    assert len(lst) == 3
    for _ in range(2):
        total, want = norm(lst), exact(grads)
        assert abs(float(total) - want) <= F * want * 1.001
        Q.moe_grad_clip(lst, total, 4.0)
    assert abs(float(norm(lst)) - 4.0) < 0.02 and not torch.equal(first[0], grads[0])


@pytest.mark.parametrize("big,small", [(3e38, 1.0), (1e25, 1e-10), (1e-30, 1e-38), (1e-38, 1e-40)])
def test_ends_of_the_range(big, small):
    """Squares beyond fp32's range, both ways; totals beyond it are infinite."""
    g = [torch.tensor([big, -big / 2, small]), torch.full((5000,), small)]
    dev, want = [t.cuda() for t in g], exact(g)
    total = norm(dev)
    if want > 3.4028235677973366e38:
        assert float(total) == math.inf
        return
    assert abs(float(total) - want) <= F * want * 1.001 + 1e-45
    limit = want / 2
    Q.moe_grad_clip(dev, total, limit, 0.0)
    limit = float(torch.tensor(limit, dtype=F32))
    for a, b in zip(g, dev):
        w = a.to(D) * min(1.0, limit / want)
        within(b, w, 4 * F * w.abs() + 2.0 ** -149 + (1e-38 * 2 ** -20 if big < 1e-37 else 0) + F * want * 0 + 1.5e-45, "clipped")


def test_long_sums_do_not_drift():
    """2^26 equal squares and one that a 32-bit sum would lose."""
    g = torch.full((1 << 26,), 1e-3, device="cuda")
    total = norm([g, torch.full((1,), 0.5, device="cuda")])
    want = math.sqrt(float(g[0].double()) ** 2 * (1 << 26) + 0.25)
    assert abs(float(total) - want) <= F * want * 1.001


def test_more_than_2_to_31_elements():
    g = torch.zeros((1 << 31) + 4097, dtype=BF, device="cuda")
    g[-1], g[-4097], g[0], g[1 << 31] = 3.0, 4.0, 12.0, 84.0  # the second and the last are one element: 84
    total, want = norm([g]), math.sqrt(9 + 144 + 7056)
    assert abs(float(total) - want) <= F * want * 1.001
    assert float(norm([g], Q.MOE_NORM_MAX)) == 84.0
    Q.moe_grad_clip([g], total, 42.5, 0.0)
    w = torch.tensor([3.0, 84.0, 12.0, 84.0, 0.0], dtype=D) * (42.5 / want)
    within(torch.stack((g[-1], g[-4097], g[0], g[1 << 31], g[1])), w, 3 * F * w + store_bound(w, BF), "clipped")


@pytest.mark.parametrize("kind", [BF, HF, F32])
def test_largest_magnitude(kind):
    sizes = [1, 0, 70001, 33]
    grads = [rand((n,), kind, i).cuda() for i, n in enumerate(sizes)]
    grads[2][60000] = -100.0
    assert float(norm(grads, Q.MOE_NORM_MAX, 0.5)) == 50.0
    grads[3][2] = math.inf
    assert float(norm(grads, Q.MOE_NORM_MAX)) == math.inf
    grads[0][0] = -math.nan
    assert math.isnan(float(norm(grads, Q.MOE_NORM_MAX)))
    assert math.isnan(float(norm(grads)))


def test_infinite_and_nan_totals():
    g = [torch.tensor([1.0, math.inf, 2.0], device="cuda"), torch.tensor([5.0], device="cuda")]
    total = norm(g)
    assert float(total) == math.inf
    out = [torch.zeros(3, device="cuda"), torch.zeros(1, device="cuda")]
    Q.moe_grad_clip(g, total, 1.0, outs=out)
    assert out[0][0] == 0 and math.isnan(out[0][1]) and out[1][0] == 0
    g[0][1] = math.nan
    total = norm(g)
    assert math.isnan(float(total))
    Q.moe_grad_clip(g, total, 1.0)
    assert torch.isnan(g[0]).all() and torch.isnan(g[1]).all()

@pytest.mark.parametrize("kind", [BF, HF, F32])
@pytest.mark.parametrize("place", ["in place", "another type", "odd place"])
@pytest.mark.parametrize("total,max_norm,factor", [
    (math.inf, math.inf, 1.0), (5.0, math.inf, 1.0), (0.0, math.inf, 1.0), (math.inf, 3.4028234663852886e38, 0.0),
    (math.inf, 0.0, 0.0), (math.nan, math.inf, math.nan), (0.0, 0.0, 1.0),
])
def test_infinite_largest_norm_clips_nothing(kind, place, total, max_norm, factor):
    """max_norm = inf leaves the gradients as they are whatever their total, NaN aside; scale still counts."""
    for scale in (1.0, 0.5):
        g = [rand((n,), kind, n).cuda() for n in (1, 1000, 4103)]
        if place == "odd place":
            g = [torch.cat((t[:1], t))[1:] for t in g]
        first = [t.clone() for t in g]
        outs = [torch.full(t.shape, -7.0, device="cuda") for t in g] if place == "another type" else None
        Q.moe_grad_clip(g, torch.full((1,), total, device="cuda"), max_norm, 0.0, scale=scale, outs=outs)
        for t, o in zip(first, outs or g):
            want = t.to(o.dtype) * (scale * factor)  # a half, exactly, or one rounding of fp16's smallest
            assert torch.equal(o, want) if factor == factor else torch.isnan(o).all()


def test_overflowing_total_of_finite_gradients():
    """The norm of finite gradients may lie beyond fp32: nothing is lost where no clipping is asked for."""
    g = [torch.full((1000,), 3e38, device="cuda"), rand((5000,), F32, 1).cuda()]
    first = [t.clone() for t in g]
    total = norm(g)
    assert float(total) == math.inf
    Q.moe_grad_clip(g, total, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(first, g))


def test_zero_gradients_stay_zero():
    g = [torch.zeros(100, device="cuda"), torch.zeros(9, dtype=BF, device="cuda")]
    total = norm(g)
    for max_norm, eps in ((1.0, 0.0), (0.0, 0.0), (0.0, 1e-6)):
        out = [torch.full_like(t, 3.0) for t in g]
        Q.moe_grad_clip(g, total, max_norm, eps, outs=out)
        assert float(total) == 0.0 and all((o == 0).all() for o in out)


def test_small_norms_leave_the_gradients():
    g = [rand((100,), BF, 1).cuda(), rand((7,), F32, 2).cuda()]
    keep = [t.clone() for t in g]
    Q.moe_grad_clip(g, norm(g), 1e4)
    assert all(torch.equal(a, b) for a, b in zip(g, keep))
    out = [torch.zeros_like(t) for t in g]
    Q.moe_grad_clip(g, norm(g), 1e4, outs=out)
    assert all(torch.equal(a, b) for a, b in zip(out, keep))


def test_equal_calls_give_equal_bits_and_replays_follow():
    grads = [rand((n,), F32, n).cuda() for n in (5, 100001, 33, 7000)]
    lst, outs = Q.moe_tensor_list(grads), [torch.zeros(g.shape, dtype=BF, device="cuda") for g in grads]
    total, ws = torch.zeros(1, device="cuda"), torch.empty(Q.moe_grad_norm_workspace_size(4), dtype=torch.uint8, device="cuda")

    def step():
        Q.moe_grad_norm(lst, total, ws=ws)
        Q.moe_grad_clip(lst, total, 3.0, outs=outs)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        for g in grads:
            g.copy_(rand(g.shape, F32, seed * 7 + g.numel(), 0.5 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [total.clone()] + [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, [total] + outs))


def test_on_another_stream():
    g = [rand((50000,), F32, 1).cuda()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        total = norm(g)
    s.synchronize()
    want = exact(g)
    assert abs(float(total) - want) <= F * want * 1.001


def test_binding_refuses():
    a, b = torch.zeros(10, device="cuda"), torch.zeros(10, dtype=BF, device="cuda")
    total = torch.ones(1, device="cuda")
    ws = torch.empty(Q.moe_grad_norm_workspace_size(2), dtype=torch.uint8, device="cuda")
    Q.moe_grad_norm([a, b], total, ws=ws)
    for bad, error in (([a, a], ValueError), ([a, a[5:]], ValueError), ([a[::2]], ValueError), ([a.cpu()], TypeError),
                       ([a.double()], TypeError), ([a.clone().requires_grad_()], ValueError), ([None], TypeError)):
        with pytest.raises(error):
            Q.moe_grad_norm(bad, total, ws=ws)
        with pytest.raises(error):
            Q.moe_grad_clip(bad, total, 1.0)
    with pytest.raises(Q.QmoeError):
        Q.moe_grad_norm([a], total, ws=None)
    with pytest.raises(ValueError):
        Q.moe_grad_norm([a], total.bfloat16(), ws=ws)
    for outs in ([a[:5]], [a, b], [b[:5]]):
        with pytest.raises(ValueError):
            Q.moe_grad_clip([a], total, 1.0, outs=outs)
    with pytest.raises(ValueError):  # an output in another gradient's place
        Q.moe_grad_clip([a, b], total, 1.0, outs=[b.view(BF), b.clone()])
    with pytest.raises(ValueError):  # its own gradient in another type
        Q.moe_grad_clip([a[:5]], total, 1.0, outs=[a.view(BF)[:5]])
    Q.moe_grad_clip([a, b], total, 1.0, outs=[a, b])
