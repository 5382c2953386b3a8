"""moe_balance_loss and moe_route_backward against their formulas in 64 bits: both scores, widths, ragged and empty
sequences, padding, masked logits, and the gradient against autograd of the formula and against differences."""
import math

import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D
from tests.train_util import F, losses, probabilities, rand, store_bound, weights, within

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16
SOFT, SIGM = Q.MOE_SCORE_SOFTMAX, Q.MOE_SCORE_SIGMOID


def batch(T, E, k, seed, shift=0.0):
    l = rand((T, E), F32, seed) + shift
    return l, torch.topk(l, k, dim=1).indices.to(torch.int32)


def run_losses(l, ids, score, bounds):
    G, E = len(bounds) - 1, l.shape[1]
    counts = torch.full((G, E), -7, dtype=torch.int32, device="cuda")
    probs, out = torch.full((G, E), -7.0, device="cuda"), torch.full((2,), -7.0, device="cuda")
    ws = torch.empty(Q.moe_balance_loss_workspace_size(l.shape[0], E, G), dtype=torch.uint8, device="cuda")
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    Q.moe_balance_loss(l.cuda(), ids.cuda(), score, counts, probs, out, off, ws=ws)
    return counts.cpu(), probs.cpu(), out.cpu()


def check_losses(l, ids, score, bounds):
    counts, probs, out = run_losses(l, ids, score, bounds)
    c, p, balance, z = losses(l.to(D), ids, score, bounds)
    assert torch.equal(counts.to(D), c)
    # a probability: the rounding of logit - largest (|.| <= 16, and 2^-24 of it in the exponent), the
    # exponential or sigmoid, the row's sum over 64 lanes, two divisions: below 60 half steps.  The mean: a sum of
    # positive terms in a chain of n / 16 rows of a wave, 16 waves, 32 parts and 16 lanes at most.
    n = max(b - a for a, b in zip(bounds, bounds[1:]))
    rel = (60 + min(n, 64 + n / 16) / 4 + 80) * F
    within(probs, p, rel * p, "probs")
    within(out[:1], balance.reshape(1), rel * balance.reshape(1) + 20 * F * balance, "balance")
    # lse is off by a few roundings of |logit| + log E <= 16
    within(out[1:], z.reshape(1), rel * z.reshape(1) + 60 * F * 16, "z")


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (8, 2), (60, 4), (64, 6), (65, 8), (128, 8), (256, 8), (300, 2), (1000, 4), (1024, 64), (1023, 64)])
@pytest.mark.parametrize("T", [1, 5, 64, 65, 1001])
def test_losses(score, E, k, T):
    l, ids = batch(T, E, k, T + E)
    check_losses(l, ids, score, [0, T])


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("bounds", [[0, 0], [0, 40], [3, 40], [0, 1, 1, 70, 100], [5, 5, 5], [0, 64, 128, 200], [10, 200, 200]])
def test_losses_of_sequences(score, bounds):
    l, ids = batch(200, 60, 4, len(bounds))
    check_losses(l, ids, score, bounds)


@pytest.mark.parametrize("score", [SOFT, SIGM])
def test_losses_of_many_sequences(score):
    cut = torch.randint(0, 3000, (1023,), generator=torch.Generator().manual_seed(2)).sort().values.tolist()
    l, ids = batch(3000, 24, 3, 4)
    check_losses(l, ids, score, [0] + cut + [3000])


def test_losses_of_many_rows():
    l, ids = batch(70001, 16, 2, 4)
    check_losses(l, ids, SIGM, [0, 70001])


def test_losses_without_rows():
    ids = torch.zeros((0, 2), dtype=torch.int32)
    counts, probs, out = run_losses(torch.zeros((0, 8)), ids, SOFT, [0, 0])
    assert (counts == 0).all() and (probs == 0).all() and (out == 0).all()
    counts, probs, out = run_losses(torch.zeros((0, 8)), ids, SIGM, [0, 0, 0])
    assert (counts == 0).all() and (probs == 0).all() and (out == 0).all()


@pytest.mark.parametrize("score", [SOFT, SIGM])
def test_even_routing_has_a_balance_of_one(score):
    l = torch.zeros((64, 8))
    ids = torch.stack([(torch.arange(2) + 2 * t) % 8 for t in range(64)]).to(torch.int32)
    _, _, out = run_losses(l, ids, score, [0, 64])
    assert abs(float(out[0]) - 1) < 1e-6 and abs(float(out[1]) - math.log(8) ** 2) < 1e-5


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("mask", [-math.inf, -1e9, float(torch.finfo(F32).min)])
def test_masked_experts_and_ids(score, mask):
    """Masked logits have probability 0, ids outside [0, E) are not counted."""
    l, ids = batch(90, 60, 4, 1)
    l[:, 7] = mask
    l[:45, 20:50] = mask
    ids = torch.topk(l, 4, dim=1).indices.to(torch.int32)
    ids[3, 1], ids[4, 0], ids[80, 3] = -1, 60, 2 ** 30
    check_losses(l, ids, score, [0, 33, 90])


def test_rows_of_nothing_but_masked_experts():
    l, ids = batch(10, 12, 2, 1)
    l[4] = -math.inf
    for score in (SOFT, SIGM):
        counts, probs, out = run_losses(l, ids, score, [0, 10])
        p = probabilities(l.to(D), score)
        assert torch.isfinite(probs).all() and torch.isfinite(out).all()
        within(probs[0], p.mean(0), 200 * F * p.mean(0), "probs")


@pytest.mark.parametrize("shift", [-200.0, -90.0, 0.0, 80.0])
def test_sigmoid_scores_of_far_logits(shift):
    """Normalised sigmoid scores where every sigmoid underflows, or is one."""
    l, ids = batch(70, 20, 2, 1)
    l = l + shift
    _, probs, _ = run_losses(l, ids, SIGM, [0, 70])
    ld = l.to(D)
    p = torch.exp(torch.nn.functional.logsigmoid(ld) - torch.logsumexp(torch.nn.functional.logsigmoid(ld), 1, keepdim=True))
    within(probs[0], p.mean(0), 200 * F * p.mean(0), "probs")


# --------------------------------------------------------------- gradient

def reference(l, ids, dw, score, renorm, scale, counts, dl, bounds):
    """(gradient by autograd of the formula, its size of terms) in 64 bits."""
    ld = l.to(D).requires_grad_()
    valid = (ids >= 0) & (ids < l.shape[1])
    total = torch.zeros((), dtype=D)
    if dw is not None:
        total = total + (weights(ld, ids.clamp(0, l.shape[1] - 1), score, renorm, scale) * torch.where(valid, dw, 0).to(D)).sum()
    if counts is not None:
        _, _, balance, z = losses(ld, ids, score, bounds, counts)
        total = total + float(dl[0]) * balance + float(dl[1]) * z
    return torch.autograd.grad(total, ld)[0]


def run_grad(l, ids, dw, score, renorm, scale, counts, dl, bounds, out=F32):
    got = torch.full(l.shape, -7.0, dtype=out, device="cuda")
    dev = lambda t: None if t is None else t.cuda()
    off = None if counts is None else torch.tensor(bounds, dtype=torch.int32, device="cuda")
    Q.moe_route_backward(l.cuda(), ids.cuda(), dev(dw), score, renorm, scale, dev(counts), dev(dl), off, got)
    return got.cpu()


def terms(l, ids, dw, score, renorm, scale, counts, dl, bounds):
    """What the parts of each logit's gradient amount to before they cancel."""
    T, E = l.shape
    ld = l.to(D)
    m = torch.zeros((T, E), dtype=D)
    if dw is not None:
        w = weights(ld, ids, score, renorm, abs(scale)).nan_to_num(0.0)
        pull = (w * dw.to(D).abs()).sum(1, keepdim=True) / max(abs(scale), 1e-30)
        if renorm or score == SIGM:
            m.scatter_add_(1, ids.long(), w * (dw.to(D).abs() + (pull if renorm else 0)))
        else:
            m = torch.softmax(ld, 1) * abs(scale) * pull
            m.scatter_add_(1, ids.long(), w * dw.to(D).abs())
    if counts is not None:
        n, k = bounds[-1] - bounds[0], ids.shape[1]
        p = probabilities(ld, score)
        for g in range(len(bounds) - 1):
            a, b = bounds[g], bounds[g + 1]
            if b > a:
                f = abs(float(dl[0])) * E / (k * n * (b - a)) * counts[g].to(D)
                m[a:b] += p[a:b] * (f + (p[a:b] * f).sum(1, keepdim=True))
        lse = torch.logsumexp(ld, 1, keepdim=True).abs() + 1
        a, b = bounds[0], bounds[-1]
        m[a:b] += abs(float(dl[1])) * 2 / max(n, 1) * (lse * torch.softmax(ld, 1).nan_to_num(0.0))[a:b]
    return m


def check_grad(l, ids, dw, score, renorm, scale, counts, dl, bounds, out=F32):
    got = run_grad(l, ids, dw, score, renorm, scale, counts, dl, bounds, out)
    want = reference(l, ids, dw, score, renorm, scale, counts, dl, bounds)
    # each part: a probability or two (60 half steps each, as in check_losses), sums over 64 lanes, a few products
    m = terms(l, ids, dw, score, renorm, scale, counts, dl, bounds)
    # the reference's own roundings: autograd adds and subtracts equal terms of a row, off by a few 2^-53 of the
    # largest, where the written-out formula (the weights renormalised over the selected) gives exactly 0
    bound = 200 * F * m + store_bound(want, out) + 64 * 2.0 ** -53 * m.sum(1, keepdim=True)
    within(got, want, bound, "dlogits")


def inputs(T, E, k, bounds, seed):
    l, ids = batch(T, E, k, seed)
    counts = losses(l.to(D), ids, SOFT, bounds)[0].to(torch.int32)
    return l, ids, rand((T, k), F32, seed + 1), counts, torch.tensor([0.3, 0.02])


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(2, 2), (7, 3), (8, 2), (60, 4), (64, 64), (65, 8), (128, 8), (256, 8), (300, 2), (1000, 4), (1024, 64), (1023, 64)])
@pytest.mark.parametrize("T", [1, 6, 301])
def test_gradient(score, renorm, E, k, T):
    bounds = [0, T // 3, T // 3, T - T // 6]
    l, ids, dw, counts, dl = inputs(T, E, k, bounds, E + T)
    check_grad(l, ids, dw, score, renorm, 2.5, counts, dl, bounds)


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("renorm,with_dw,with_losses", [(True, True, False), (False, True, False), (True, False, True)])
def test_gradient_parts_and_types(score, out, renorm, with_dw, with_losses):
    bounds = [4, 50, 77]
    for E, k in ((60, 4), (61, 4), (256, 8)):
        l, ids, dw, counts, dl = inputs(80, E, k, bounds, 3)
        check_grad(l, ids, dw if with_dw else None, score, renorm, 1.0, counts if with_losses else None,
                   dl if with_losses else None, bounds, out)


def test_gradient_of_one_expert_per_token_renormalised_is_zero():
    l, ids, dw, _, _ = inputs(40, 16, 1, [0, 40], 3)
    for score in (SOFT, SIGM):
        assert (run_grad(l, ids, dw, score, True, 1.0, None, None, None) == 0).all()


def test_gradient_in_place_and_of_unaligned_rows():
    bounds = [0, 30, 60]
    l, ids, dw, counts, dl = inputs(60, 64, 4, bounds, 3)
    want = run_grad(l, ids, dw, SOFT, False, 1.0, counts, dl, bounds)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    own = l.cuda()
    Q.moe_route_backward(own, ids.cuda(), dw.cuda(), SOFT, False, 1.0, counts.cuda(), dl.cuda(), off, own)
    assert torch.equal(own.cpu(), want)
    odd = torch.zeros(60 * 64 + 1, device="cuda")[1:].view(60, 64)  # 4 bytes behind a 16-byte boundary
    odd.copy_(l)
    got = torch.zeros((60, 64), device="cuda")
    Q.moe_route_backward(odd, ids.cuda(), dw.cuda(), SOFT, False, 1.0, counts.cuda(), dl.cuda(), off, got)
    within(got, want.to(D), 200 * F * want.to(D).abs() + 1e-6, "unaligned")
    p = torch.zeros((2, 64), device="cuda")
    c, o = torch.zeros((2, 64), dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    ws = torch.empty(Q.moe_balance_loss_workspace_size(60, 64, 2), dtype=torch.uint8, device="cuda")
    Q.moe_balance_loss(odd, ids.cuda(), SOFT, c, p, o, off, ws=ws)
    assert torch.equal(c.cpu(), counts)


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_with_masked_experts(score, renorm):
    """Masked logits get no gradient, a row of nothing else gets none at all, invalid ids are passed over."""
    l, ids, dw, counts, dl = inputs(30, 20, 3, [0, 30], 8)
    l[:, 5] = -math.inf
    l[3, 8:] = -math.inf
    l[9] = -math.inf
    ids = torch.topk(l, 3, dim=1).indices.to(torch.int32)
    got = run_grad(l, ids, dw, score, renorm, 1.0, counts, dl, [0, 30])
    assert torch.isfinite(got).all() and (got[9] == 0).all() and (got[:, 5] == 0).all() and (got[3, 8:] == 0).all()
    rest = [t for t in range(30) if t != 9]
    lf = l.clone()
    lf[lf == -math.inf] = -500.0  # the formula in 64 bits: probabilities of e^-500 and less
    want = reference(lf, ids, dw, score, renorm, 1.0, counts, dl, [0, 30])
    m = terms(lf, ids, dw, score, renorm, 1.0, counts, dl, [0, 30])
    # the mean over 30 rows counts the empty one, whose own terms the formula at -500 has in row 9 alone
    within(got[rest], want[rest], 200 * F * m[rest] + 64 * 2.0 ** -53 * m[rest].sum(1, keepdim=True), "masked")
    bad = ids.clone()
    bad[2, 1], bad[4, 0] = -1, 99
    dwn = dw.clone()
    dwn[2, 1] = dwn[4, 0] = math.nan  # weights of no expert: not used
    got = run_grad(l, bad, dwn, score, renorm, 1.0, None, None, None)
    assert torch.isfinite(got).all()
    same = [t for t in range(30) if t not in (2, 4)]
    assert torch.equal(got[same], run_grad(l, ids, dw, score, renorm, 1.0, None, None, None)[same])


def test_gradient_of_the_same_expert_twice():
    l, ids, dw, _, _ = inputs(9, 16, 3, [0, 9], 3)
    ids[:, 2] = ids[:, 0]
    for score in (SOFT, SIGM):
        for renorm in (True, False):
            check_grad(l, ids, dw, score, renorm, 1.0, None, None, [0, 9])


@pytest.mark.parametrize("score", [SOFT, SIGM])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    bounds = [0, 11, 24]
    l, ids, dw, counts, dl = inputs(24, 16, 3, bounds, 5)
    got = run_grad(l, ids, dw, score, renorm, 2.5, counts, dl, bounds).to(D)
    v = rand(l.shape, D, 9)

    def f(step):
        x = l.to(D) + step * v
        _, _, balance, z = losses(x, ids, score, bounds, counts)
        return float((weights(x, ids, score, renorm, 2.5) * dw.to(D)).sum() + float(dl[0]) * balance + float(dl[1]) * z)

    h = 1e-4
    # third derivatives of at most 72 weights of 2.5 (below 15 each) and of the losses, along |v| < 4
    assert abs((f(h) - f(-h)) / (2 * h) - float((got * v).sum())) < h * h * 72 * 15 * 64 / 6 + 24 * 16 * 200 * F


def test_equal_calls_give_equal_bits_and_replays_follow():
    bounds = [0, 400, 900]
    l, ids, dw, counts, dl = inputs(1000, 128, 8, bounds, 1)
    a, b = run_losses(l, ids, SIGM, bounds), run_losses(l, ids, SIGM, bounds)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ld, idd, dwd, dld = l.cuda(), ids.cuda(), dw.cuda(), dl.cuda()
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    c, p, o = torch.zeros((2, 128), dtype=torch.int32, device="cuda"), torch.zeros((2, 128), device="cuda"), torch.zeros(2, device="cuda")
    d = torch.zeros((1000, 128), dtype=BF, device="cuda")
    ws = torch.empty(Q.moe_balance_loss_workspace_size(1000, 128, 2), dtype=torch.uint8, device="cuda")

    def step():
        Q.moe_balance_loss(ld, idd, SIGM, c, p, o, off, ws=ws)
        Q.moe_route_backward(ld, idd, dwd, SIGM, True, 2.5, c, dld, off, d)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cut in ([0, 400, 900], [0, 0, 1000], [100, 101, 102], [0, 1000, 1000]):
        off.copy_(torch.tensor(cut, dtype=torch.int32))
        ld.copy_(rand((1000, 128), F32, cut[1] + 5))
        for t in (c, p, o, d):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c, p, o, d)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (c, p, o, d)))


def test_offsets_that_decrease_stay_in_bounds():
    """A precondition broken: wrong values, nothing outside the buffers."""
    l, ids = batch(300, 16, 2, 1)
    for bounds in ([0, 300, 0, 300, 0, 300], [300, 0], [-5, 1000], [2 ** 31 - 1, -2 ** 31, 7]):
        counts, probs, out = run_losses(l, ids, SOFT, bounds)
        d = run_grad(l, ids, None, SOFT, True, 1.0, counts, torch.ones(2), bounds)
        assert d.shape == l.shape


def inside(shape, dtype, mark):
    """A tensor in the middle of a marked buffer, on a 16-byte boundary, and the check of what lies around it."""
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    whole = torch.full((4096 + n + 4096,), mark, dtype=torch.uint8, device="cuda")
    t = whole[4096:4096 + n].view(dtype).reshape(shape)
    return t, lambda: bool((whole[:4096] == mark).all() and (whole[4096 + n:] == mark).all())


@pytest.mark.parametrize("T,E", [(300, 16), (37, 16), (1000, 264), (300, 30)])
@pytest.mark.parametrize("score", [SOFT, SIGM])
def test_offsets_that_decrease_leave_what_lies_around(T, E, score):
    """As above, with marked memory on both sides of everything that the calls write, the workspace of its exact size."""
    l, ids = batch(T, E, 2, 1)
    l, ids, dw, ones = l.cuda(), ids.cuda(), torch.ones((T, 2), device="cuda"), torch.ones(2, device="cuda")
    for bounds in ([0, T, 0, T, 0, T], [T, 0], [-5, T + 700], [2 ** 31 - 1, -2 ** 31, 7], [T] * 9 + [0], list(range(T, -1, -1))):
        G, off = len(bounds) - 1, torch.tensor(bounds, dtype=torch.int32, device="cuda")
        counts, c = inside((G, E), torch.int32, 0x5A)
        probs, p = inside((G, E), F32, 0x5A)
        losses, o = inside((2,), F32, 0x5A)
        ws, w = inside((Q.moe_balance_loss_workspace_size(T, E, G),), torch.uint8, 0x5A)
        grads = [inside((T, E), t, 0x5A) for t in (F32, BF)]
        Q.moe_balance_loss(l, ids, score, counts, probs, losses, off, ws=ws)
        for d, _ in grads:
            Q.moe_route_backward(l, ids, dw, score, True, 1.0, counts, ones, off, d)
        torch.cuda.synchronize()
        assert c() and p() and o() and w() and all(check() for _, check in grads), bounds
        # whatever the values, all of them are written (the mark is 1.5e16 in both types)
        for t in (counts, probs, losses, grads[0][0], grads[1][0]):
            assert not (t == torch.full((16,), 0x5A, dtype=torch.uint8, device="cuda").view(t.dtype)[0]).any(), bounds


def test_binding_refuses():
    l, ids = batch(6, 16, 2, 1)
    l, ids = l.cuda(), ids.cuda()
    c, p, o = torch.zeros((1, 16), dtype=torch.int32, device="cuda"), torch.zeros((1, 16), device="cuda"), torch.zeros(2, device="cuda")
    ws = torch.empty(Q.moe_balance_loss_workspace_size(6, 16, 1), dtype=torch.uint8, device="cuda")
    good = dict(logits=l, topk_ids=ids, score=SOFT, counts=c, probs=p, losses=o, ws=ws)
    Q.moe_balance_loss(**good)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    for kw, error in ((dict(logits=l.bfloat16()), ValueError), (dict(topk_ids=ids.long()), ValueError),
                      (dict(topk_ids=ids[:5]), ValueError), (dict(counts=c.float()), ValueError), (dict(seq_offsets=off), ValueError),
                      (dict(losses=o[:1]), ValueError), (dict(ws=None), Q.QmoeError), (dict(logits=l.t().contiguous().t()), ValueError),
                      (dict(logits=l.clone().requires_grad_()), ValueError), (dict(probs=p.cpu()), TypeError)):
        with pytest.raises(error):
            Q.moe_balance_loss(**{**good, **kw})
    dw, d = torch.zeros((6, 2), device="cuda"), torch.zeros((6, 16), device="cuda")
    good = dict(logits=l, topk_ids=ids, dtopk_w=dw, score=SOFT, renormalize=True, scale=1.0, counts=c, dlosses=o, seq_offsets=None,
                dlogits=d)
    Q.moe_route_backward(**good)
    for kw, error in ((dict(dtopk_w=dw[:, :1]), ValueError), (dict(counts=None), ValueError), (dict(dlosses=o[:1]), ValueError),
                      (dict(dlogits=d[:5]), ValueError), (dict(dlogits=d.double()), TypeError), (dict(seq_offsets=off), ValueError),
                      (dict(dtopk_w=None, counts=None, dlosses=None), Q.QmoeError)):
        with pytest.raises(error):
            Q.moe_route_backward(**{**good, **kw})
