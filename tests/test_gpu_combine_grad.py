"""moe_combine_backward against its formula in 64 bits: types, widths, numbers of pairs, pairs that are not resident, in
place, and the weights' gradient against differences of the combine itself."""
import math

import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, EPS16
from tests.train_util import F, rand, store_bound, sum_terms, within

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def setup(T, k, E, S, H, pairs, dy, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else \
        torch.zeros((0, k), dtype=torch.int32)
    w = torch.rand((T, k), generator=g)
    soe = torch.full((E,), -1, dtype=torch.int32)
    soe[torch.randperm(E, generator=g)[:S]] = torch.randperm(S, generator=g).to(torch.int32)
    return ids, w, soe, rand((T * k, H), pairs, seed + 1), rand((T, H), dy, seed + 2)


def expected(ids, w, soe, S, yp, dy):
    T, k = ids.shape
    E = soe.shape[0]
    valid = (ids >= 0) & (ids < E)
    slot = soe[ids.clamp(0, E - 1).long()]
    here = valid & (slot >= 0) & (slot < S)
    y = torch.where(here.reshape(-1, 1), yp.to(D), 0.0).reshape(T, k, yp.shape[1])
    d = dy.to(D).reshape(T, 1, yp.shape[1])
    dyp = torch.where(here.unsqueeze(2), w.to(D).unsqueeze(2) * d, 0.0).reshape(T * k, yp.shape[1])
    return dyp, (y * d).sum(2), (y * d).abs().sum(2), here


def run(ids, w, soe, S, yp, dy, inplace=False):
    ypd = yp.cuda()
    dyp = ypd if inplace else torch.full(yp.shape, -7.0, dtype=yp.dtype, device="cuda")
    dw = torch.full(w.shape, -7.0, device="cuda")
    Q.moe_combine_backward(dy.cuda(), ypd, ids.cuda(), w.cuda(), soe.cuda(), S, dyp, dw)
    return dyp.cpu(), dw.cpu()


def check(ids, w, soe, S, yp, dy, inplace=False):
    dyp, dw = run(ids, w, soe, S, yp, dy, inplace)
    want, wdw, mag, here = expected(ids, w, soe, S, yp, dy)
    within(dyp, want, F * want.abs() + store_bound(want, yp.dtype), "dy_pairs")
    within(dw, wdw, sum_terms(dy.shape[1]) * mag, "dtopk_w")
    assert (dw[~here] == 0).all() and (dyp.reshape(*here.shape, dy.shape[1])[~here] == 0).all()


@pytest.mark.parametrize("pairs", [BF, HF, F32])
@pytest.mark.parametrize("dy", [BF, HF, F32])
@pytest.mark.parametrize("T,H", [(1, 8), (5, 200), (37, 1032), (9, 7168)])
def test_types_and_widths(pairs, dy, T, H):
    check(*(s := setup(T, 4, 16, 12, H, pairs, dy, T))[:3], 12, *s[3:])


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 23, 64])
@pytest.mark.parametrize("T", [1, 3, 70])
def test_numbers_of_pairs(k, T):
    check(*(s := setup(T, k, 64, 40, 264, BF, BF, k))[:3], 40, *s[3:])


@pytest.mark.parametrize("H", [8, 16, 504, 512, 520, 1016, 1024, 1032, 2040, 2048, 2056, 4096, 16384, 16392])
@pytest.mark.parametrize("T", [2, 600])
def test_row_widths(H, T):
    check(*(s := setup(min(T, 600 if H <= 4096 else 90), 2, 8, 8, H, BF, F32, H))[:3], 8, *s[3:])


@pytest.mark.parametrize("S", [0, 1, 16])
def test_residency(S):
    ids, w, soe, yp, dy = setup(20, 4, 16, S, 64, F32, F32, S)
    check(ids, w, soe, S, yp, dy)


def test_rows_that_are_not_resident_are_not_read_and_bad_ids_count_as_such():
    ids, w, soe, yp, dy = setup(20, 4, 16, 8, 64, BF, BF, 3)
    ids[2, 1], ids[7, 3], ids[9, 0] = -1, 16, 2 ** 30
    soe[3] = 100  # a slot beyond S
    here = expected(ids, w, soe, 8, yp, dy)[3].reshape(-1)
    yp[~here] = math.nan
    w.reshape(-1)[~here] = math.inf
    check(ids, w, soe, 8, yp, dy)


def test_infinities_pass():
    ids, w, soe, yp, dy = setup(4, 2, 4, 4, 64, F32, F32, 3)
    yp[0, 5], yp[3, 1], dy[1, 1], dy[3, 2] = math.inf, -math.inf, 2.0, math.nan
    dyp, dw = run(ids, w, soe, 4, yp, dy)
    want, wdw, _, _ = expected(ids, w, soe, 4, yp, dy)
    assert torch.equal(torch.isnan(dyp), torch.isnan(want)) and torch.equal(torch.isnan(dw), torch.isnan(wdw))
    assert torch.equal(torch.isinf(dw), torch.isinf(wdw))


@pytest.mark.parametrize("pairs", [BF, F32])
@pytest.mark.parametrize("k,H", [(2, 264), (12, 2056), (8, 2048)])
def test_in_place(pairs, k, H):
    ids, w, soe, yp, dy = setup(31, k, 16, 12, H, pairs, F32, 3)
    a, b = run(ids, w, soe, 12, yp, dy), run(ids, w, soe, 12, yp, dy, inplace=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows():
    check(*(s := setup(0, 2, 4, 4, 64, BF, BF, 1))[:3], 4, *s[3:])


def test_many_rows():
    """More than 2^31 bytes of pairs, every one of them checked on the card."""
    T, k, H = 70000, 8, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 16, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    soe = torch.arange(16, dtype=torch.int32, device="cuda")
    yp = torch.randn((T * k, H), generator=g, device="cuda", dtype=BF)
    dy = torch.randn((T, H), generator=g, device="cuda", dtype=BF)
    dyp, dw = torch.empty_like(yp), torch.empty_like(w)
    Q.moe_combine_backward(dy, yp, ids, w, soe, 16, dyp, dw)
    for a in range(0, T, 10000):
        b, d = a + 10000, dy[a:a + 10000].float().unsqueeze(1)
        want = (w[a:b].unsqueeze(2) * d).to(BF)
        assert torch.equal(dyp[a * k:b * k].reshape(want.shape), want)  # one product, one rounding
        y = yp[a * k:b * k].reshape(10000, k, H).double() * d
        assert ((dw[a:b] - y.sum(2)).abs() <= sum_terms(H) * y.abs().sum(2)).all()


@pytest.mark.parametrize("k,H", [(1, 8), (9, 520)])
def test_more_tokens_than_workgroups(k, H):
    """2^20 workgroups at most: the others' tokens are taken in turn."""
    T = (1 << 20) + 777 if k == 1 else 120000
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 16, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w, soe = torch.rand((T, k), generator=g, device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda")
    yp = torch.randn((T * k, H), generator=g, device="cuda", dtype=BF)
    dy = torch.randn((T, H), generator=g, device="cuda", dtype=BF)
    dyp, dw = torch.empty_like(yp), torch.empty_like(w)
    Q.moe_combine_backward(dy, yp, ids, w, soe, 16, dyp, dw)
    d = dy.float().unsqueeze(1)
    assert torch.equal(dyp.view(T, k, H), (w.unsqueeze(2) * d).to(BF))
    y = yp.view(T, k, H).double() * d
    assert ((dw - y.sum(2)).abs() <= sum_terms(H) * y.abs().sum(2) + 1e-37).all()


def test_against_differences_of_the_combine():
    """The combine is linear in the weights and in the pairs: its own differences are the gradients, up to its fp32
    roundings (each of k + 1 sums below 2^-23 of about 8, over 64 columns of |dy| below 5)."""
    ids, w, soe, yp, dy = setup(6, 3, 8, 6, 64, F32, F32, 3)
    dyp, dw = run(ids, w, soe, 6, yp, dy)

    def combined(w, yp):
        y = torch.empty((6, 64), device="cuda")
        Q.moe_combine(yp.cuda(), ids.cuda(), w.cuda(), soe.cuda(), 6, None, y)
        return float((y.cpu().to(D) * dy.to(D)).sum())

    v, u = rand(w.shape, F32, 8), rand(yp.shape, F32, 9)
    tolerance = 6 * 64 * 5 * 4 * 2.0 ** -23 * 16 + 2 * sum_terms(64) * 6 * 3 * 64 * 4
    assert abs((combined(w + v, yp) - combined(w - v, yp)) / 2 - float((dw.to(D) * v.to(D)).sum())) < tolerance
    assert abs((combined(w, yp + u) - combined(w, yp - u)) / 2 - float((dyp.to(D) * u.to(D)).sum())) < tolerance


def test_binding_refuses():
    ids, w, soe, yp, dy = (t.cuda() for t in setup(4, 2, 4, 4, 64, BF, BF, 1))
    good = dict(dy=dy, y_pairs=yp, topk_ids=ids, topk_w=w, slot_of_expert=soe, S=4, dy_pairs=torch.empty_like(yp),
                dtopk_w=torch.empty_like(w))
    Q.moe_combine_backward(**good)
    for kw, error in ((dict(topk_ids=ids.long()), ValueError), (dict(topk_w=w[:3]), ValueError), (dict(y_pairs=yp[:7]), ValueError),
                      (dict(dy_pairs=torch.empty_like(yp, dtype=F32)), ValueError), (dict(dy=dy[:3]), ValueError),
                      (dict(S=5), Q.QmoeError), (dict(slot_of_expert=soe.long()), ValueError), (dict(dy=dy.cpu()), TypeError),
                      (dict(y_pairs=yp.clone().requires_grad_()), ValueError), (dict(dtopk_w=w), Q.QmoeError)):
        with pytest.raises(error):
            Q.moe_combine_backward(**{**good, **kw})
