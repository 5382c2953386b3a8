"""64-bit plain forms of the biased products, the router's losses and gradients, the combine's gradient and the gradient
norm, for their tests (CPU tensors)."""
from __future__ import annotations

import math

import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, EPS16, rows_of

F = 2.0 ** -24  # half a step of fp32
ACTS = [Q.MOE_ACT_NONE, Q.MOE_ACT_SWIGLU, Q.MOE_ACT_SILU, Q.MOE_ACT_GELU, Q.MOE_ACT_GELU_TANH, Q.MOE_ACT_RELU]
ROOT = math.sqrt(2 / math.pi)


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale).to(dtype)


def act(z, kind):
    """act(z) in z's type; SwiGLU of halves."""
    if kind == Q.MOE_ACT_SWIGLU:
        g, u = z.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    if kind == Q.MOE_ACT_SILU:
        return z * torch.sigmoid(z)
    if kind == Q.MOE_ACT_GELU:
        return z * torch.special.ndtr(z)
    if kind == Q.MOE_ACT_GELU_TANH:
        return z * torch.sigmoid(2 * ROOT * (z + 0.044715 * z ** 3))
    return torch.clamp(z, min=0) if kind == Q.MOE_ACT_RELU else z


def act_grad(z, d, kind):
    """The written-out derivative, in 64 bits."""
    if kind == Q.MOE_ACT_SWIGLU:
        g, u = z.chunk(2, 1)
        s = torch.sigmoid(g)
        return torch.cat((d * u * s * (1 + g * (1 - s)), d * g * s), 1)
    if kind == Q.MOE_ACT_SILU:
        s = torch.sigmoid(z)
        return d * s * (1 + z * (1 - s))
    if kind == Q.MOE_ACT_GELU:
        return d * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if kind == Q.MOE_ACT_GELU_TANH:
        s = torch.sigmoid(2 * ROOT * (z + 0.044715 * z ** 3))
        return d * (s + z * s * (1 - s) * 2 * ROOT * (1 + 3 * 0.044715 * z * z))
    return torch.where(z > 0, d, torch.zeros_like(d)) if kind == Q.MOE_ACT_RELU else d


def within(got, want, bound, what=""):
    """Every element within its bound; infinities and NaN in the same places."""
    got = got.to(D).cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities differ"
    off = (got - want).abs()[fine]
    limit = bound.expand_as(want)[fine] + 1e-37
    assert (off <= limit).all(), (f"{what}: {int((off > limit).sum())} of {off.numel()} out of bound, worst "
                                  f"{float((off / limit).max()):.2f} x")


def sum_terms(n):
    """What n fp32 additions of terms of changing sign lose, relative to the sum of magnitudes: each rounds (or in a
    matrix instruction cuts) by 2^-23 of the running sum, a random walk within 4 / sqrt(n) of the magnitudes' sum."""
    return min(2 * n, 8 * n ** 0.5) * F


def store_bound(want, dtype):
    """Half a step of the type (2^-25 for fp16 below its normal range)."""
    return EPS16[dtype] * want.abs() * (1 + 2.0 ** -7) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def bias_product(x, w, bias, residual, offsets, R, perm, k, x_rows, y_rows, kind, out):
    """(y, z, written rows, bound of y before the store, bound of z before the store)."""
    S, N, K = w.shape
    width = N // 2 if kind == Q.MOE_ACT_SWIGLU else N
    y, by = torch.zeros((R, width), dtype=D), torch.zeros((R, width), dtype=D)
    z, bz = torch.zeros((R, N), dtype=D), torch.zeros((R, N), dtype=D)
    written = torch.zeros(R, dtype=torch.bool)
    for s in range(S):
        a, b = (int(offsets[s]), int(offsets[s + 1])) if offsets is not None else (0, R)
        ix, iy = rows_of(x_rows, perm, k, a, b), rows_of(y_rows, perm, k, a, b)
        xs, m = x[ix].to(D), w[s].to(D).t()
        v = xs @ m
        err = sum_terms(K) * (xs.abs() @ m.abs())
        if bias is not None:
            v = v + bias[s].to(D)
            err = err + F * v.abs()
        z[iy], bz[iy] = v, err
        o = act(v, kind)
        # act' is below 1.13 in magnitude; its evaluation is off by a few roundings of act and of v (1 + erf cancels)
        if kind == Q.MOE_ACT_SWIGLU:
            g, u = v.chunk(2, 1)
            eg, eu = err.chunk(2, 1)
            e = 1.13 * eg * u.abs() + (g * torch.sigmoid(g)).abs() * eu + 8 * F * o.abs()
        elif kind == Q.MOE_ACT_NONE:
            e = err
        else:
            e = 1.13 * err + 8 * F * v.abs()
        if residual is not None:
            o = o + residual[iy].to(D)
            e = e + F * o.abs()
        y[iy], by[iy] = o, e
        written[iy] = True
    return y, z, written, by, bz


def probabilities(l, score):
    if score == Q.MOE_SCORE_SOFTMAX:
        p = torch.softmax(l, 1)
    else:
        s = torch.sigmoid(l)
        p = s / s.sum(1, keepdim=True)
    return torch.nan_to_num(p, nan=0.0) if bool((l == -math.inf).all(1).any()) else p


def weights(l, ids, score, renormalize, scale):
    """moe_route_topk's weights of given ids, differentiable."""
    p = torch.softmax(l, 1) if score == Q.MOE_SCORE_SOFTMAX else torch.sigmoid(l)
    w = p.gather(1, ids.long())
    return scale * (w / w.sum(1, keepdim=True) if renormalize else w)


def losses(l, ids, score, bounds, counts=None):
    """(counts, probs, balance, z), differentiable in l; counts may be given."""
    T, E = l.shape
    k, G, n = ids.shape[1], len(bounds) - 1, bounds[-1] - bounds[0]
    p = probabilities(l, score)
    own = torch.zeros((G, E), dtype=D)
    probs = torch.zeros((G, E), dtype=D)
    for g in range(G):
        a, b = bounds[g], bounds[g + 1]
        flat = ids[a:b].reshape(-1)
        flat = flat[(flat >= 0) & (flat < E)].long()
        own[g] = torch.bincount(flat, minlength=E).to(D)
        if b > a:
            probs[g] = p[a:b].sum(0) / (b - a)
    c = own if counts is None else counts.to(D)
    lse = torch.logsumexp(l[bounds[0]:bounds[-1]], 1)
    lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    if n == 0:
        return own, probs, torch.zeros((), dtype=D), torch.zeros((), dtype=D)
    return own, probs, E / (k * n) * (c * probs).sum(), (lse ** 2).sum() / n
