"""Inputs and 64-bit plain forms of the expert products, the 4-bit products,
the block norms and SwiGLU, for their tests (CPU tensors)."""
from __future__ import annotations

import torch

import quantized_routed_expert_moe_amd as Q

D = torch.float64
EPS16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step of a type


def batches(sizes, P, k, seed):
    """Offsets of the given slot sizes and a permutation of the P pairs, as moe_build_expert_batches lays them out."""
    g = torch.Generator().manual_seed(seed)
    offsets = torch.zeros(len(sizes) + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(torch.tensor(sizes), 0).to(torch.int32)
    perm = torch.randperm(P, generator=g).to(torch.int32)
    return offsets, perm


def rows_of(mode, perm, k, a, b):
    if mode == Q.MOE_ROWS_POSITION:
        return torch.arange(a, b)
    p = perm[a:b].long()
    return p if mode == Q.MOE_ROWS_PAIR else p // k


def silu(v):
    return v / (1 + torch.exp(-v))


def w4_matrix(q, scales, zeros, group):
    """float64 [S, N, K] of codes, scales and zeros."""
    S, N, _ = q.shape
    code = torch.stack((q & 15, q >> 4), -1).reshape(S, N, -1).to(D)
    z = 8.0 if zeros is None else zeros.to(D).repeat_interleave(group, 2)
    return (code - z) * scales.to(D).repeat_interleave(group, 2)


def w4_magnitude(q, scales, zeros, group):
    """scale (code + zero): what the terms of code x and zero x amount to when their sums are taken apart."""
    return w4_matrix(q, scales, zeros, group) + 2 * (8.0 if zeros is None else zeros.to(D).repeat_interleave(group, 2)) \
        * scales.to(D).repeat_interleave(group, 2)


def product(x, w, offsets, R, perm, k, x_rows, y_rows, transpose, act, w_mag=None):
    """(y, written rows, scale): y in 64 bits; scale = sum |x| |w| (or |x| w_mag), what an fp32 sum's error is
    relative to."""
    S, N, K = w.shape
    width = K if transpose else N // 2 if act else N
    y, mag = torch.zeros((R, width), dtype=D), torch.zeros((R, width), dtype=D)
    written = torch.zeros(R, dtype=torch.bool)
    for s in range(S):
        a, b = (int(offsets[s]), int(offsets[s + 1])) if offsets is not None else (0, R)
        xs, m = x[rows_of(x_rows, perm, k, a, b)].to(D), w[s].to(D)
        m = m if transpose else m.t()
        v, t = xs @ m, xs.abs() @ (m.abs() if w_mag is None else w_mag[s].t())
        if act:
            g, u, tg, tu = v[:, :width], v[:, width:], t[:, :width], t[:, width:]
            # |d(silu(g) u)| <= 1.1 |dg| |u| + |silu(g)| |du|
            v, t = silu(g) * u, 1.1 * tg * u.abs() + silu(g).abs() * tu
        iy = rows_of(y_rows, perm, k, a, b)
        y[iy], mag[iy] = v, t
        written[iy] = True
    return y, written, mag


def wgrad(dy, x, offsets, S, R, perm, k, dy_rows, x_rows):
    """(dw, sum |dy| |x|) in 64 bits."""
    out, mag = [], []
    for s in range(S):
        a, b = (int(offsets[s]), int(offsets[s + 1])) if offsets is not None else (0, R)
        u, v = dy[rows_of(dy_rows, perm, k, a, b)].to(D), x[rows_of(x_rows, perm, k, a, b)].to(D)
        out.append(u.t() @ v)
        mag.append(u.abs().t() @ v.abs())
    return torch.stack(out), torch.stack(mag)


def check_sums(got, want, mag, terms, dtype, act=False):
    """Every element within what its roundings allow.

    The products of two 16-bit values are exact in fp32.  Each of the n
    additions rounds (or, inside a matrix instruction, cuts) by at most 2^-23
    of the running sum.  The terms are zero-mean, so a running sum is a
    random walk that stays within about 4 sum|terms| / sqrt(n): together
    n 2^-23 4 sum|terms| / sqrt(n) = 8 sqrt(n) 2^-24 sum|terms|, and never
    more than 2 n 2^-24 sum|terms|.
    The activation adds a few relative roundings (8 * 2^-24), the store half a
    step of its type.  fp16 results below its normal range are off by up to
    half its smallest step, 2^-25.
    """
    got, f = got.to(D), 2.0 ** -24
    bound = min(2 * terms, 8 * terms ** 0.5) * f * mag + EPS16[dtype] * want.abs() * (1 + 2.0 ** -7)
    if act:
        bound = bound + 8 * f * want.abs()
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25
    bad = ~((got - want).abs() <= bound + 1e-35)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} elements out of bound, worst "
                           f"{float(((got - want).abs() / (bound + 1e-35)).max()):.2f} x, first at "
                           f"{[int(v) for v in bad.nonzero()[0]]}")
