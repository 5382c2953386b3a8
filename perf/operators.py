"""The measured cases of the expert products, the 4-bit products, the block norms and SwiGLU.

Each case is one pass through one operator of quantized_routed_expert_moe_amd.
With `own` false, `run` computes it in its plain form (elementary torch
operations in 32 bits); with `own` true it makes the library's call.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases
# op      "gemm": y = x w^T per expert; "gemm_t": y = x w (the data gradient); "wgrad": dw = dy^T x;
#         "w4": y = x w^T with 4-bit w; "norm" / "norm_bwd"; "swiglu" / "swiglu_bwd".
# T, k    tokens and experts per token (k = 0: one dense matrix, no routing).
# E, S    experts, and how many of them are on the card (the other experts' pairs are not computed).
# zipf    exponent of the experts' popularity (0: uniform).
# N, K    rows and columns of each expert's matrix.
# x_rows, y_rows   how the operand and the result are addressed: by batch position, by token-expert pair or by token.

def _routed(op, T, k, E, S, zipf, N, K, dtype, out, x_rows, y_rows, act, **more):
    return dict(op=op, T=T, k=k, E=E, S=S, zipf=zipf, N=N, K=K, dtype=dtype, out=out, x_rows=x_rows, y_rows=y_rows,
                act=act, **more)


def listed():
    return [
        # one decode step of two tokens through unquantized experts: gate and up with SwiGLU; weights stream once
        dict(_routed("gemm", 2, 8, 128, 128, 0.0, 1536, 2048, "bf16", "bf16", "token", "position", True),
             name="experts gate/up, decode T=2"),
        # a prompt's gate/up with SwiGLU, an odd token count, a quarter of the experts on the host
        dict(_routed("gemm", 2999, 8, 64, 48, 0.7, 2816, 2048, "fp16", "fp16", "token", "position", True),
             name="experts gate/up, prompt T=2999, 48 of 64 resident"),
        # training: the gradient through the gate/up matrices back to the pairs
        dict(_routed("gemm_t", 4096, 8, 128, 128, 0.5, 1536, 2048, "bf16", "bf16", "position", "pair", False),
             name="experts gate/up data gradient T=4096"),
        # training: the weight gradient of the gate/up matrices, held in fp32
        dict(_routed("wgrad", 4096, 8, 64, 64, 0.5, 1536, 2048, "bf16", "fp32", "token", "position", False),
             name="experts gate/up weight gradient T=4096"),
        # one token through a dense 4-bit projection: the smallest call
        dict(_routed("w4", 1, 0, 1, 1, 0.0, 4096, 2048, "fp16", "fp16", "position", "position", False, group=128,
                     zeros=False), name="4-bit projection, one token"),
        # a decode step of two tokens through 4-bit experts with zero points: gate and up with SwiGLU
        dict(_routed("w4", 2, 8, 128, 128, 0.0, 1536, 2048, "bf16", "bf16", "token", "position", True, group=64,
                     zeros=True), name="4-bit experts gate/up, decode T=2"),
        # a batch of 48 requests, large experts: the whole 4-bit pool is read
        dict(_routed("w4", 48, 8, 256, 256, 0.3, 4096, 7168, "bf16", "fp32", "token", "pair", False, group=128,
                     zeros=True), name="4-bit experts, 48 tokens, H=7168"),
        # decode: the sum after one block and the norm before the next, four rows
        dict(op="norm", T=4, H=7168, dtype="bf16", y="fp32", w="fp32", post=True, gate="channel", a=1.0,
             name="block norm, decode T=4"),
        # training: the block norm's gradient over a large batch
        dict(op="norm_bwd", T=8192, H=7168, dtype="bf16", y="bf16", w="fp32", post=True, gate="channel", a=0.5,
             name="block norm gradient T=8192"),
        # a prompt's block norm with a gate for each token, an odd row count
        dict(op="norm", T=4099, H=2048, dtype="fp16", y="fp16", w="fp16", post=True, gate="token", a=1.0,
             name="block norm, prompt T=4099"),
        # the activation between unfused products, an odd count of pairs of a short prompt
        dict(op="swiglu", T=1001, I=2048, dtype="fp16", name="SwiGLU, 1001 pairs"),
        # training: SwiGLU's gradient over the pairs of a prompt
        dict(op="swiglu_bwd", T=32768, I=768, dtype="bf16", name="SwiGLU gradient, 32768 pairs"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(v / step) * step)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm_t", "wgrad", "w4", "w4", "norm", "norm_bwd", "swiglu", "swiglu_bwd"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("norm", "norm_bwd"):
        H = _log(rng, 128, 7168, 8)
        T = _log(rng, 1, 8192 * 7168 // (2 * H) if H > 2048 else 16384)
        return dict(op=op, T=T, H=H, dtype=dtype, y=rng.choice([dtype, "fp32"]), w=rng.choice([dtype, "fp32"]),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]),
                    a=rng.choice([1.0, 0.5, 1.25]))
    if op in ("swiglu", "swiglu_bwd"):
        return dict(op=op, T=_log(rng, 1, 32768), I=_log(rng, 64, 2048, 8), dtype=dtype)
    if op == "w4":
        group = rng.choice([32, 64, 128])
        k = rng.choice([0, 2, 8])
        E = 1 if k == 0 else rng.choice([8, 24, 64, 128])
        act = rng.random() < 0.4
        N, K = _log(rng, 256, 4096, 16), max(group, _log(rng, 256, 4096, group))
        T = _log(rng, 1, 64)
        return _routed(op, T, k, E, E if k == 0 else rng.choice([E, E * 3 // 4]), 0.3 if k else 0.0, N, K, dtype,
                       rng.choice([dtype, "fp32"]), "position" if k == 0 else "token",
                       "position" if k == 0 or act else rng.choice(["position", "pair"]), act, group=group,
                       zeros=rng.random() < 0.6)
    E, k = rng.choice([(1, 1), (8, 2), (16, 4), (60, 4), (128, 8)])
    S = E if E == 1 else rng.choice([E, E * 3 // 4])
    N, K = _log(rng, 128, 2816, 16), _log(rng, 128, 2048, 8)
    T = _log(rng, 1, 32768 // k)
    act = op == "gemm" and rng.random() < 0.4
    x_rows, y_rows = {"gemm": ("token", "position") if act else rng.choice([("token", "position"), ("position", "pair")]),
                      "gemm_t": rng.choice([("pair", "position"), ("position", "pair")]),
                      "wgrad": rng.choice([("token", "position"), ("position", "pair")])}[op]
    return _routed(op, T, k, E, S, rng.choice([0.0, 0.5, 1.0]), N, K, dtype, rng.choice([dtype, "fp32"]), x_rows,
                   y_rows, act)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(gen, shape, dtype):
    """Rows of a residual stream: normal values, a few channels an order of magnitude larger."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    big = torch.rand(shape[-1], generator=gen, device="cuda") < 0.005
    return (x * torch.where(big, 12.0, 1.0)).to(dtype)


def _routing(case, gen):
    """Batches of a routed step: offsets of the resident experts' rows, and the pairs in batch order."""
    T, k, E, S = case["T"], max(case["k"], 1), case["E"], case["S"]
    P = T * k
    if E == 1:
        ids = torch.zeros((T, k), dtype=torch.int64, device="cuda")
    else:
        rank = torch.randperm(E, generator=gen, device="cuda").float() + 1.0
        u = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
        ids = torch.topk(-case["zipf"] * torch.log(rank) - torch.log(-torch.log(u)), k, dim=1).indices
    flat, order = torch.sort(ids.reshape(-1), stable=True)
    counts = torch.bincount(flat, minlength=E)[:S]
    offsets = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    sizes = counts.tolist()
    n = sum(sizes)
    perm = torch.zeros(P, dtype=torch.int32, device="cuda")
    perm[:n] = order[:n].to(torch.int32)
    slots = [s for s in range(S) if sizes[s]]
    return dict(offsets=offsets, perm=perm, P=P, n=n, k=k, slots=slots, sizes=[sizes[s] for s in slots])


def _rows(state, how):
    """Row numbers of the batch positions, as indices."""
    r = state["route"]
    if how == "position":
        return torch.arange(r["n"], device="cuda")
    pair = r["perm"][:r["n"]].long()
    return pair if how == "pair" else pair // r["k"]


def _count(case, how):
    return case["T"] if how == "token" else case["T"] * max(case["k"], 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    d = DTYPES[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        T, H, wd = case["T"], case["H"], DTYPES[case["w"]]
        s["x"] = _activations(gen, (T, H), d)
        s["y"] = _normal(gen, (T, H), DTYPES[case["y"]], 0.7)
        s["w_pre"] = (1.0 + _normal(gen, (H,), torch.float32, 0.1)).to(wd)
        s["w_post"] = (1.0 + _normal(gen, (H,), torch.float32, 0.1)).to(wd) if case["post"] else None
        s["gate"] = {"none": None, "channel": (0.4 + _normal(gen, (H,), torch.float32, 0.1)).to(wd),
                     "token": (0.4 + _normal(gen, (T, 1), torch.float32, 0.1)).to(wd)}[case["gate"]]
        if op == "norm":
            s["x_out"], s["h"] = torch.zeros_like(s["x"]), torch.zeros_like(s["x"])
        else:
            s["dx_out"], s["dh"] = _normal(gen, (T, H), d, 0.02), _normal(gen, (T, H), d, 0.02)
            s["dx"], s["dy"] = torch.zeros_like(s["x"]), torch.zeros_like(s["y"])
            f = dict(dtype=torch.float32, device="cuda")
            s["dw_pre"] = torch.zeros(H, **f)
            s["dw_post"] = torch.zeros(H, **f) if case["post"] else None
            s["dgate"] = None if s["gate"] is None else torch.zeros(s["gate"].shape, **f)
            if own:
                import quantized_routed_expert_moe_amd as Q
                s["ws"] = torch.empty(max(1, Q.moe_block_norm_backward_workspace_size(T, H)), dtype=torch.uint8,
                                      device="cuda")
        return s
    if op in ("swiglu", "swiglu_bwd"):
        T, I = case["T"], case["I"]
        s["gu"] = _normal(gen, (T, 2 * I), d, 1.5)
        s["h"] = torch.zeros((T, I), dtype=d, device="cuda")
        if op == "swiglu_bwd":
            s["dh"] = _normal(gen, (T, I), d, 0.02)
            s["dgu"] = torch.zeros((T, 2 * I), dtype=d, device="cuda")
        return s
    S, N, K = case["S"], case["N"], case["K"]
    s["route"] = r = _routing(case, gen)
    nx, ny = _count(case, case["x_rows"]), _count(case, case["y_rows"])
    out = DTYPES[case["out"]]
    if op == "w4":
        s["q"] = torch.randint(0, 256, (S, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        G = K // case["group"]
        s["scales"] = (0.004 * torch.exp(0.3 * torch.randn((S, N, G), generator=gen, device="cuda"))).to(d)
        s["zeros"] = torch.randint(4, 12, (S, N, G), generator=gen, device="cuda", dtype=torch.uint8) \
            if case["zeros"] else None
    elif op != "wgrad":
        s["w"] = _normal(gen, (S, N, K), d, 0.02)
    if op == "wgrad":
        s["x"] = _activations(gen, (nx, K), d)
        s["dy"] = _normal(gen, (ny, N), d, 0.02)
        s["dw"] = torch.zeros((S, N, K), dtype=out, device="cuda")
        if own:
            import quantized_routed_expert_moe_amd as Q
            s["ws"] = torch.empty(max(1, Q.moe_expert_gemm_wgrad_workspace_size(S, N, K, r["P"])), dtype=torch.uint8,
                                  device="cuda")
        return s
    s["x"] = _activations(gen, (nx, N if op == "gemm_t" else K), d)
    width = K if op == "gemm_t" else N // 2 if case["act"] else N
    s["y_out"] = torch.zeros((ny, width), dtype=out, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _weights4(q, scales, zeros, group):
    """The fp32 matrix [N, K] that the codes, scales and zeros of one expert stand for."""
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(q.shape[0], -1, group).float()
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((v - z) * scales.float().unsqueeze(-1)).reshape(q.shape[0], -1)


def _norm_forward(s):
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    i1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) if c["post"] else None
    p = y * i1 if c["post"] else y
    r = p * s["w_post"].float() if c["post"] else y
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    xo = c["a"] * x + gate * r
    i2 = torch.rsqrt((xo * xo).mean(1, keepdim=True) + EPS)
    return i1, p, r, gate, xo, i2


def _plain(s):
    c = s["case"]
    op, d = c["op"], DTYPES[c["dtype"]]
    if op == "norm":
        _, _, _, _, xo, i2 = _norm_forward(s)
        return dict(x_out=xo.to(d), h=(xo * i2 * s["w_pre"].float()).to(d))
    if op == "norm_bwd":
        i1, p, r, gate, xo, i2 = _norm_forward(s)
        dh, n = s["dh"].float(), xo * i2
        dn = dh * s["w_pre"].float()
        dxo = s["dx_out"].float() + i2 * (dn - n * (dn * n).mean(1, keepdim=True))
        dr = dxo * gate
        out = dict(dx=(c["a"] * dxo).to(d), dw_pre=(dh * n).sum(0))
        if c["gate"] != "none":
            out["dgate"] = (dxo * r).sum(1, keepdim=True) if c["gate"] == "token" else (dxo * r).sum(0)
        if c["post"]:
            out["dw_post"] = (dr * p).sum(0)
            dp = dr * s["w_post"].float()
            dr = i1 * (dp - p * (dp * p).mean(1, keepdim=True))
        out["dy"] = dr.to(s["y"].dtype)
        return out
    if op in ("swiglu", "swiglu_bwd"):
        g, u = s["gu"].float().chunk(2, dim=1)
        sg = _sigmoid(g)
        h = (g * sg * u).to(d)
        if op == "swiglu":
            return dict(h=h)
        dh = s["dh"].float()
        return dict(h=h, dgu=torch.cat((dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg), dim=1).to(d))
    r = s["route"]
    x = s["x"].float()[_rows(s, c["x_rows"])]
    if op == "wgrad":
        dy = s["dy"].float()[_rows(s, c["y_rows"])]
        dw = torch.zeros(s["dw"].shape, dtype=s["dw"].dtype, device="cuda")
        if r["slots"]:
            dw[r["slots"]] = torch.stack([(b.t() @ a).to(dw.dtype)
                                          for a, b in zip(x.split(r["sizes"]), dy.split(r["sizes"]))])
        return dict(dw=dw)
    y = torch.zeros(s["y_out"].shape, dtype=s["y_out"].dtype, device="cuda")
    if not r["slots"]:
        return dict(y=y)
    if op == "w4":
        parts = [a @ _weights4(s["q"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e],
                               c["group"]).t() for e, a in zip(r["slots"], x.split(r["sizes"]))]
    else:
        parts = [a @ (s["w"][e].float() if op == "gemm_t" else s["w"][e].float().t())
                 for e, a in zip(r["slots"], x.split(r["sizes"]))]
    v = torch.cat(parts)
    if c["act"]:
        g, u = v.chunk(2, dim=1)
        v = g * _sigmoid(g) * u
    y[_rows(s, c["y_rows"])] = v.to(y.dtype)
    return dict(y=y)


# -------------------------------------------------------- the library's calls

def _library(s):
    import quantized_routed_expert_moe_amd as Q
    c = s["case"]
    op = c["op"]
    if op == "norm":
        Q.moe_block_norm(s["x"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["x_out"], s["h"], EPS, c["a"])
        return dict(x_out=s["x_out"], h=s["h"])
    if op == "norm_bwd":
        Q.moe_block_norm_backward(s["x"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["dx_out"], s["dh"], s["dx"],
                                  s["dy"], s["dw_post"], s["dgate"], s["dw_pre"], EPS, c["a"], s["ws"])
        return {k: s[k] for k in ("dx", "dy", "dw_post", "dgate", "dw_pre") if s[k] is not None}
    if op == "swiglu":
        Q.moe_swiglu(s["gu"], s["h"])
        return dict(h=s["h"])
    if op == "swiglu_bwd":
        Q.moe_swiglu_backward(s["gu"], s["dh"], s["dgu"], s["h"])
        return dict(h=s["h"], dgu=s["dgu"])
    r = s["route"]
    how = {"position": Q.MOE_ROWS_POSITION, "pair": Q.MOE_ROWS_PAIR, "token": Q.MOE_ROWS_TOKEN}
    xr, yr = how[c["x_rows"]], how[c["y_rows"]]
    if op == "wgrad":
        Q.moe_expert_gemm_wgrad(s["dy"], s["x"], r["offsets"], s["dw"], r["perm"], r["k"], yr, xr, s["ws"])
        return dict(dw=s["dw"])
    act = Q.MOE_ACT_SWIGLU if c["act"] else Q.MOE_ACT_NONE
    if op == "w4":
        Q.moe_expert_gemv_w4(s["x"], s["q"], s["scales"], s["zeros"], c["group"], r["offsets"], s["y_out"], r["perm"],
                             r["k"], xr, yr, act)
    else:
        Q.moe_expert_gemm(s["x"], s["w"], r["offsets"], s["y_out"], r["perm"], r["k"], xr, yr, op == "gemm_t", act)
    return dict(y=s["y_out"])


def run(state):
    return _library(state) if own else _plain(state)


# -------------------------------------------------------------------- work

def _active(case):
    """Resident experts that a step of T tokens is expected to use (independent picks by popularity)."""
    E, S, P = case["E"], case["S"], case["T"] * max(case["k"], 1)
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    return float(S) / E * float(np.sum(1.0 - (1.0 - p / p.sum()) ** P))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, e, ey = case["T"] * case["H"], BYTES[case["dtype"]], BYTES[case["y"]]
        if op == "norm":
            return {"bytes": n * (3 * e + ey), "flops": 12 * n}
        return {"bytes": n * (4 * e + 2 * ey), "flops": 30 * n}
    if op in ("swiglu", "swiglu_bwd"):
        n, e = case["T"] * case["I"], BYTES[case["dtype"]]
        return {"bytes": n * e * (3 if op == "swiglu" else 6), "flops": n * (8 if op == "swiglu" else 16)}
    N, K, e = case["N"], case["K"], BYTES[case["dtype"]]
    rows = case["T"] * max(case["k"], 1) * case["S"] / case["E"]
    x = min(rows, _count(case, case["x_rows"]))
    flops = 2.0 * rows * N * K
    if op == "wgrad":
        y = min(rows, _count(case, case["y_rows"]))
        return {"bytes": (x * K + y * N) * e + case["S"] * N * K * BYTES[case["out"]], "flops": flops}
    width_in, width = (N, K) if op == "gemm_t" else (K, N // 2 if case["act"] else N)
    weight = N * K * e
    if op == "w4":
        weight = N * K // 2 + N * K // case["group"] * (e + (1 if case["zeros"] else 0))
    return {"bytes": x * width_in * e + _active(case) * weight + rows * width * BYTES[case["out"]], "flops": flops}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, row by row groups, from the same inputs."""
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op in ("norm", "norm_bwd"):
        return _exact_norm(s)
    if op in ("swiglu", "swiglu_bwd"):
        I = case["I"]
        gate, up = s["gu"][:, :I].to(D), s["gu"][:, I:].to(D)
        act = torch.sigmoid(gate)
        h = up * gate * act
        if op == "swiglu":
            return dict(h=h)
        dh = s["dh"].to(D)
        dgu = torch.empty(s["dgu"].shape, dtype=D, device="cuda")
        dgu[:, :I] = dh * up * (act + gate * act * (1 - act))
        dgu[:, I:] = dh * gate * act
        return dict(h=h, dgu=dgu)
    offsets, perm = s["route"]["offsets"].tolist(), s["route"]["perm"].long()
    k = s["route"]["k"]

    def at(how, a, b):
        if how == "position":
            return torch.arange(a, b, device="cuda")
        return perm[a:b] if how == "pair" else torch.div(perm[a:b], k, rounding_mode="floor")

    result = torch.zeros((s["dw"] if op == "wgrad" else s["y_out"]).shape, dtype=D, device="cuda")
    for e in range(case["S"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        x = s["x"][at(case["x_rows"], a, b)].to(D)
        iy = at(case["y_rows"], a, b)
        if op == "wgrad":
            result[e] = torch.mm(s["dy"][iy].to(D).t().contiguous(), x)
            continue
        if op == "w4":
            code = s["q"][e].to(torch.int64)
            w = torch.empty((case["N"], case["K"]), dtype=D, device="cuda")
            w[:, 0::2] = (code % 16).to(D)
            w[:, 1::2] = (code // 16).to(D)
            zero = torch.full_like(s["scales"][e], 8.0, dtype=D) if s["zeros"] is None else s["zeros"][e].to(D)
            w -= zero.repeat_interleave(case["group"], dim=1)
            w *= s["scales"][e].to(D).repeat_interleave(case["group"], dim=1)
        else:
            w = s["w"][e].to(D)
        v = torch.mm(x, w if op == "gemm_t" else w.t().contiguous())
        if case["act"]:
            half = case["N"] // 2
            v = torch.sigmoid(v[:, :half]) * v[:, :half] * v[:, half:]
        result[iy] = v
    return dict(dw=result) if op == "wgrad" else dict(y=result)


def _exact_norm(s):
    c, D = s["case"], torch.float64
    H = c["H"]
    x, y = s["x"].to(D), s["y"].to(D)
    w_pre = s["w_pre"].to(D)
    w_post = s["w_post"].to(D) if c["post"] else torch.ones(H, dtype=D, device="cuda")
    gate = torch.ones(1, dtype=D, device="cuda") if s["gate"] is None else s["gate"].to(D)
    ry = torch.sqrt(y.square().sum(1, keepdim=True) / H + EPS) if c["post"] else torch.ones_like(y[:, :1])
    xo = x * c["a"] + y / ry * w_post * gate
    rx = torch.sqrt(xo.square().sum(1, keepdim=True) / H + EPS)
    if c["op"] == "norm":
        return dict(x_out=xo, h=xo / rx * w_pre)
    dh = s["dh"].to(D)
    out = dict(dw_pre=(dh * xo / rx).sum(0))
    v = dh * w_pre
    dxo = s["dx_out"].to(D) + v / rx - xo * (v * xo).sum(1, keepdim=True) / (H * rx ** 3)
    out["dx"] = dxo * c["a"]
    branch = dxo * gate
    if c["gate"] == "channel":
        out["dgate"] = (dxo * (y / ry * w_post)).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (dxo * (y / ry * w_post)).sum(1, keepdim=True)
    if c["post"]:
        out["dw_post"] = (branch * (y / ry)).sum(0)
        v = branch * w_post
        branch = v / ry - y * (v * y).sum(1, keepdim=True) / (H * ry ** 3)
    out["dy"] = branch
    return out
