"""The measured cases of the biased products, the router's losses and gradients, the combine's gradient and the
gradient norm with clipping.

Each case is one pass through one operator of quantized_routed_expert_moe_amd.
With `own` false, `run` computes it in its plain form (elementary torch
operations in 32 bits, sums over whole gradients in 64); with `own` true it
makes the library's call.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases
# op      "gemm": y = act(x w^T + b) + residual per expert; "act_bwd": its activation's and bias's gradients;
#         "losses": balance loss, z loss and counts; "route_bwd": the logits' gradient;
#         "combine_bwd": the weighted combine's gradients; "clip": norm over a list of gradients, and clipping.
# T, k    tokens and experts per token (k = 0: one dense matrix, no routing).
# E, S    experts, and how many of them are on the card.
# N, K    rows and columns of each expert's matrix.  segs: sequences of the batch.
# x_rows, y_rows   how the operand and the result are addressed: by batch position, by token-expert pair or by token.

def _gemm(T, k, E, zipf, N, K, dtype, out, x_rows, y_rows, act, bias, residual, keep, S=None):
    return dict(op="gemm", T=T, k=k, E=E, S=E if S is None else S, zipf=zipf, N=N, K=K, dtype=dtype, out=out,
                x_rows=x_rows, y_rows=y_rows, act=act, bias=bias, residual=residual, keep=keep)


def listed():
    return [
        # one decode step of four tokens through experts with biases: gate and up with SwiGLU; weights stream once
        dict(_gemm(4, 8, 128, 0.0, 1536, 2048, "bf16", "bf16", "token", "position", "swiglu", "bf16", "none", False),
             name="biased experts gate/up, decode T=4"),
        # training: gate/up of a batch with biases and SwiGLU, z kept for the backward pass
        dict(_gemm(4096, 8, 64, 0.5, 1536, 2048, "bf16", "bf16", "token", "position", "swiglu", "fp32", "none", True),
             name="biased experts gate/up, training T=4096"),
        # a prompt's output projection with bias, added to the residual stream, an odd token count
        dict(_gemm(2999, 0, 1, 0.0, 2048, 4096, "fp16", "fp16", "position", "position", "none", "fp16", "fp16", False),
             name="projection with bias and residual, T=2999"),
        # training: SwiGLU's gradient and the biases' gradients over the pairs of a batch, h written again
        dict(op="act_bwd", T=4096, k=8, E=128, S=128, zipf=0.5, N=1536, dtype="bf16", act="swiglu", rows="position",
             h=True, name="SwiGLU and bias gradients, 32768 pairs"),
        # a short batch through a dense GELU layer, an odd row count
        dict(op="act_bwd", T=1001, k=0, E=1, S=1, zipf=0.0, N=2048, dtype="fp16", act="gelu", rows="position", h=False,
             name="GELU and bias gradients, 1001 rows"),
        # training: the router's losses over a batch of eight ragged sequences and some padding
        dict(op="losses", T=16384, E=256, k=8, score="sigmoid", segs=8, pad=0.1, name="router losses, 8 sequences, T=16384"),
        # the smallest call: the losses of a short sequence
        dict(op="losses", T=37, E=128, k=8, score="softmax", segs=1, pad=0.0, name="router losses, T=37"),
        # training: the logits' gradient from the routing weights and both losses
        dict(op="route_bwd", T=16384, E=256, k=8, score="sigmoid", renorm=True, scale=2.5, segs=8, pad=0.1, out="bf16",
             balance=True, name="router gradient, T=16384"),
        # training: the combine's gradients of a batch
        dict(op="combine_bwd", T=4096, k=8, E=128, S=128, H=2048, dtype="bf16", dy="bf16", name="combine gradient T=4096"),
        # wide rows, a quarter of the experts elsewhere, an odd token count
        dict(op="combine_bwd", T=333, k=6, E=64, S=48, H=7168, dtype="bf16", dy="fp32",
             name="combine gradient T=333, 48 of 64 resident"),
        # the expert gradients of two layers, bf16, clipped into fp32 buffers
        dict(op="clip", n=4, lo=100663296, hi=201326592, types="bf16", out="fp32", flat=False, seed=5, clip=0.5, scale=1.0,
             name="norm and clipping of two layers' expert gradients"),
        # the many small gradients of norms, gates and biases, views at odd places of one buffer
        dict(op="clip", n=317, lo=1, hi=100000, types="fp32", out="fp32", flat=True, seed=7, clip=0.25, scale=0.125,
             name="norm and clipping of 317 small gradients"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(v / step) * step)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "act_bwd", "act_bwd", "losses", "route_bwd", "combine_bwd", "clip"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("gemm", "act_bwd"):
        E, k = rng.choice([(1, 0), (1, 0), (8, 2), (16, 4), (60, 4), (128, 8)])
        S = E if E == 1 else rng.choice([E, E * 3 // 4])
        N = _log(rng, 64, 2816, 16)
        K = _log(rng, 64, min(4096, 1536 * 2048 // N), 8)
        act = rng.choice(["none", "swiglu", "silu", "gelu", "gelu_tanh", "relu"])
        zipf = rng.choice([0.0, 0.5, 1.0]) if E > 1 else 0.0
        T = _log(rng, 1, 32768 // max(k, 2))
        if op == "act_bwd":
            return dict(op=op, T=T, k=k, E=E, S=S, zipf=zipf, N=min(N, 1536), dtype=rng.choice([dtype, dtype, "fp32"]),
                        act=act, rows=rng.choice(["position", "pair"]) if k else "position", h=rng.random() < 0.5)
        x_rows, y_rows = ("position", "position") if k == 0 else rng.choice([("token", "position"), ("position", "pair")])
        return _gemm(T, k, E, zipf, N, K, dtype, rng.choice([dtype, "fp32"]), x_rows, y_rows, act,
                     rng.choice(["none", dtype, "fp32"]), rng.choice(["none", "none", dtype, "fp32"]),
                     rng.random() < 0.4, S)
    if op in ("losses", "route_bwd"):
        E = rng.choice([2, 8, 60, 64, 128, 256, 256, 1000])
        T = _log(rng, 1, 16384 * 256 // max(E, 256))
        c = dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 4, 8, 8])), score=rng.choice(["softmax", "sigmoid"]),
                 segs=rng.choice([1, 1, 3, 8, 16]), pad=rng.choice([0.0, 0.1]))
        if op == "route_bwd":
            c.update(renorm=c["k"] > 1 and rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), out=rng.choice(["fp32", "bf16", "fp16"]),
                     balance=rng.random() < 0.8)
        return c
    if op == "combine_bwd":
        E, k = rng.choice([(8, 2), (16, 4), (64, 6), (128, 8)])
        H = _log(rng, 64, 7168, 8)
        return dict(op=op, T=_log(rng, 1, max(1, 4096 * 8 * 2048 // (2 * k * H)) if H > 1024 else 8192), k=k, E=E,
                    S=rng.choice([E, E * 3 // 4]), H=H, dtype=rng.choice([dtype, "fp32"]), dy=rng.choice([dtype, "fp32"]))
    hi = _log(rng, 10, 20000000)
    types = rng.choice(["bf16", "fp16", "fp32", "mixed"])
    flat = types != "mixed" and rng.random() < 0.4
    return dict(op=op, n=_log(rng, 1, max(2, min(400 if flat else 40, 200000000 // hi))), lo=1, hi=hi, types=types,
                out=rng.choice(["same", "fp32"]), flat=flat, seed=rng.randrange(1 << 30), clip=rng.choice([0.01, 0.5, 2.0]), scale=rng.choice([1.0, 0.125]))


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(gen, shape, dtype):
    """Rows of a residual stream: normal values, a few channels an order of magnitude larger."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    big = torch.rand(shape[-1], generator=gen, device="cuda") < 0.005
    return (x * torch.where(big, 12.0, 1.0)).to(dtype)


def _picks(T, E, k, zipf, gen):
    """Each token's k different experts, by popularity (rank + 1)^-zipf."""
    rank = torch.randperm(E, generator=gen, device="cuda").float() + 1.0
    u = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return torch.topk(-zipf * torch.log(rank) - torch.log(-torch.log(u)), k, dim=1).indices


def _routing(case, gen):
    """Batches of a routed step: offsets of the resident experts' rows, and the pairs in batch order."""
    T, k, E, S = case["T"], max(case["k"], 1), case["E"], case["S"]
    ids = torch.zeros((T, k), dtype=torch.int64, device="cuda") if E == 1 else _picks(T, E, k, case["zipf"], gen)
    flat, order = torch.sort(ids.reshape(-1), stable=True)
    counts = torch.bincount(flat, minlength=E)[:S]
    offsets = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    sizes = counts.tolist()
    n = sum(sizes)
    perm = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    perm[:n] = order[:n].to(torch.int32)
    slots = [s for s in range(S) if sizes[s]]
    return dict(offsets=offsets, perm=perm, P=T * k, n=n, k=k, slots=slots, sizes=[sizes[s] for s in slots])


def _rows(state, how):
    """Row numbers of the batch positions, as indices."""
    r = state["route"]
    if how == "position":
        return torch.arange(r["n"], device="cuda")
    pair = r["perm"][:r["n"]].long()
    return pair if how == "pair" else pair // r["k"]


def _count(case, how):
    return case["T"] if how == "token" else case["T"] * max(case["k"], 1)


def _segments(case):
    """Ragged sequences' bounds: rows behind the last one are padding."""
    rng = random.Random(case["T"] * 31 + case["segs"])
    end = max(1, int(case["T"] * (1.0 - case["pad"])))
    cuts = sorted(rng.randint(0, end) for _ in range(case["segs"] - 1))
    return [0] + cuts + [end]


def _sizes(case):
    rng = random.Random(case["seed"])
    sizes = [min(case["hi"], max(case["lo"], round(math.exp(rng.uniform(math.log(case["lo"]), math.log(case["hi"]))))))
             for _ in range(case["n"])]
    types = [rng.choice(["bf16", "fp16", "fp32"]) if case["types"] == "mixed" else case["types"] for _ in sizes]
    return sizes, types


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if own:
        import quantized_routed_expert_moe_amd as Q
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == "clip":
        sizes, types = _sizes(case)
        outs = ["fp32" if case["out"] == "fp32" else t for t in types]
        if case["flat"]:
            flat = _normal(gen, (sum(sizes),), DTYPES[types[0]], 0.01)
            s["grads"] = list(flat.split(sizes))
            s["flat"] = torch.zeros(sum(sizes), dtype=DTYPES[outs[0]], device="cuda")
            s["outs"] = list(s["flat"].split(sizes))
        else:
            s["grads"] = [_normal(gen, (n,), DTYPES[t], 0.01) for n, t in zip(sizes, types)]
            s["outs"] = [torch.zeros(n, dtype=DTYPES[t], device="cuda") for n, t in zip(sizes, outs)]
        s["total"] = torch.zeros(1, **f32)
        # the limit, as a share of the norm that such values have on average
        s["max_norm"] = case["clip"] * case["scale"] * 0.01 * math.sqrt(sum(sizes))
        if own:
            s["grad_list"], s["out_list"] = Q.moe_tensor_list(s["grads"]), Q.moe_tensor_list(s["outs"])
            s["ws"] = torch.empty(Q.moe_grad_norm_workspace_size(case["n"]), dtype=torch.uint8, device="cuda")
        return s
    if op == "combine_bwd":
        T, k, H = case["T"], case["k"], case["H"]
        s["ids"] = _picks(T, case["E"], k, 0.5, gen).to(torch.int32)
        s["w"] = torch.softmax(_normal(gen, (T, k), torch.float32), 1)
        where = torch.arange(case["E"], dtype=torch.int32, device="cuda")
        s["slot_of_expert"] = torch.where(where < case["S"], where, -1).to(torch.int32)
        s["y_pairs"] = _normal(gen, (T * k, H), DTYPES[case["dtype"]], 0.7)
        s["dy"] = _normal(gen, (T, H), DTYPES[case["dy"]], 0.02)
        s["dy_pairs"], s["dw"] = torch.zeros_like(s["y_pairs"]), torch.zeros((T, k), **f32)
        return s
    if op in ("losses", "route_bwd"):
        T, E, k, G = case["T"], case["E"], case["k"], case["segs"]
        spread = _normal(gen, (E,), torch.float32, 0.7)
        s["logits"] = _normal(gen, (T, E), torch.float32) + spread
        s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["bounds"] = _segments(case)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        if op == "losses":
            s["counts"] = torch.zeros((G, E), dtype=torch.int32, device="cuda")
            s["probs"], s["losses"] = torch.zeros((G, E), **f32), torch.zeros(2, **f32)
            if own:
                s["ws"] = torch.empty(Q.moe_balance_loss_workspace_size(T, E, G), dtype=torch.uint8, device="cuda")
            return s
        s["counts"] = torch.stack([torch.bincount(s["ids"][a:b].reshape(-1).long(), minlength=E)
                                   for a, b in zip(s["bounds"], s["bounds"][1:])]).to(torch.int32)
        s["dw"] = _normal(gen, (T, k), torch.float32, 0.02)
        s["dlosses"] = 0.01 * (1.0 + torch.rand(2, generator=gen, device="cuda"))
        s["dlogits"] = torch.zeros((T, E), dtype=DTYPES[case["out"]], device="cuda")
        return s
    d, N, S = DTYPES[case["dtype"]], case["N"], case["S"]
    s["route"] = r = _routing(case, gen)
    if op == "act_bwd":
        I = N // 2 if case["act"] == "swiglu" else N
        s["z"] = _normal(gen, (r["P"], N), d, 1.5) if case["act"] != "none" else None
        s["dy"] = _normal(gen, (r["P"], I), d, 0.02)
        s["dz"] = torch.zeros((r["P"], N), dtype=d, device="cuda") if case["act"] != "none" else None
        s["h"] = torch.zeros((r["P"], I), dtype=d, device="cuda") if case["h"] and case["act"] != "none" else None
        s["dbias"] = torch.zeros((S, N), **f32)
        if own:
            s["ws"] = torch.empty(max(1, Q.moe_expert_act_backward_workspace_size(S, N, r["P"])), dtype=torch.uint8,
                                  device="cuda")
        return s
    K, out = case["K"], DTYPES[case["out"]]
    width = N // 2 if case["act"] == "swiglu" else N
    s["w"] = _normal(gen, (S, N, K), d, K ** -0.5)
    s["x"] = _activations(gen, (_count(case, case["x_rows"]), K), d)
    s["bias"] = None if case["bias"] == "none" else _normal(gen, (S, N), DTYPES[case["bias"]], 0.3)
    ny = _count(case, case["y_rows"])
    s["residual"] = None if case["residual"] == "none" else _activations(gen, (ny, width), DTYPES[case["residual"]])
    s["y"] = torch.zeros((ny, width), dtype=out, device="cuda")
    s["z"] = torch.zeros((ny, N), dtype=d, device="cuda") if case["keep"] else None
    return s


# -------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


_ROOT = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "none":
        return z
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        return g * _sigmoid(g) * u
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_ROOT * (z + 0.044715 * z * z * z)))
    return torch.clamp(z, min=0.0)


def _act_grad(z, dy, act):
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        sg = _sigmoid(g)
        return torch.cat((dy * u * sg * (1.0 + g * (1.0 - sg)), dy * g * sg), dim=1)
    if act == "silu":
        sg = _sigmoid(z)
        return dy * sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(_ROOT * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _ROOT * (1.0 + 0.134145 * z * z))
    return torch.where(z > 0.0, dy, torch.zeros_like(dy))


def _probs(logits, score):
    """(p, 1 or 1 - s, log sum of exp): what the losses' gradients take of a row."""
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if score == "softmax":
        return e / total, 1.0, e / total, lse
    sg = _sigmoid(logits)
    return sg / sg.sum(1, keepdim=True), 1.0 - sg, e / total, lse


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "clip":
        total = 0.0
        for g in s["grads"]:
            v = g.float()
            total = total + (v * v).sum(dtype=torch.float64)
        total = c["scale"] * torch.sqrt(total)
        factor = (c["scale"] * torch.clamp(s["max_norm"] / (total + EPS), max=1.0)).float()
        outs = [(g.float() * factor).to(o.dtype) for g, o in zip(s["grads"], s["outs"])]
        return dict(total=total.float().reshape(1), outs=torch.cat(outs) if c["flat"] else outs)
    if op == "combine_bwd":
        T, k, H = c["T"], c["k"], c["H"]
        dy, yp = s["dy"].float().reshape(T, 1, H), s["y_pairs"].float().reshape(T, k, H)
        here = (s["slot_of_expert"][s["ids"].long()] >= 0).reshape(T, k, 1)
        dyp = torch.where(here, s["w"].reshape(T, k, 1) * dy, 0.0).to(s["y_pairs"].dtype).reshape(T * k, H)
        return dict(dy_pairs=dyp, dw=torch.where(here[..., 0], (yp * dy).sum(2), 0.0))
    if op in ("losses", "route_bwd"):
        T, E, k, b = c["T"], c["E"], c["k"], s["bounds"]
        p, slope, soft, lse = _probs(s["logits"], c["score"])
        n = b[-1] - b[0]
        if op == "losses":
            counts = torch.stack([torch.bincount(s["ids"][i:j].reshape(-1).long(), minlength=E)
                                  for i, j in zip(b, b[1:])]).to(torch.int32)
            probs = torch.stack([p[i:j].sum(0) / max(j - i, 1) for i, j in zip(b, b[1:])])
            losses = torch.stack(((counts.float() * probs).sum() * (E / (k * n)), (lse[b[0]:b[-1]] ** 2).sum() / n))
            return dict(counts=counts, probs=probs, losses=losses)
        ids = s["ids"].long()
        d = torch.zeros((T, E), dtype=torch.float32, device="cuda")
        if c["score"] == "softmax":
            q, own_slope = soft.gather(1, ids), 1.0
        else:
            q = _sigmoid(s["logits"]).gather(1, ids)
            own_slope = 1.0 - q
        if c["renorm"]:
            q = q / q.sum(1, keepdim=True)
            d.scatter_(1, ids, c["scale"] * own_slope * q * (s["dw"] - (q * s["dw"]).sum(1, keepdim=True)))
        else:
            d.scatter_(1, ids, c["scale"] * own_slope * q * s["dw"])
            if c["score"] == "softmax":
                d = d - c["scale"] * soft * (q * s["dw"]).sum(1, keepdim=True)
        if c["balance"]:
            for g, (i, j) in enumerate(zip(b, b[1:])):
                a = s["dlosses"][0] * (E / (k * n * max(j - i, 1))) * s["counts"][g].float()
                pg = p[i:j]
                d[i:j] += pg * (slope if c["score"] == "softmax" else slope[i:j]) * (a - (pg * a).sum(1, keepdim=True))
            d[b[0]:b[-1]] += s["dlosses"][1] * (2.0 / n) * lse[b[0]:b[-1]] * soft[b[0]:b[-1]]
        return dict(dlogits=d.to(s["dlogits"].dtype))
    r = s["route"]
    if op == "act_bwd":
        at = _rows(s, c["rows"])
        dy = s["dy"][at].float()
        out = {}
        dz = dy
        if c["act"] != "none":
            z = s["z"][at].float()
            dz = _act_grad(z, dy, c["act"])
            out["dz"] = torch.zeros_like(s["dz"])
            out["dz"][at] = dz.to(s["dz"].dtype)
            if s["h"] is not None:
                out["h"] = torch.zeros_like(s["h"])
                out["h"][at] = _act(z, c["act"]).to(s["h"].dtype)
        out["dbias"] = torch.zeros_like(s["dbias"])
        if r["slots"]:
            out["dbias"][r["slots"]] = torch.stack([v.sum(0) for v in dz.split(r["sizes"])])
        return out
    y = torch.zeros_like(s["y"])
    z_out = None if s["z"] is None else torch.zeros_like(s["z"])
    if r["slots"]:
        x = s["x"].float()[_rows(s, c["x_rows"])]
        parts = []
        for e, a in zip(r["slots"], x.split(r["sizes"])):
            v = a @ s["w"][e].float().t()
            parts.append(v if s["bias"] is None else v + s["bias"][e].float())
        z, at = torch.cat(parts), _rows(s, c["y_rows"])
        v = _act(z, c["act"])
        if s["residual"] is not None:
            v = v + s["residual"][at].float()
        y[at] = v.to(y.dtype)
        if z_out is not None:
            z_out[at] = z.to(z_out.dtype)
    return dict(y=y) if z_out is None else dict(y=y, z=z_out)


# -------------------------------------------------------- the library's calls

def _library(s):
    import quantized_routed_expert_moe_amd as Q
    c = s["case"]
    op = c["op"]
    score = Q.MOE_SCORE_SOFTMAX if c.get("score") == "softmax" else Q.MOE_SCORE_SIGMOID
    if op == "clip":
        Q.moe_grad_norm(s["grad_list"], s["total"], scale=c["scale"], ws=s["ws"])
        Q.moe_grad_clip(s["grad_list"], s["total"], s["max_norm"], eps=EPS, scale=c["scale"], outs=s["out_list"])
        return dict(total=s["total"], outs=s["flat"] if c["flat"] else s["outs"])
    if op == "combine_bwd":
        Q.moe_combine_backward(s["dy"], s["y_pairs"], s["ids"], s["w"], s["slot_of_expert"], c["S"], s["dy_pairs"], s["dw"])
        return dict(dy_pairs=s["dy_pairs"], dw=s["dw"])
    if op == "losses":
        Q.moe_balance_loss(s["logits"], s["ids"], score, s["counts"], s["probs"], s["losses"], s["offsets"], ws=s["ws"])
        return dict(counts=s["counts"], probs=s["probs"], losses=s["losses"])
    if op == "route_bwd":
        losses = (s["counts"], s["dlosses"], s["offsets"]) if c["balance"] else (None, None, None)
        Q.moe_route_backward(s["logits"], s["ids"], s["dw"], score, c["renorm"], c["scale"], *losses, s["dlogits"])
        return dict(dlogits=s["dlogits"])
    r = s["route"]
    how = {"position": Q.MOE_ROWS_POSITION, "pair": Q.MOE_ROWS_PAIR, "token": Q.MOE_ROWS_TOKEN}
    act = {"none": Q.MOE_ACT_NONE, "swiglu": Q.MOE_ACT_SWIGLU, "silu": Q.MOE_ACT_SILU, "gelu": Q.MOE_ACT_GELU,
           "gelu_tanh": Q.MOE_ACT_GELU_TANH, "relu": Q.MOE_ACT_RELU}[c["act"]]
    if op == "act_bwd":
        Q.moe_expert_act_backward(s["dy"], s["z"], r["offsets"], s["dz"], s["dbias"], r["perm"], how[c["rows"]], act,
                                  h=s["h"], ws=s["ws"])
        return {k: s[k] for k in ("dz", "h", "dbias") if s[k] is not None}
    Q.moe_expert_gemm_bias(s["x"], s["w"], s["bias"], s["residual"], r["offsets"], s["y"], r["perm"], r["k"],
                           how[c["x_rows"]], how[c["y_rows"]], act, z=s["z"])
    return dict(y=s["y"]) if s["z"] is None else dict(y=s["y"], z=s["z"])


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "clip":
        sizes, types = _sizes(case)
        bytes_ = sum(n * (BYTES[t] + BYTES["fp32" if case["out"] == "fp32" else t]) for n, t in zip(sizes, types))
        return dict(bytes=bytes_ + 4, flops=3 * sum(sizes))
    if op == "combine_bwd":
        T, k, H, b = case["T"], case["k"], case["H"], BYTES[case["dtype"]]
        share = case["S"] / case["E"]
        return dict(bytes=int(T * k * H * b * (1 + share)) + T * H * BYTES[case["dy"]] + 12 * T * k,
                    flops=int(3 * T * k * H * share))
    if op in ("losses", "route_bwd"):
        T, E, k, G = case["T"], case["E"], case["k"], case["segs"]
        if op == "losses":
            n = _segments(case)[-1]
            return dict(bytes=4 * n * (E + k) + 8 * G * E + 8, flops=6 * n * E)
        return dict(bytes=T * E * (4 + BYTES[case["out"]]) + 8 * T * k + (4 * G * E if case["balance"] else 0),
                    flops=10 * T * E)
    P = case["T"] * max(case["k"], 1)
    R = P if case["S"] == case["E"] else P * case["S"] // case["E"]  # the other experts' pairs are not on the card
    N, b = case["N"], BYTES[case["dtype"]]
    I = N // 2 if case["act"] == "swiglu" else N
    if op == "act_bwd":
        per = I + (2 * N if case["act"] != "none" else 0) + (I if case["h"] and case["act"] != "none" else 0)
        return dict(bytes=R * per * b + case["S"] * N * 4, flops=R * N * 6)
    K = case["K"]
    used = case["S"] * (1.0 - (1.0 - min(1.0, case["k"] / case["E"])) ** case["T"]) if case["k"] else 1
    moved = used * N * K * b + min(R, _count(case, case["x_rows"])) * K * b + R * I * BYTES[case["out"]]
    moved += used * N * BYTES.get(case["bias"], 0) + R * I * BYTES.get(case["residual"], 0) + (R * N * b if case["keep"] else 0)
    return dict(bytes=int(moved), flops=2 * R * N * K)


# -------------------------------------------------------- the definition in 64 bits

def _exact_router(case, s):
    D = torch.float64
    T, E, k = case["T"], case["E"], case["k"]
    bounds = s["offsets"].cpu().tolist()
    n = bounds[-1] - bounds[0]
    l, ids = s["logits"].to(D), s["ids"].long()
    soft, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
    gate = torch.sigmoid(l)
    p = soft if case["score"] == "softmax" else gate / gate.sum(1, keepdim=True)
    member = torch.zeros((T, E), dtype=D, device="cuda").scatter_add_(1, ids, torch.ones(ids.shape, dtype=D, device="cuda"))
    if case["op"] == "losses":
        G = case["segs"]
        counts, probs = torch.zeros((G, E), dtype=D, device="cuda"), torch.zeros((G, E), dtype=D, device="cuda")
        for g in range(G):
            a, b = bounds[g], bounds[g + 1]
            if b > a:
                counts[g], probs[g] = member[a:b].sum(0), p[a:b].mean(0)
        balance = (E / (k * n)) * (counts * probs).sum()
        return dict(counts=counts.to(torch.int32), probs=probs,
                    losses=torch.stack((balance, lse[bounds[0]:bounds[-1]].square().sum() / n)))
    # the scores' gradient first, then back through the score
    ds = torch.zeros((T, E), dtype=D, device="cuda")
    dw = s["dw"].to(D) * case["scale"]
    score = soft if case["score"] == "softmax" else gate
    picked = score.gather(1, ids)
    if case["renorm"]:
        total = picked.sum(1, keepdim=True)
        ds.scatter_(1, ids, dw / total - (dw * picked).sum(1, keepdim=True) / total ** 2)
    else:
        ds.scatter_(1, ids, dw)
    if case["balance"]:
        dp = torch.zeros((T, E), dtype=D, device="cuda")
        for g in range(case["segs"]):
            a, b = bounds[g], bounds[g + 1]
            if b > a:
                dp[a:b] = s["dlosses"][0].to(D) * E / (k * n) * s["counts"][g].to(D) / (b - a)
        if case["score"] == "softmax":
            ds = ds + dp
        else:
            total = gate.sum(1, keepdim=True)
            ds = ds + (dp - (dp * p).sum(1, keepdim=True)) / total
    if case["score"] == "softmax":
        d = soft * (ds - (soft * ds).sum(1, keepdim=True))
    else:
        d = ds * gate * (1 - gate)
    if case["balance"]:
        inside = slice(bounds[0], bounds[-1])
        d[inside] += s["dlosses"][1].to(D) * 2 / n * lse[inside].unsqueeze(1) * soft[inside]
    return dict(dlogits=d)


def _exact_act(z, act):
    if act == "swiglu":
        half = z.shape[1] // 2
        return torch.sigmoid(z[:, :half]) * z[:, :half] * z[:, half:]
    if act == "silu":
        return torch.sigmoid(z) * z
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return torch.relu(z) if act == "relu" else z


def exact(case, seed):
    s = prepare(case, seed)
    D, op = torch.float64, case["op"]
    if op == "clip":
        norm = case["scale"] * math.sqrt(sum(float(g.to(D).square().sum()) for g in s["grads"]))
        factor = case["scale"] * min(1.0, s["max_norm"] / (norm + EPS))
        outs = [g.to(D) * factor for g in s["grads"]]
        return dict(total=torch.tensor([norm], dtype=D), outs=torch.cat(outs) if case["flat"] else outs)
    if op == "combine_bwd":
        T, k = case["T"], case["k"]
        here = torch.zeros((T, k), dtype=torch.bool, device="cuda")
        for e in range(case["E"]):
            if int(s["slot_of_expert"][e]) >= 0:
                here |= s["ids"] == e
        dyp, dw = torch.zeros_like(s["y_pairs"], dtype=D), torch.zeros((T, k), dtype=D, device="cuda")
        dy = s["dy"].to(D)
        for j in range(k):
            rows = here[:, j].to(D)
            dyp[j::k] = dy * (s["w"][:, j].to(D) * rows).unsqueeze(1)
            dw[:, j] = (s["y_pairs"][j::k].to(D) * dy).sum(1) * rows
        return dict(dy_pairs=dyp, dw=dw)
    if op in ("losses", "route_bwd"):
        return _exact_router(case, s)
    offsets = s["route"]["offsets"].cpu().tolist()
    if op == "act_bwd":
        P = s["dy"].shape[0]
        dz, db = torch.zeros((P, case["N"]), dtype=D, device="cuda"), torch.zeros((case["S"], case["N"]), dtype=D, device="cuda")
        h = torch.zeros_like(s["dy"], dtype=D)
        at = _rows(s, case["rows"])
        for e in range(case["S"]):
            if offsets[e + 1] == offsets[e]:
                continue
            i = at[offsets[e]:offsets[e + 1]]
            dy = s["dy"][i].to(D)
            if case["act"] == "none":
                db[e] = dy.sum(0)
                continue
            with torch.enable_grad():
                z = s["z"][i].to(D).requires_grad_()
                v = _exact_act(z, case["act"])
                dz[i] = torch.autograd.grad(v, z, dy)[0]
            h[i] = v.detach()
            db[e] = dz[i].sum(0)
        out = {} if case["act"] == "none" else dict(dz=dz)
        if s["h"] is not None:
            out["h"] = h
        return dict(out, dbias=db)
    y, z_out = torch.zeros_like(s["y"], dtype=D), None if s["z"] is None else torch.zeros_like(s["z"], dtype=D)
    ix, iy = _rows(s, case["x_rows"]), _rows(s, case["y_rows"])
    for e in range(case["S"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        z = torch.mm(s["x"][ix[a:b]].to(D), s["w"][e].to(D).t().contiguous())
        if s["bias"] is not None:
            z = z + s["bias"][e].to(D)
        v = _exact_act(z, case["act"])
        y[iy[a:b]] = v if s["residual"] is None else v + s["residual"][iy[a:b]].to(D)
        if z_out is not None:
            z_out[iy[a:b]] = z
    return dict(y=y) if z_out is None else dict(y=y, z=z_out)
