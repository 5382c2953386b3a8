"""The operators together, as a block runs them: norm, routing, expert
products, SwiGLU, combine, residual and norm; a training step's gradients
through it; streams and captured graphs."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D, silu, w4_matrix

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


class Block:
    """One block's buffers and calls: x -> x + experts(norm(x)), and the next block's normed input."""

    def __init__(self, T, H, I, E, S, k, w4=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.H, self.I, self.E, self.S, self.k, self.w4 = T, H, I, E, S, k, w4
        P = T * k

        def n(shape, scale, dtype=BF, base=0.0):
            return (base + scale * torch.randn(shape, generator=g)).to(dtype).cuda()

        self.x = n((T, H), 1.0)
        self.w_in, self.w_next, self.gate = n((H,), 0.1, F32, 1.0), n((H,), 0.1, F32, 1.0), n((H,), 0.1, F32, 0.5)
        self.w_post = n((H,), 0.1, F32, 1.0)
        self.router = n((1, E, H), H ** -0.5)
        if w4:
            self.group = 64
            self.q1 = torch.randint(0, 256, (S, 2 * I, H // 2), generator=g, dtype=torch.uint8).cuda()
            self.q2 = torch.randint(0, 256, (S, H, I // 2), generator=g, dtype=torch.uint8).cuda()
            self.s1 = n((S, 2 * I, H // 64), 0.01, BF, 0.04 * (256 / H) ** 0.5)
            self.s2 = n((S, H, I // 64), 0.01, BF, 0.04 * (256 / I) ** 0.5)
        else:
            self.w1, self.w2 = n((S, 2 * I, H), H ** -0.5), n((S, H, I), I ** -0.5)
        i = dict(dtype=torch.int32, device="cuda")
        self.soe = torch.arange(E, **i)
        self.soe[S:] = -1
        self.h = torch.zeros((T, H), dtype=BF, device="cuda")
        self.logits = torch.zeros((T, E), device="cuda")
        self.ids, self.tw = torch.zeros((T, k), **i), torch.zeros((T, k), device="cuda")
        self.off, self.act, self.na = torch.zeros(S + 1, **i), torch.zeros(min(S, P), **i), torch.zeros(1, **i)
        self.perm = torch.zeros(P, **i)
        self.ht, self.he, self.hc = torch.zeros(P, **i), torch.zeros(P, **i), torch.zeros(1, **i)
        self.hw = torch.zeros(P, device="cuda")
        ws = Q.moe_batches_workspace_size(T, k, E, S)
        self.bws = torch.zeros(max(ws, 1), dtype=torch.uint8, device="cuda")
        self.mid = torch.zeros((P, I), dtype=BF, device="cuda")
        self.pairs = torch.zeros((P, H), device="cuda")
        self.y = torch.zeros((T, H), device="cuda")
        self.x_out, self.h_next = torch.zeros_like(self.x), torch.zeros_like(self.x)

    def route(self, stream=None):
        Q.moe_block_norm(self.x, None, None, None, self.w_in, None, self.h, EPS, stream=stream)
        Q.moe_expert_gemm(self.h, self.router, None, self.logits, stream=stream)
        Q.moe_route_and_batch(self.logits, self.k, Q.MOE_SCORE_SOFTMAX, True, 1.0, self.ids, self.tw, self.E, self.soe,
                              self.S, self.off, self.act, self.na, self.perm, self.ht, self.he, self.hw, self.hc,
                              self.bws, stream)

    def forward(self, stream=None):
        self.route(stream)
        rows = dict(perm_pair=self.perm, k=self.k, stream=stream)
        up = dict(x_rows=Q.MOE_ROWS_TOKEN, act=Q.MOE_ACT_SWIGLU, **rows)
        down = dict(y_rows=Q.MOE_ROWS_PAIR, **rows)
        if self.w4:
            Q.moe_expert_gemv_w4(self.h, self.q1, self.s1, None, self.group, self.off, self.mid, **up)
            Q.moe_expert_gemv_w4(self.mid, self.q2, self.s2, None, self.group, self.off, self.pairs, **down)
        else:
            Q.moe_expert_gemm(self.h, self.w1, self.off, self.mid, **up)
            Q.moe_expert_gemm(self.mid, self.w2, self.off, self.pairs, **down)
        Q.moe_combine(self.pairs, self.ids, self.tw, self.soe, self.S, None, self.y, stream)
        Q.moe_block_norm(self.x, self.y, self.w_post, self.gate, self.w_next, self.x_out, self.h_next, EPS,
                         stream=stream)
        return self.x_out, self.h_next

    def plain(self):
        """The block in 64 bits from its stored tensors (routing taken from the device's ids)."""
        x = self.x.to(D)
        h = (x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * self.w_in.to(D)).to(BF).to(D)
        logits = h @ self.router[0].to(D).t()
        top = torch.topk(logits, self.k, dim=1)
        wt = torch.softmax(top.values, 1)
        if self.w4:
            w1, w2 = w4_matrix(self.q1, self.s1, None, 64), w4_matrix(self.q2, self.s2, None, 64)
        else:
            w1, w2 = self.w1.to(D), self.w2.to(D)
        y = torch.zeros((self.T, self.H), dtype=D, device="cuda")
        for t in range(self.T):
            for j in range(self.k):
                e = int(top.indices[t, j])
                if e < self.S:
                    gu = w1[e] @ h[t]
                    m = (silu(gu[:self.I]) * gu[self.I:]).to(BF).to(D)
                    y[t] += wt[t, j] * (w2[e] @ m)
        r = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * self.w_post.to(D)
        xo = x + self.gate.to(D) * r
        return top.indices, xo, xo / torch.sqrt((xo * xo).mean(1, keepdim=True) + EPS) * self.w_next.to(D)


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("T,H,I,E,S,k", [(1, 256, 128, 8, 8, 2), (6, 512, 256, 16, 12, 4), (150, 256, 192, 8, 6, 2)])
def test_block_forward(T, H, I, E, S, k, w4):
    b = Block(T, H, I, E, S, k, w4, seed=T)
    x_out, h_next = b.forward()
    ids, xo, h = b.plain()
    assert torch.equal(b.ids.long(), ids), "routing differs (the inputs leave no near ties)"
    # one bf16 rounding in h and one in the activation stand in both; a value
    # of either may round the other way (a whole step, 2^-7 of it), which moves
    # y by a random share of its terms, and the outputs round once more
    for got, want in ((x_out, xo), (h_next, h)):
        err, big = (got.to(D) - want).abs(), want.abs().amax(1, keepdim=True)
        assert (err <= 2.0 ** -8 * want.abs() * 1.02 + 2.0 ** -7 * big).all(), float((err / big).max())


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("T", [2, 130])
def test_captured_block_replays_equal_the_eager_call(T, w4):
    b = Block(T, 256, 192, 8, 6, 2, w4)
    inputs = [torch.randn((T, 256), device="cuda").to(BF) for _ in range(4)]
    want = []
    for v in inputs:
        b.x.copy_(v)
        want.append([t.clone() for t in b.forward()])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.forward()
    for _ in range(2):
        for v, (xo, h) in zip(inputs, want):
            b.x.copy_(v)
            b.x_out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(b.x_out, xo) and torch.equal(b.h_next, h)
            (xo.float() * 2).sum()  # eager work of the program between replays


def test_two_blocks_on_two_streams():
    blocks = [Block(130, 256, 192, 8, 6, 2, seed=s) for s in (1, 2)]
    want = []
    for b in blocks:
        want.append([t.clone() for t in b.forward()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for b in blocks:
            b.x_out.zero_()
        torch.cuda.synchronize()
        for b, s in zip(blocks, streams):
            b.forward(s)
        torch.cuda.synchronize()
        for b, (xo, h) in zip(blocks, want):
            assert torch.equal(b.x_out, xo) and torch.equal(b.h_next, h)


def test_training_step_gradients():
    """Gradients of sum(c * y_pairs) through down product, SwiGLU and gate/up
    product, for x's pairs and both weight pools, against 64 bits."""
    T, H, I, E, S, k = 60, 136, 72, 8, 6, 2
    b = Block(T, H, I, E, S, k, seed=3)
    b.route()
    P, rows = T * k, dict(perm_pair=b.perm, k=k)
    POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
    gu, h = torch.zeros((P, 2 * I), dtype=BF, device="cuda"), torch.zeros((P, I), dtype=BF, device="cuda")
    Q.moe_expert_gemm(b.h, b.w1, b.off, gu, x_rows=TOKEN, **rows)
    Q.moe_swiglu(gu, h, b.off)
    dy = torch.randn((P, H), device="cuda").to(BF)  # per pair
    dh, dgu, h2 = torch.zeros_like(h), torch.zeros_like(gu), torch.zeros_like(h)
    Q.moe_expert_gemm(dy, b.w2, b.off, dh, x_rows=PAIR, transpose=True, **rows)
    Q.moe_swiglu_backward(gu, dh, dgu, h2, b.off)
    dx = torch.zeros((P, H), device="cuda")
    Q.moe_expert_gemm(dgu, b.w1, b.off, dx, y_rows=PAIR, transpose=True, **rows)
    dw1, dw2 = torch.empty((S, 2 * I, H), device="cuda"), torch.empty((S, H, I), device="cuda")
    ws = [torch.empty(max(1, Q.moe_expert_gemm_wgrad_workspace_size(*d.shape, P)), dtype=torch.uint8, device="cuda")
          for d in (dw1, dw2)]
    Q.moe_expert_gemm_wgrad(dgu, b.h, b.off, dw1, dy_rows=POS, x_rows=TOKEN, ws=ws[0], **rows)
    Q.moe_expert_gemm_wgrad(dy, h2, b.off, dw2, dy_rows=PAIR, x_rows=POS, ws=ws[1], **rows)
    assert torch.equal(h, h2)

    x = b.h.to(D)[torch.arange(P, device="cuda") // k].requires_grad_()  # a row for each pair
    w1, w2 = b.w1.to(D).requires_grad_(), b.w2.to(D).requires_grad_()
    e = b.ids.reshape(-1).long()
    loss = torch.zeros((), dtype=D, device="cuda")
    for s in range(S):
        p = (e == s).nonzero().flatten()
        v = x[p] @ w1[s].t()
        loss = loss + ((silu(v[:, :I]) * v[:, I:]) @ w2[s].t() * dy[p].to(D)).sum()
    gx, g1, g2 = torch.autograd.grad(loss, (x, w1, w2))
    # gu, h, dh and dgu are rounded to bf16 on the way (half a step, 2^-8, of
    # each): in the 2-norm at most 4 * 2^-8 of the gradient together
    for got, want in ((dx, gx), (dw1, g1), (dw2, g2)):
        assert float((got.to(D) - want).norm() / want.norm()) <= 4 * 2.0 ** -8
