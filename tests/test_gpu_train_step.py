"""A training step of a routed block through the library's calls, as a program makes them: gate with bias, routing and its
losses, experts with biases and SwiGLU, combine, output projection added to the residual stream; then every gradient, and
their norm and clipping.  Against autograd in 64 bits, captured and replayed over new inputs, and on two streams at once."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests.expert_util import D
from tests.train_util import act, losses, rand

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PAIR, TOKEN = Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
SWI = Q.MOE_ACT_SWIGLU
T, H, I, E, K, G = 90, 64, 48, 16, 4, 3
P = T * K
BALANCE, ZLOSS, MAX_NORM = 0.05, 0.01, 0.7


class Step:
    """Weights, inputs and every buffer of one step."""

    def __init__(self, seed, score):
        dev = lambda t: t.cuda()
        self.score, self.renorm, self.scale = score, score == Q.MOE_SCORE_SIGMOID, 1.5
        self.x, self.dout = dev(rand((T, H), BF, seed)), dev(rand((T, H), BF, seed + 1))
        w = lambda s, i, scale: dev(rand(s, BF, seed + i, scale))
        b = lambda s, i: dev(rand(s, F32, seed + i, 0.2))
        self.wg, self.bg = w((1, E, H), 2, H ** -0.5), b((1, E), 3)
        self.w1, self.b1 = w((E, 2 * I, H), 4, H ** -0.5), b((E, 2 * I), 5)
        self.w2, self.b2 = w((E, H, I), 6, I ** -0.5), b((E, H), 7)
        self.wo, self.bo = w((1, H, H), 8, H ** -0.5), b((1, H), 9)
        self.bounds = [0, 40, 40, 80]  # an empty sequence, ten rows of padding
        e = lambda s, t=F32: torch.zeros(s, dtype=t, device="cuda")
        self.seqs = torch.tensor(self.bounds, dtype=I32, device="cuda")
        self.soe = torch.arange(E, dtype=I32, device="cuda")
        self.logits, self.ids, self.topw = e((T, E)), e((T, K), I32), e((T, K))
        self.off, self.active, self.n, self.perm = e(E + 1, I32), e(E, I32), e(1, I32), e(P, I32)
        self.host = (e(P, I32), e(P, I32), e(P), e(1, I32))
        self.counts, self.probs, self.losses = e((G, E), I32), e((G, E)), e(2)
        self.z, self.h, self.pairs, self.y = e((P, 2 * I), BF), e((P, I), BF), e((P, H), BF), e((T, H), BF)
        self.out = e((T, H), BF)
        self.dlosses = torch.tensor([BALANCE, ZLOSS], device="cuda")
        self.dy, self.dpairs, self.dw = e((T, H), BF), e((P, H), BF), e((T, K))
        self.dh, self.dz, self.dxp, self.dlogits, self.dxg = e((P, I), BF), e((P, 2 * I), BF), e((P, H), BF), e((T, E), BF), e((T, H), BF)
        self.dx, self.ones = e((T, H)), torch.ones((T, K), device="cuda")
        self.gates = e((T, H))
        self.grads = dict(wg=e((1, E, H)), bg=e((1, E)), w1=e((E, 2 * I, H)), b1=e((E, 2 * I)), w2=e((E, H, I)), b2=e((E, H)),
                          wo=e((1, H, H)), bo=e((1, H)))
        self.clipped = [torch.zeros_like(g, dtype=BF) for g in self.grads.values()]
        self.list, self.outs = Q.moe_tensor_list(self.grads.values()), Q.moe_tensor_list(self.clipped)
        self.total = e(1)
        size = max(Q.moe_batches_workspace_size(T, K, E, E), Q.moe_balance_loss_workspace_size(T, E, G),
                   Q.moe_grad_norm_workspace_size(8), Q.moe_expert_gemm_wgrad_workspace_size(1, H, H, T),
                   Q.moe_expert_gemm_wgrad_workspace_size(E, 2 * I, H, P), Q.moe_expert_act_backward_workspace_size(E, 2 * I, P),
                   Q.moe_expert_act_backward_workspace_size(1, H, T), Q.moe_expert_act_backward_workspace_size(1, E, T))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")  # every call of the step, one after another

    def run(self):
        s, g = self, self.grads
        # forward
        Q.moe_expert_gemm_bias(s.x, s.wg, s.bg, None, None, s.logits)
        Q.moe_route_and_batch(s.logits, K, s.score, s.renorm, s.scale, s.ids, s.topw, E, s.soe, E, s.off, s.active, s.n, s.perm,
                              *s.host, s.ws)
        Q.moe_balance_loss(s.logits, s.ids, s.score, s.counts, s.probs, s.losses, s.seqs, ws=s.ws)
        Q.moe_expert_gemm_bias(s.x, s.w1, s.b1, None, s.off, s.h, s.perm, K, x_rows=TOKEN, act=SWI, z=s.z)
        Q.moe_expert_gemm_bias(s.h, s.w2, s.b2, None, s.off, s.pairs, s.perm, K, y_rows=PAIR)
        Q.moe_combine(s.pairs, s.ids, s.topw, s.soe, E, None, s.y)
        Q.moe_expert_gemm_bias(s.y, s.wo, s.bo, s.x, None, s.out)
        # backward
        Q.moe_expert_act_backward(s.dout, None, None, None, g["bo"], ws=s.ws)
        Q.moe_expert_gemm_wgrad(s.dout, s.y, None, g["wo"], ws=s.ws)
        Q.moe_expert_gemm(s.dout, s.wo, None, s.dy, transpose=True)
        Q.moe_combine_backward(s.dy, s.pairs, s.ids, s.topw, s.soe, E, s.dpairs, s.dw)
        Q.moe_expert_act_backward(s.dpairs, None, s.off, None, g["b2"], s.perm, PAIR, ws=s.ws)
        Q.moe_expert_gemm(s.dpairs, s.w2, s.off, s.dh, s.perm, K, x_rows=PAIR, transpose=True)
        Q.moe_expert_act_backward(s.dh, s.z, s.off, s.dz, g["b1"], s.perm, act=SWI, h=s.h, ws=s.ws)
        Q.moe_expert_gemm_wgrad(s.dpairs, s.h, s.off, g["w2"], s.perm, K, dy_rows=PAIR, ws=s.ws)
        Q.moe_expert_gemm_wgrad(s.dz, s.x, s.off, g["w1"], s.perm, K, x_rows=TOKEN, ws=s.ws)
        Q.moe_expert_gemm(s.dz, s.w1, s.off, s.dxp, s.perm, K, y_rows=PAIR, transpose=True)
        Q.moe_route_backward(s.logits, s.ids, s.dw, s.score, s.renorm, s.scale, s.counts, s.dlosses, s.seqs, s.dlogits)
        Q.moe_expert_act_backward(s.dlogits, None, None, None, g["bg"], ws=s.ws)
        Q.moe_expert_gemm_wgrad(s.dlogits, s.x, None, g["wg"], ws=s.ws)
        Q.moe_expert_gemm(s.dlogits, s.wg, None, s.gates, transpose=True)
        Q.moe_combine(s.dxp, s.ids, s.ones, s.soe, E, s.gates, s.dx)  # the sum over a token's pairs, and the gate's part
        Q.moe_grad_norm(s.list, s.total, ws=s.ws)
        Q.moe_grad_clip(s.list, s.total, MAX_NORM, outs=s.outs)

    def results(self):
        return [self.out, self.counts, self.probs, self.losses, self.dx, self.total, *self.grads.values(), *self.clipped]


def reference(s):
    """(outputs, losses, dx, gradients) by autograd in 64 bits, with the step's own experts."""
    d = lambda t: t.cpu().to(D).requires_grad_()
    x, wg, bg, w1, b1, w2, b2, wo, bo = (d(t) for t in (s.x, s.wg, s.bg, s.w1, s.b1, s.w2, s.b2, s.wo, s.bo))
    ids = s.ids.cpu().long()
    l = x @ wg[0].t() + bg[0]
    p = torch.softmax(l, 1) if s.score == Q.MOE_SCORE_SOFTMAX else torch.sigmoid(l)
    w = p.gather(1, ids)
    w = s.scale * (w / w.sum(1, keepdim=True) if s.renorm else w)
    y = torch.zeros((T, H), dtype=D)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = act(x[t] @ w1[e].t() + b1[e], SWI)
        y = y.index_add(0, t, w[t, j].unsqueeze(1) * (h @ w2[e].t() + b2[e]))
    out = y @ wo[0].t() + bo[0] + x
    counts, probs, balance, z = losses(l, s.ids.cpu(), s.score, s.bounds)
    total = (out * s.dout.cpu().to(D)).sum() + BALANCE * balance + ZLOSS * z
    leaves = (x, wg, bg, w1, b1, w2, b2, wo, bo)
    return out.detach(), counts, probs.detach(), torch.stack((balance, z)).detach(), torch.autograd.grad(total, leaves)


def near(got, want, roundings, what):
    """Norm of the difference against the norm: so many roundings to bf16 (half a step each, 2^-8) on the way."""
    off = float((got.cpu().to(D) - want).norm() / want.norm())
    assert off <= roundings * 2.0 ** -8, f"{what}: {off:.2e}"


@pytest.mark.parametrize("score", [Q.MOE_SCORE_SOFTMAX, Q.MOE_SCORE_SIGMOID])
def test_step_against_autograd(score):
    s = Step(3, score)
    s.run()
    out, counts, probs, loss, grads = reference(s)
    assert torch.equal(s.counts.cpu().to(D), counts)
    near(s.probs, probs, 0.01, "probs")  # fp32 all the way from the gate's sums
    near(s.losses, loss, 0.01, "losses")
    near(s.out, out, 4, "out")  # h, pairs, y, out
    dx = grads[0] - s.dout.cpu().to(D)  # what the residual hands through is the caller's sum
    # of the longest way: h, pairs, y | dy, dpairs, dh, dz (with z), dxp, dlogits: nine roundings
    near(s.dx, dx, 9, "dx")
    for (name, g), want in zip(s.grads.items(), grads[1:]):
        near(g, want, 8, name)
    total = torch.sqrt(sum((g.cpu().to(D) ** 2).sum() for g in s.grads.values()))
    assert abs(float(s.total) - float(total)) <= 2.0 ** -23 * float(total)
    for c, g in zip(s.clipped, s.grads.values()):
        near(c, g.cpu().to(D) * min(1.0, MAX_NORM / (float(total) + 1e-6)), 1, "clipped")


def test_captured_step_follows_its_inputs():
    s = Step(11, Q.MOE_SCORE_SIGMOID)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (20, 30, 40):
        s.x.copy_(rand((T, H), BF, seed))
        s.dout.copy_(rand((T, H), BF, seed + 1))
        s.seqs.copy_(torch.tensor([0, seed, 60, 90 - seed // 2], dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in s.results()]
        for t in s.results():
            t.zero_()
        s.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, s.results()))


def test_two_steps_on_two_streams():
    """Each with its own buffers and workspace: the results of either are those of the step alone."""
    steps = [Step(50, Q.MOE_SCORE_SIGMOID), Step(60, Q.MOE_SCORE_SOFTMAX)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.results()])
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
