"""Streamed products of batches in which one slot holds most of the rows: its
rows go to several workgroups, each row's result as in even batches."""
import pytest
import torch

import quantized_routed_expert_moe_amd as Q
from tests import test_gpu_expert_w4 as w4
from tests.expert_util import batches
from tests.test_gpu_expert_gemm import run_product

pytestmark = pytest.mark.gpu

POS, PAIR, TOKEN = Q.MOE_ROWS_POSITION, Q.MOE_ROWS_PAIR, Q.MOE_ROWS_TOKEN
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def skewed(slots, hot, others, seed):
    """`hot` maps slots to their rows; `others` rows fall on slots at random."""
    sizes = torch.bincount(torch.randint(0, slots, (others,), generator=torch.Generator().manual_seed(seed)),
                           minlength=slots).tolist()
    for s, n in hot.items():
        sizes[s] = n
    return sizes


CASES = [skewed(20, {7: 200}, 15, 0), skewed(20, {0: 129, 19: 64, 5: 65, 6: 0}, 9, 1), skewed(40, {39: 300}, 60, 2),
         skewed(1000, {3: 177, 640: 33, 999: 48}, 40, 3), skewed(130, {64: 257, 63: 17, 65: 16}, 100, 4)]


@pytest.mark.parametrize("sizes", CASES)
@pytest.mark.parametrize("N,K,act", [(64, 136, 0), (264, 200, 0), (160, 264, 1)])
def test_streamed_product(sizes, N, K, act):
    if len(sizes) > 500 and N > 64:
        N = 64
    run_product(sizes, N, K, BF, F32, k=2, P=sum(sizes) + 2, x_rows=TOKEN, y_rows=PAIR, act=act, seed=K)


@pytest.mark.parametrize("sizes", CASES)
@pytest.mark.parametrize("group,dtype", [(32, BF), (64, HF), (128, BF)])
@pytest.mark.parametrize("act", [0, 1])
def test_4_bit_product(sizes, group, dtype, act):
    w4.run(sizes, 48, 256, group, dtype, F32, scale_dtype=F32 if act else None, k=2, P=sum(sizes) + 2, x_rows=PAIR,
           y_rows=POS, act=act, seed=group)


def test_rows_do_not_depend_on_the_other_slots():
    """A slot's rows give the same bits alone as beside a slot of many rows (one pass of 16 rows in both)."""
    S, N, K, group = 64, 96, 256, 64
    sizes = skewed(S, {9: 400}, 500, 5)
    P = sum(sizes)
    off, _ = batches(sizes, P, 1, 0)
    q, sc, z = w4.weights(S, N, K, group, BF, True, 1)
    x = torch.randn((P, K), generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    y = torch.empty((P, N), device="cuda")
    Q.moe_expert_gemv_w4(x, q.cuda(), sc.cuda(), z.cuda(), group, off.cuda(), y)
    for s in (0, 9, 10, 63):
        a, b = int(off[s]), min(int(off[s + 1]), int(off[s]) + 16)
        one = torch.empty((b - a, N), device="cuda")
        Q.moe_expert_gemv_w4(x[a:b].contiguous(), q[s:s + 1].cuda(), sc[s:s + 1].cuda(), z[s:s + 1].cuda(), group, None, one)
        assert torch.equal(one, y[a:b])


@pytest.mark.parametrize("group", [32, 128])
def test_more_blocks_of_rows_than_workgroups(group):
    """One matrix and 1.15 million rows (and as many in the last of three slots): rows repeat, and so must results."""
    R, N, K = 1_150_000, 32, 128
    q, sc, z = (t.cuda() for t in w4.weights(3, N, K, group, BF, True, 3))
    few = torch.randn((251, K), generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    at = torch.arange(R, device="cuda") % 251
    x, y, want = few[at], torch.full((R, N), 7.0, device="cuda"), torch.empty((251, N), device="cuda")
    Q.moe_expert_gemv_w4(few, q[2:], sc[2:], z[2:], group, None, want)
    Q.moe_expert_gemv_w4(x, q[2:], sc[2:], z[2:], group, None, y)
    assert torch.equal(y, want[at])
    off = torch.tensor([0, 1, 5, R], dtype=torch.int32, device="cuda")
    y.fill_(7.0)
    Q.moe_expert_gemv_w4(x, q, sc, z, group, off, y)
    assert torch.equal(y[5:], want[at[5:]])


def test_captured_calls_follow_the_offsets():
    """One graph of a product, a 4-bit product and a weight gradient, replayed over batches that are even, in one slot,
    nearly empty and empty: each replay equals the eager calls."""
    S, N, K, group, P = 24, 72, 256, 64, 400
    g = torch.Generator().manual_seed(6)
    x, dy = (torch.randn((P, n), generator=g).to(BF).cuda() for n in (K, N))
    w = torch.randn((S, N, K), generator=g).to(BF).cuda()
    q, sc, z = (t.cuda() for t in w4.weights(S, N, K, group, BF, True, 7))
    off, out = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), {}
    out["y"], out["y4"] = (torch.zeros((P, N), device="cuda") for _ in range(2))
    out["dw"] = torch.zeros((S, N, K), dtype=BF, device="cuda")
    ws = torch.empty(max(1, Q.moe_expert_gemm_wgrad_workspace_size(S, N, K, P)), dtype=torch.uint8, device="cuda")

    def calls():
        Q.moe_expert_gemm(x, w, off, out["y"])
        Q.moe_expert_gemv_w4(x, q, sc, z, group, off, out["y4"])
        Q.moe_expert_gemm_wgrad(dy, x, off, out["dw"], ws=ws)

    sizes = [[16] * 24 + [0], [0] * 11 + [400] + [0] * 12, [0] * 5 + [2] + [0] * 18, [0] * 24, skewed(24, {3: 250}, 100, 8)]
    starts = [torch.tensor([0] + s[:24]).cumsum(0).to(torch.int32) for s in sizes]
    want = []
    for o in starts:
        off.copy_(o)
        for v in out.values():
            v.fill_(7.0)
        calls()
        want.append([v.clone() for v in out.values()])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        calls()
    for _ in range(2):
        for o, expected in zip(starts, want):
            off.copy_(o)
            for v in out.values():
                v.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(v, e) for v, e in zip(out.values(), expected))
            (out["y"] * 2).sum()  # eager work of the program between replays
