"""The biased products, the activations' gradients, the router's losses and gradient, the combine's gradient and the
gradient norm without a GPU: every refusal of the C ABI names its argument before anything is enqueued, and workspace
queries answer 0 out of range."""
import ctypes

import pytest

import quantized_routed_expert_moe_amd as Q

FAKE = 1 << 20  # aligned non-null address; never dereferenced on these paths
INV, UNS, WSS = Q.MOE_ERR_INVALID_ARGUMENT, Q.MOE_ERR_UNSUPPORTED, Q.MOE_ERR_WORKSPACE_TOO_SMALL
f32 = ctypes.c_float


def _call(name, *args):
    st = getattr(Q.lib(), name)(*args)
    return st, Q.lib().moe_last_error().decode()


def _refused(got, want, needle):
    assert got[0] == want and needle in got[1], got


def _bias(**kw):
    a = dict(x=FAKE, dtype=Q.MOE_BF16, w=FAKE, stride=64 * 128 * 2, S=4, N=64, K=128, bias=FAKE, bt=Q.MOE_F32,
             res=FAKE * 3, rt=Q.MOE_BF16, off=FAKE, R=8, perm=FAKE, k=2, xr=0, yr=0, act=0, y=FAKE * 2, yt=Q.MOE_BF16,
             z=FAKE * 4)
    a.update(kw)
    return _call("moe_expert_gemm_bias", *a.values(), None)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(dtype=Q.MOE_F32), UNS, "dtype"), (dict(S=0), INV, "S = 0"), (dict(S=1025), INV, "S = 1025"),
    (dict(N=0), INV, "positive"), (dict(N=60), UNS, "multiples of 8"), (dict(K=100), UNS, "multiples of 8"),
    (dict(N=1 << 20, K=2048), UNS, "2^30"), (dict(R=-1), INV, "R = -1"), (dict(R=(1 << 24) + 1), INV, "2^24"),
    (dict(k=0), INV, "k = 0"), (dict(k=65), INV, "k = 65"), (dict(xr=3), INV, "row mode"), (dict(yr=2), INV, "TOKEN"),
    (dict(off=None), INV, "slot_offsets"), (dict(perm=None, xr=1), INV, "perm_pair"), (dict(act=-1), INV, "act"),
    (dict(act=6), INV, "act"), (dict(act=1, N=56), UNS, "multiple of 16"), (dict(yt=Q.MOE_F16), UNS, "y dtype"),
    (dict(bt=Q.MOE_F16), UNS, "bias dtype"), (dict(rt=Q.MOE_F16), UNS, "residual dtype"), (dict(w=None), INV, "NULL"),
    (dict(x=None), INV, "NULL"), (dict(y=None), INV, "NULL"), (dict(bias=FAKE + 8), INV, "aligned"),
    (dict(res=FAKE + 8), INV, "aligned"), (dict(z=FAKE + 4), INV, "aligned"), (dict(stride=64), INV, "smaller"),
    (dict(stride=64 * 128 * 2 + 8), INV, "aligned"), (dict(res=FAKE * 2, yt=Q.MOE_F32), INV, "residual"),
    (dict(z=FAKE * 2), INV, "overlaps"), (dict(z=FAKE * 3), INV, "overlaps"),
])
def test_biased_product_refusals(kw, want, needle):
    _refused(_bias(**kw), want, needle)


def _act(**kw):
    a = dict(dy=FAKE, z=FAKE * 2, dtype=Q.MOE_BF16, S=4, N=64, off=FAKE, R=8, perm=FAKE, rows=0, act=Q.MOE_ACT_GELU,
             dz=FAKE * 3, h=FAKE * 4, db=FAKE * 5, ws=FAKE * 6, wsb=1 << 40)
    a.update(kw)
    return _call("moe_expert_act_backward", *a.values(), None)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(S=0), INV, "S = 0"), (dict(N=0), INV, "positive"), (dict(N=60), UNS, "multiple of 8"),
    (dict(N=(1 << 20) + 8), UNS, "2^20"), (dict(R=-1), INV, "R = -1"), (dict(dtype=3), INV, "dtype"),
    (dict(act=9), INV, "act"), (dict(act=1, N=56), UNS, "multiple of 16"), (dict(rows=2), INV, "row mode"),
    (dict(off=None), INV, "slot_offsets"), (dict(perm=None, rows=1), INV, "perm_pair"), (dict(dy=None), INV, "NULL"),
    (dict(z=None), INV, "NULL"), (dict(dz=None), INV, "NULL"), (dict(act=0), INV, "MOE_ACT_NONE"),
    (dict(act=0, z=None, dz=None, h=None, db=None), INV, "MOE_ACT_NONE"), (dict(dz=FAKE + 8), INV, "aligned"),
    (dict(db=FAKE + 4), INV, "aligned"), (dict(act=1, dz=FAKE), INV, "overlaps"), (dict(h=FAKE * 3), INV, "overlaps"),
    (dict(h=FAKE * 2), INV, "overlaps"), (dict(wsb=8), WSS, "needed"), (dict(ws=None), INV, "workspace"),
    (dict(ws=FAKE + 8), INV, "workspace"),
])
def test_act_backward_refusals(kw, want, needle):
    _refused(_act(**kw), want, needle)


def test_act_backward_without_rows_or_sums():
    assert _act(R=0, db=None)[0] == Q.MOE_OK  # nothing to do, nothing enqueued


@pytest.mark.parametrize("args", [(0, 64, 8), (1025, 64, 8), (4, 60, 8), (4, 0, 8), (4, 64, -1), (4, 64, (1 << 24) + 1)])
def test_act_backward_workspace_out_of_range(args):
    assert Q.moe_expert_act_backward_workspace_size(*args) == 0


def _losses(**kw):
    a = dict(l=FAKE, ids=FAKE, T=8, E=16, k=2, score=0, off=FAKE, G=2, counts=FAKE, probs=FAKE, losses=FAKE, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return _call("moe_balance_loss", *a.values(), None)


def _route(**kw):
    a = dict(l=FAKE, ids=FAKE, dw=FAKE, T=8, E=16, k=2, score=0, renorm=1, scale=1.0, counts=FAKE, dl=FAKE, off=FAKE, G=2,
             out=FAKE * 2, ot=Q.MOE_BF16)
    a.update(kw)
    a["scale"] = f32(a["scale"])
    return _call("moe_route_backward", *a.values(), None)


@pytest.mark.parametrize("call", [_losses, _route])
@pytest.mark.parametrize("kw,needle", [
    (dict(E=0), "E = 0"), (dict(E=1025), "E = 1025"), (dict(k=0), "k = 0"), (dict(k=17), "k = 17"),
    (dict(E=128, k=65), "k = 65"), (dict(T=-1), "T = -1"), (dict(T=(1 << 23) + 1), "2^24"), (dict(score=2), "score"),
    (dict(G=0), "G = 0"), (dict(G=1025), "G = 1025"), (dict(off=None), "seq_offsets"), (dict(l=None), "NULL"),
    (dict(ids=None), "NULL"),
])
def test_router_refusals(call, kw, needle):
    _refused(call(**kw), INV, needle)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(counts=None), INV, "NULL"), (dict(probs=None), INV, "NULL"), (dict(losses=None), INV, "NULL"),
    (dict(wsb=8), WSS, "needed"), (dict(ws=None), INV, "workspace"), (dict(ws=FAKE + 4), INV, "workspace"),
])
def test_balance_loss_refusals(kw, want, needle):
    _refused(_losses(**kw), want, needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(counts=None), "go together"), (dict(dl=None), "go together"), (dict(counts=None, dl=None, dw=None), "neither"),
    (dict(out=None), "NULL"), (dict(ot=4), "dtype"), (dict(scale=float("nan")), "scale"), (dict(out=FAKE), "MOE_F32"),
])
def test_route_backward_refusals(kw, needle):
    _refused(_route(**kw), INV, needle)


def test_route_backward_of_no_rows():
    assert _route(T=0)[0] == Q.MOE_OK


@pytest.mark.parametrize("args", [(-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, 0), (8, 8, 1025)])
def test_balance_loss_workspace_out_of_range(args):
    assert Q.moe_balance_loss_workspace_size(*args) == 0


def _combine(**kw):
    a = dict(dy=FAKE, dt=Q.MOE_F32, yp=FAKE * 2, pt=Q.MOE_BF16, ids=FAKE, w=FAKE, soe=FAKE, E=16, S=8, T=4, k=2, H=64,
             dyp=FAKE * 3, dw=FAKE * 4)
    a.update(kw)
    return _call("moe_combine_backward", *a.values(), None)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(dt=3), INV, "dy dtype"), (dict(pt=-1), INV, "pairs dtype"), (dict(E=0), INV, "E = 0"), (dict(S=17), INV, "S = 17"),
    (dict(S=-1), INV, "S = -1"), (dict(k=0), INV, "k = 0"), (dict(k=65), INV, "k = 65"), (dict(T=-1), INV, "T = -1"),
    (dict(T=(1 << 23) + 1), INV, "2^24"), (dict(H=0), INV, "positive"), (dict(H=60), UNS, "multiple of 8"),
    (dict(dy=None), INV, "NULL"), (dict(dw=None), INV, "NULL"), (dict(soe=None), INV, "NULL"),
    (dict(yp=FAKE + 8), INV, "aligned"), (dict(dyp=FAKE), INV, "overlaps"), (dict(dw=FAKE), INV, "overlaps"),
])
def test_combine_backward_refusals(kw, want, needle):
    _refused(_combine(**kw), want, needle)


def test_combine_backward_of_no_rows():
    assert _combine(T=0, dy=None, dw=None)[0] == Q.MOE_OK


def _list(values, ctype):
    return None if values is None else (ctype * len(values))(*values)


def _norm(at=(FAKE,), counts=(8,), types=(0,), n=None, table=None, kind=0, scale=1.0, total=FAKE, ws=FAKE, wsb=1 << 40):
    return _call("moe_grad_norm", _list(at, ctypes.c_void_p), _list(counts, ctypes.c_int64), _list(types, ctypes.c_int32),
                 len(at) if n is None else n, table, kind, f32(scale), total, ws, wsb, None)


def _clip(at=(FAKE,), counts=(8,), types=(0,), n=None, table=None, outs=None, otypes=None, otable=None, total=FAKE, max_norm=1.0,
          eps=1e-6, scale=1.0):
    return _call("moe_grad_clip", _list(at, ctypes.c_void_p), _list(counts, ctypes.c_int64), _list(types, ctypes.c_int32),
                 len(at) if n is None else n, table, _list(outs, ctypes.c_void_p), _list(otypes, ctypes.c_int32), otable, total,
                 f32(max_norm), f32(eps), f32(scale), None)


@pytest.mark.parametrize("call", [_norm, _clip])
@pytest.mark.parametrize("kw,needle", [
    (dict(n=-1), "n = -1"), (dict(n=(1 << 20) + 1), "2^20"), (dict(at=None, n=1), "NULL"), (dict(counts=None), "NULL"),
    (dict(types=None), "NULL"), (dict(types=(3,)), "grads[0]"), (dict(counts=(-1,)), "grads[0]"),
    (dict(counts=((1 << 40) + 1,)), "2^40"), (dict(at=(None,)), "grads[0] is NULL"), (dict(at=(FAKE + 2,)), "aligned"),
    (dict(at=(FAKE, FAKE + 1), counts=(8, 8), types=(0, 1)), "grads[1]"), (dict(total=None), "NULL"),
    (dict(scale=float("inf")), "scale"), (dict(table=FAKE + 4), "table"),
])
def test_gradient_list_refusals(call, kw, needle):
    _refused(call(**kw), INV, needle)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(kind=2), INV, "norm kind"), (dict(wsb=16), WSS, "needed"), (dict(ws=None), INV, "workspace"),
    (dict(ws=FAKE + 8), INV, "workspace"),
])
def test_gradient_norm_refusals(kw, want, needle):
    _refused(_norm(**kw), want, needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(max_norm=-1.0), "max_norm"), (dict(max_norm=float("nan")), "max_norm"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(outs=(FAKE * 2,)), "go together"), (dict(otypes=(0,)), "go together"),
    (dict(outs=(FAKE * 2,), otypes=(5,)), "outs[0]"), (dict(outs=(FAKE * 2 + 1,), otypes=(0,)), "outs[0]"),
    (dict(outs=(FAKE,), otypes=(1,)), "another type"), (dict(otable=FAKE + 2), "table"),
])
def test_gradient_clip_refusals(kw, needle):
    _refused(_clip(**kw), INV, needle)


def test_gradient_clip_of_an_empty_list():
    assert _clip(at=(), counts=(), types=(), n=0)[0] == Q.MOE_OK
    assert _clip(at=(None,), counts=(0,), types=(1,))[0] == Q.MOE_OK


def test_gradient_table():
    """Empty tensors are left out; chunks are of 4096 elements while the list is short."""
    at, counts, types = (FAKE, None, FAKE * 2, FAKE * 3), (5000, 0, 3, 4096), (1, 0, 0, 2)
    size = Q.lib().moe_grad_table_size(4)
    assert size == 4 * 24 and Q.lib().moe_grad_table_size(-1) == 0 and Q.lib().moe_grad_table_size((1 << 20) + 1) == 0
    table = (ctypes.c_uint64 * 12)()
    args = lambda **kw: [_list(kw.get("at", at), ctypes.c_void_p), _list(kw.get("counts", counts), ctypes.c_int64),
                         _list(kw.get("types", types), ctypes.c_int32), 4, kw.get("table", table), kw.get("size", size)]
    assert _call("moe_grad_table", *args())[0] == Q.MOE_OK
    both = lambda first: first | first << 32
    assert list(table) == [FAKE, 5000 | 1 << 60, both(0), FAKE * 2, 3, both(2), FAKE * 3, 4096 | 2 << 60, both(3), 0, 0, 0]
    _refused(_call("moe_grad_table", *args(size=size - 1)), WSS, "needed")
    _refused(_call("moe_grad_table", *args(table=None)), INV, "NULL")
    _refused(_call("moe_grad_table", *args(types=(1, 0, 0, 3))), INV, "at[3]")
    _refused(_call("moe_grad_table", *args(counts=(5000, 0, -3, 1))), INV, "at[2]")


def test_gradient_table_of_the_largest_lists():
    """The chunks of any list, a workgroup of 256 threads each, stay below 2^32 threads."""
    n = 4
    table = (ctypes.c_uint64 * (3 * n))()
    st, _ = _call("moe_grad_table", _list([FAKE << 20] * n, ctypes.c_void_p), _list([1 << 40] * n, ctypes.c_int64),
                  _list([1] * n, ctypes.c_int32), n, table, ctypes.sizeof(table))
    assert st == Q.MOE_OK
    last = table[3 * n - 1]
    for first in (last & 0xFFFFFFFF, last >> 32):  # three quarters of the chunks lie before the last tensor
        assert 0 < first * 4 // 3 * 256 < 1 << 32


def test_gradient_norm_workspace():
    size = Q.moe_grad_norm_workspace_size
    assert size(-1) == 0 and size((1 << 20) + 1) == 0 and size(0) > 0 and size(1 << 20) > size(1) > 0
