"""The expert products, 4-bit products, block norms and SwiGLU without a GPU:
every refusal of the C ABI names its argument before anything is enqueued,
and the binding refuses what the kernels could not address."""
import ctypes

import pytest
import torch

import quantized_routed_expert_moe_amd as Q

FAKE = 1 << 20  # aligned non-null address; never dereferenced on these paths
INV, UNS, WSS = Q.MOE_ERR_INVALID_ARGUMENT, Q.MOE_ERR_UNSUPPORTED, Q.MOE_ERR_WORKSPACE_TOO_SMALL


def _call(name, *args):
    st = getattr(Q.lib(), name)(*args)
    return st, Q.lib().moe_last_error().decode()


def _gemm(**kw):
    a = dict(x=FAKE, dtype=Q.MOE_BF16, w=FAKE, stride=64 * 128 * 2, S=4, N=64, K=128, tr=0, off=FAKE, R=8, perm=FAKE,
             k=2, xr=0, yr=0, act=0, y=FAKE, yt=Q.MOE_BF16)
    a.update(kw)
    return _call("moe_expert_gemm", *a.values(), None)


COMMON = [
    (dict(dtype=Q.MOE_F32), UNS, "dtype"), (dict(dtype=7), UNS, "dtype"),
    (dict(S=0), INV, "S = 0"), (dict(S=1025), INV, "S = 1025"), (dict(N=0), INV, "positive"),
    (dict(K=-8), INV, "positive"), (dict(N=60), UNS, "multiples of 8"), (dict(N=1 << 20, K=2048), UNS, "2^30"),
    (dict(R=-1), INV, "R = -1"), (dict(R=(1 << 24) + 1), INV, "2^24"), (dict(k=0), INV, "k = 0"),
    (dict(k=65), INV, "k = 65"), (dict(xr=3), INV, "row mode"), (dict(off=None), INV, "slot_offsets"),
    (dict(perm=None, xr=1), INV, "perm_pair"), (dict(x=None), INV, "NULL"), (dict(x=FAKE + 8), INV, "aligned"),
]
PRODUCT = COMMON + [
    (dict(act=2), INV, "act"), (dict(act=1, N=56), UNS, "multiple of 16"), (dict(yr=2), INV, "MOE_ROWS_TOKEN"),
    (dict(yt=Q.MOE_F16), UNS, "dtype"), (dict(y=None), INV, "NULL"), (dict(y=FAKE + 4), INV, "aligned"),
]


@pytest.mark.parametrize("kw,want,needle", PRODUCT + [
    (dict(K=100), UNS, "multiples of 8"), (dict(tr=2), INV, "transpose"), (dict(tr=1, act=1), INV, "transpose"),
    (dict(w=None), INV, "NULL"), (dict(stride=64 * 128 * 2 + 8), INV, "aligned"), (dict(stride=64), INV, "smaller"),
])
def test_product_refusals(kw, want, needle):
    st, msg = _gemm(**kw)
    assert st == want and needle in msg, (st, msg)


def _w4(**kw):
    a = dict(x=FAKE, dtype=Q.MOE_BF16, q=FAKE, sc=FAKE, st=Q.MOE_BF16, z=FAKE, group=64, S=4, N=64, K=128, off=FAKE,
             R=8, perm=FAKE, k=2, xr=0, yr=0, act=0, y=FAKE, yt=Q.MOE_BF16)
    a.update(kw)
    return _call("moe_expert_gemv_w4", *a.values(), None)


@pytest.mark.parametrize("kw,want,needle", PRODUCT + [
    (dict(group=48), UNS, "group"), (dict(group=256, K=512), UNS, "group"), (dict(group=0), UNS, "group"), (dict(group=128, K=192), UNS, "multiple of the group"),
    (dict(st=Q.MOE_F16), UNS, "scale"), (dict(q=None), INV, "NULL"), (dict(sc=None), INV, "NULL"),
    (dict(q=FAKE + 2), INV, "aligned"),
])
def test_w4_refusals(kw, want, needle):
    st, msg = _w4(**kw)
    assert st == want and needle in msg, (st, msg)


def _wgrad(**kw):
    a = dict(dy=FAKE, x=FAKE, dtype=Q.MOE_BF16, S=4, N=64, K=128, off=FAKE, R=8, perm=FAKE, k=2, dr=0, xr=0, dw=FAKE,
             dt=Q.MOE_F32, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return _call("moe_expert_gemm_wgrad", *a.values(), None)


@pytest.mark.parametrize("kw,want,needle", COMMON + [
    (dict(K=100), UNS, "multiples of 8"), (dict(dr=-1), INV, "row mode"), (dict(dt=Q.MOE_F16), UNS, "dtype"),
    (dict(dw=None), INV, "NULL"), (dict(dy=None), INV, "NULL"), (dict(dw=FAKE + 2), INV, "aligned"),
])
def test_wgrad_refusals(kw, want, needle):
    st, msg = _wgrad(**kw)
    assert st == want and needle in msg, (st, msg)


def test_wgrad_workspace():
    size = Q.moe_expert_gemm_wgrad_workspace_size
    assert size(0, 64, 64, 8) == 0 and size(4, 60, 64, 8) == 0 and size(4, 64, 64, -1) == 0
    need = size(1, 256, 256, 1 << 16)
    if need:
        st, msg = _wgrad(S=1, N=256, K=256, R=1 << 16, wsb=need - 1)
        assert st == WSS and str(need) in msg
        st, msg = _wgrad(S=1, N=256, K=256, R=1 << 16, ws=None)
        assert st == INV and "workspace" in msg


def _norm(backward=False, **kw):
    a = dict(x=FAKE, dtype=Q.MOE_BF16, y=FAKE, yt=Q.MOE_F32, wpost=FAKE, gate=FAKE, mode=1, wpre=FAKE, wt=Q.MOE_F32, T=4,
             H=256, eps=1e-6, a=1.0)
    f = dict(x_out=FAKE, h=FAKE)
    b = dict(dxo=FAKE, dh=FAKE, dx=FAKE, dy=FAKE, dpost=FAKE, dgate=FAKE, dpre=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(b if backward else f)
    a.update(kw)
    for n in ("eps", "a"):
        a[n] = ctypes.c_float(a[n])
    return _call("moe_block_norm_backward" if backward else "moe_block_norm", *a.values(), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,want,needle", [
    (dict(T=-1), INV, "T = -1"), (dict(H=0), INV, "positive"), (dict(H=100), UNS, "multiple of 8"),
    (dict(H=16392), UNS, "16384"), (dict(dtype=3), INV, "dtype"), (dict(yt=5), INV, "y dtype"), (dict(wt=5), INV, "w dtype"),
    (dict(mode=3), INV, "gate mode"), (dict(mode=0), INV, "gate"), (dict(gate=None), INV, "gate"),
    (dict(x=None), INV, "NULL"), (dict(y=None), INV, "need y"), (dict(eps=-1.0), INV, "eps"),
    (dict(eps=float("nan")), INV, "eps"), (dict(a=float("inf")), INV, "res_scale"), (dict(x=FAKE + 8), INV, "aligned"),
    (dict(wpre=FAKE + 4), INV, "aligned"),
])
def test_norm_refusals(backward, kw, want, needle):
    st, msg = _norm(backward, **kw)
    assert st == want and needle in msg, (st, msg)


@pytest.mark.parametrize("kw,needle", [(dict(h=None), "h and w_pre"), (dict(wpre=None), "h and w_pre"),
                                       (dict(wpre=None, h=None, x_out=None), "neither"), (dict(h=FAKE + 8), "aligned")])
def test_norm_forward_refusals(kw, needle):
    st, msg = _norm(**kw)
    assert st == INV and needle in msg, (st, msg)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(dx=None), INV, "dx"), (dict(dh=None), INV, "dh"), (dict(dy=None), INV, "dy"),
    (dict(dpost=None), INV, "dw_post"), (dict(dgate=None), INV, "dgate"), (dict(dpre=None), INV, "dw_pre"),
    (dict(wpre=None, dh=None, dpre=None, dxo=None), INV, "neither"), (dict(dx=FAKE + 8), INV, "aligned"),
    (dict(wsb=0), WSS, "workspace"), (dict(ws=None), INV, "workspace"),
])
def test_norm_backward_refusals(kw, want, needle):
    st, msg = _norm(True, **kw)
    assert st == want and needle in msg, (st, msg)


def test_norm_workspace():
    size = Q.moe_block_norm_backward_workspace_size
    assert size(-1, 64) == 0 and size(4, 60) == 0 and size(4, 16392) == 0
    assert size(1, 256) > 0 and size(10000, 256) >= size(1, 256)


@pytest.mark.parametrize("kw,want,needle", [
    (dict(dtype=9), INV, "dtype"), (dict(R=-1), INV, "R = -1"), (dict(I=0), INV, "positive"), (dict(I=12), UNS, "multiple of 8"),
    (dict(S=2, off=None), INV, "slot_offsets"), (dict(S=0), INV, "slot_offsets"), (dict(gu=None), INV, "NULL"),
    (dict(h=FAKE + 8), INV, "aligned"),
])
def test_swiglu_refusals(kw, want, needle):
    a = dict(gu=FAKE, dtype=Q.MOE_BF16, R=4, I=64, off=FAKE, S=2, h=FAKE)
    a.update(kw)
    st, msg = _call("moe_swiglu", *a.values(), None)
    assert st == want and needle in msg, (st, msg)
    b = dict(gu=a["gu"], dh=FAKE, dtype=a["dtype"], R=a["R"], I=a["I"], off=a["off"], S=a["S"], dgu=FAKE, h=a["h"])
    st, msg = _call("moe_swiglu_backward", *b.values(), None)
    assert st == want and needle in msg, (st, msg)


def test_swiglu_missing_outputs():
    st, msg = _call("moe_swiglu", FAKE, Q.MOE_BF16, 4, 64, None, 0, None, None)
    assert st == INV and "NULL" in msg
    st, msg = _call("moe_swiglu_backward", FAKE, None, Q.MOE_BF16, 4, 64, None, 0, FAKE, None, None)
    assert st == INV and "NULL" in msg


def test_nothing_to_do_needs_no_device():
    """Calls over no rows that write nothing return before any HIP call."""
    assert _gemm(R=0, x=None, y=None, perm=None)[0] == Q.MOE_OK
    assert _w4(R=0, x=None, y=None, perm=None)[0] == Q.MOE_OK
    assert _norm(T=0, x=None, y=None, x_out=None, h=None)[0] == Q.MOE_OK
    assert _call("moe_swiglu", None, Q.MOE_BF16, 0, 64, None, 0, None, None)[0] == Q.MOE_OK


class TestBinding:
    """Shape and type checks of the binding, on CPU tensors: every refusal comes before a kernel could run."""

    @pytest.fixture(autouse=True)
    def _device(self, monkeypatch):
        monkeypatch.setattr(Q, "_op_device", lambda: (Q._op_types(), 0)[1])

    def bf(self, *shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    def i32(self, *shape):
        return torch.zeros(shape, dtype=torch.int32)

    def test_tensors_must_be_on_the_current_device(self):
        with pytest.raises(TypeError, match="x must be a tensor on the current device"):
            Q.moe_expert_gemm(self.bf(4, 16), self.bf(2, 8, 16), self.i32(3), self.bf(4, 8))
        with pytest.raises(TypeError, match="current device"):
            Q.moe_swiglu(self.bf(4, 16), self.bf(4, 8))

    def test_stream_of_another_device_is_refused(self):
        from types import SimpleNamespace
        assert Q._op_stream(0, SimpleNamespace(cuda_stream=16, device_index=0)) == 16
        with pytest.raises(ValueError, match="current device"):
            Q._op_stream(0, SimpleNamespace(cuda_stream=16, device_index=1))

    @pytest.mark.parametrize("kw,match", [
        (dict(x=(4, 24)), "x has shape"), (dict(y=(3, 8)), "y has shape"), (dict(y=(4, 16)), "y has shape"),
        (dict(off=(4,)), "slot_offsets"), (dict(x_rows=1), "perm_pair"), (dict(w=(8, 16)), r"\[S, N, K\]"),
    ])
    def test_product_shapes(self, kw, match):
        a = dict(x=(4, 16), w=(2, 8, 16), off=(3,), y=(4, 8))
        more = {k: kw.pop(k) for k in ("x_rows",) if k in kw}
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            Q.moe_expert_gemm(self.bf(*a["x"]), self.bf(*a["w"]), self.i32(*a["off"]), self.bf(*a["y"]), **more)

    def test_product_types(self):
        with pytest.raises(TypeError, match="w has dtype"):
            Q.moe_expert_gemm(self.bf(4, 16), self.bf(2, 8, 16).half(), self.i32(3), self.bf(4, 8))
        with pytest.raises(ValueError, match="contiguous matrices"):
            Q.moe_expert_gemm(self.bf(4, 16), self.bf(2, 16, 8).transpose(1, 2), self.i32(3), self.bf(4, 8))
        with pytest.raises(ValueError, match="int32"):
            Q.moe_expert_gemm(self.bf(4, 16), self.bf(2, 8, 16), self.i32(3).long(), self.bf(4, 8))

    def test_token_rows(self):
        with pytest.raises(ValueError, match="at least 3 rows"):
            Q.moe_expert_gemm(self.bf(2, 16), self.bf(2, 8, 16), self.i32(3), self.bf(5, 8), self.i32(5), 2,
                              Q.MOE_ROWS_TOKEN)

    def test_w4_shapes(self):
        q = torch.zeros((2, 8, 32), dtype=torch.uint8)
        with pytest.raises(ValueError, match="scales have shape"):
            Q.moe_expert_gemv_w4(self.bf(4, 64), q, self.bf(2, 8, 1), None, 32, self.i32(3), self.bf(4, 8))
        with pytest.raises(ValueError, match="zeros"):
            Q.moe_expert_gemv_w4(self.bf(4, 64), q, self.bf(2, 8, 2), self.bf(2, 8, 2), 32, self.i32(3), self.bf(4, 8))
        with pytest.raises(ValueError, match="uint8"):
            Q.moe_expert_gemv_w4(self.bf(4, 64), self.bf(2, 8, 32), self.bf(2, 8, 2), None, 32, self.i32(3), self.bf(4, 8))

    def test_norm_shapes(self):
        x, w = self.bf(4, 64), torch.zeros(64)
        with pytest.raises(ValueError, match="one shape"):
            Q.moe_block_norm(x, self.bf(3, 64), w, None, w, x, x, 1e-6)
        with pytest.raises(ValueError, match="w_pre must be"):
            Q.moe_block_norm(x, x, w, None, w[:32], x, x, 1e-6)
        with pytest.raises(ValueError, match="gate has shape"):
            Q.moe_block_norm(x, x, w, torch.zeros(4), w, x, x, 1e-6)
        with pytest.raises(TypeError, match="one dtype"):
            Q.moe_block_norm(x, x, w, None, w.half(), x, x, 1e-6)
        with pytest.raises(ValueError, match="x_out must have"):
            Q.moe_block_norm(x, x, w, None, w, x.float(), x, 1e-6)
        with pytest.raises(ValueError, match="dw_pre must be"):
            Q.moe_block_norm_backward(x, x, w, None, w, x, x, x, x, w, None, None, 1e-6)
