"""Python binding of libqmoe (include/qmoe.h): one routed-expert MoE layer on MI355X.

Argument marshalling only: every function here has the name of a C entry
point, checks that the tensors it is given are contiguous device tensors of
the right dtype, and passes their addresses, the sizes and the current HIP
stream to the library.  All compute runs in the library's HIP kernels.  If
the library is not built the first call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "qmoe.h")

MOE_OK, MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_HIP = range(5)
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_F32, MOE_BF16 = 0, 1
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL, MOE_PATH_PREFILL_I8 = 0, 1, 2, 3
MOE_FMT_Q8_0, MOE_FMT_Q4K, MOE_FMT_MXFP4, MOE_FMT_Q3K_Q4K, MOE_FMT_Q5K, MOE_FMT_Q6K = 0, 1, 2, 3, 4, 5
# (MOE_FMT_Q3K_Q4K: Q3_K gate and up, Q4_K down)
STAGES = ("route", "batches", "prefill_tiles", "ffn_gateup", "ffn_down", "combine", "prefill_gateup", "prefill_down",
          "route_batches")


class QmoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_status_name(status)}: {message}")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        i32, f32, vp, sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
        L.moe_status_name.argtypes = [i32]
        L.moe_status_name.restype = ctypes.c_char_p
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_route_topk.argtypes = [vp, i32, i32, i32, i32, i32, f32, vp, vp, vp]
        L.moe_batches_workspace_size.argtypes = [i32, i32, i32, i32]
        L.moe_batches_workspace_size.restype = sz
        L.moe_build_expert_batches.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                               vp]
        L.moe_route_and_batch.argtypes = [vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp, sz, vp]
        L.moe_count_routes.argtypes = [vp, i32, i32, i32, vp, vp]
        L.moe_expert_blob_bytes.argtypes = [i32, i32, i32]
        L.moe_expert_blob_bytes.restype = sz
        L.moe_packed_blob_bytes.argtypes = [i32, i32, i32]
        L.moe_packed_blob_bytes.restype = sz
        L.moe_pack_expert.argtypes = [i32, vp, vp, i32, i32]
        L.moe_unpack_expert.argtypes = [i32, vp, vp, i32, i32]
        L.moe_pack_q4k.argtypes = [vp, vp, i32, i32, i32]
        L.moe_pack_q8_0.argtypes = [vp, vp, i32, i32, i32]
        L.moe_validate_slot_map.argtypes = [vp, i32, i32]
        L.moe_ffn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.moe_ffn_workspace_size.restype = sz
        ffn = [vp, sz, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp, sz, vp]
        L.moe_expert_ffn_q4k.argtypes = ffn
        L.moe_expert_ffn_q8_0.argtypes = ffn
        L.moe_expert_ffn_mxfp4.argtypes = ffn
        L.moe_expert_ffn_q3k_q4k.argtypes = ffn
        L.moe_expert_ffn_q5k.argtypes = ffn
        L.moe_expert_ffn_q6k.argtypes = ffn
        L.moe_expert_ffn_q4k_noalloc.argtypes = ffn[:16] + [vp]
        L.moe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i32, vp, i32, i32, i32, vp, i32, vp]
        L.moe_layer_decode_workspace_size.argtypes = [i32] * 8
        L.moe_layer_decode_workspace_size.restype = sz
        L.moe_layer_decode.argtypes = [i32, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp, sz, i32, i32, vp,
                                       i32] + \
            [vp] * 13 + [vp, sz, vp]
        L.moe_timer_begin.argtypes = [i32, i32]
        L.moe_timer_end.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]
        L.moe_timer_read.argtypes = [i32, vp, i32, ctypes.POINTER(ctypes.c_int)]
        L.moe_hbm_read_probe.argtypes = [vp, sz, i32, i32, vp, ctypes.POINTER(ctypes.c_size_t), vp]
        L.moe_prefill_inner_probe.argtypes = [i32, i32, vp, sz, vp]
        L.moe_expert_gemm.argtypes = [vp, i32, vp, sz, i32, i32, i32, i32, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp]
        L.moe_expert_gemm_wgrad_workspace_size.argtypes = [i32] * 4
        L.moe_expert_gemm_wgrad_workspace_size.restype = sz
        L.moe_expert_gemm_wgrad.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, i32, i32, i32, vp, i32, vp, sz, vp]
        L.moe_expert_gemv_w4.argtypes = [vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, i32, i32, i32, i32,
                                         vp, i32, vp]
        L.moe_block_norm.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, i32, i32, i32, f32, f32, vp, vp, vp]
        L.moe_block_norm_backward_workspace_size.argtypes = [i32, i32]
        L.moe_block_norm_backward_workspace_size.restype = sz
        L.moe_block_norm_backward.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, i32, i32, i32, f32, f32] + [vp] * 8 + \
            [sz, vp]
        L.moe_swiglu.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp]
        L.moe_swiglu_backward.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, vp, vp]
        for name in ("moe_route_topk", "moe_build_expert_batches", "moe_route_and_batch", "moe_count_routes",
                     "moe_pack_expert", "moe_unpack_expert", "moe_pack_q4k", "moe_pack_q8_0",
                     "moe_validate_slot_map", "moe_expert_ffn_q4k", "moe_expert_ffn_q8_0", "moe_expert_ffn_mxfp4",
                     "moe_expert_ffn_q3k_q4k", "moe_expert_ffn_q5k", "moe_expert_ffn_q6k", "moe_expert_ffn_q4k_noalloc",
                     "moe_combine", "moe_layer_decode",
                     "moe_timer_begin", "moe_timer_end", "moe_timer_read", "moe_hbm_read_probe",
                     "moe_prefill_inner_probe", "moe_expert_gemm", "moe_expert_gemm_wgrad", "moe_expert_gemv_w4",
                     "moe_block_norm", "moe_block_norm_backward", "moe_swiglu", "moe_swiglu_backward"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def header_functions(header: str | None = None) -> list[str]:
    """Names of the functions a header declares (default include/qmoe.h)."""
    text = open(header or HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def _status_name(st: int) -> str:
    return lib().moe_status_name(st).decode()


def _check(st: int) -> None:
    if st != MOE_OK:
        raise QmoeError(st, lib().moe_last_error().decode())


# ------------------------------------------------------------ marshalling

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev(t, dtypes=None, name="tensor") -> int:
    if t is None:
        return 0
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


_MAPPED = {}  # pinned host allocation base -> its device address


def _dev_or_mapped(t, dtypes=None, name="tensor") -> int:
    """Device address of a device tensor, or of a pinned host tensor (the
    device-side address of its pinned allocation from hipHostGetDevicePointer;
    an allocation the device cannot address raises here, before any launch)."""
    import torch
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.is_pinned():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtypes is not None and t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
        base = t.untyped_storage().data_ptr()
        if base not in _MAPPED:
            hip = ctypes.CDLL("libamdhip64.so")
            dptr = ctypes.c_void_p()
            rc = hip.hipHostGetDevicePointer(ctypes.byref(dptr), ctypes.c_void_p(base), 0)
            if rc != 0 or not dptr.value:
                raise QmoeError(MOE_ERR_HIP, f"{name}: pinned host memory has no device address (hip error {rc})")
            _MAPPED[base] = dptr.value
        return _MAPPED[base] + (t.data_ptr() - base)
    return _dev(t, dtypes, name)


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _i32():
    import torch
    return (torch.int32,)


def _f32():
    import torch
    return (torch.float32,)


def _fb():
    import torch
    return (torch.float32, torch.bfloat16)


def _u32():
    """Counters: uint32 in the ABI; an int32 tensor holds the same bits."""
    import torch
    return tuple(t for t in (torch.int32, getattr(torch, "uint32", None)) if t is not None)


# ------------------------------------------------------------------ calls

def moe_route_topk(logits, k: int, score: int, renormalize: bool, scale: float, topk_ids, topk_w, stream=None):
    T, E = logits.shape
    _check(lib().moe_route_topk(_dev(logits, _f32(), "logits"), T, E, k, score, int(bool(renormalize)), float(scale),
                                _dev(topk_ids, _i32(), "topk_ids"), _dev(topk_w, _f32(), "topk_w"),
                                _stream(stream)))


def moe_batches_workspace_size(T: int, k: int, E: int, S: int) -> int:
    return int(lib().moe_batches_workspace_size(T, k, E, S))


def moe_build_expert_batches(topk_ids, topk_w, E: int, slot_of_expert, S: int, slot_offsets, active_slots, num_active,
                             perm_pair, host_token, host_expert, host_weight, host_count, ws=None, stream=None):
    T, k = topk_ids.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_build_expert_batches(
        _dev(topk_ids, _i32(), "topk_ids"), _dev(topk_w, _f32(), "topk_w"), T, k, E,
        _dev(slot_of_expert, _i32(), "slot_of_expert"), S, _dev(slot_offsets, _i32(), "slot_offsets"),
        _dev(active_slots, _i32(), "active_slots"), _dev(num_active, _i32(), "num_active"),
        _dev(perm_pair, _i32(), "perm_pair"), _dev_or_mapped(host_token, _i32(), "host_token"),
        _dev_or_mapped(host_expert, _i32(), "host_expert"), _dev_or_mapped(host_weight, _f32(), "host_weight"),
        _dev_or_mapped(host_count, _i32(), "host_count"), _dev(ws, None, "ws"), ws_bytes, _stream(stream)))


def moe_route_and_batch(logits, k: int, score: int, renormalize: bool, scale: float, topk_ids, topk_w, E: int,
                        slot_of_expert, S: int, slot_offsets, active_slots, num_active, perm_pair, host_token,
                        host_expert, host_weight, host_count, ws=None, stream=None, route_counts=None):
    """route_counts: optional device int32/uint32 [E] routing counters (each
    pair adds one to its expert)."""
    T, E_ = logits.shape
    if E_ != E:
        raise ValueError(f"logits have {E_} experts, E = {E}")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_route_and_batch(
        _dev(logits, _f32(), "logits"), T, E, k, score, int(bool(renormalize)), float(scale),
        _dev(topk_ids, _i32(), "topk_ids"), _dev(topk_w, _f32(), "topk_w"),
        _dev(slot_of_expert, _i32(), "slot_of_expert"), S, _dev(slot_offsets, _i32(), "slot_offsets"),
        _dev(active_slots, _i32(), "active_slots"), _dev(num_active, _i32(), "num_active"),
        _dev(perm_pair, _i32(), "perm_pair"), _dev_or_mapped(host_token, _i32(), "host_token"),
        _dev_or_mapped(host_expert, _i32(), "host_expert"), _dev_or_mapped(host_weight, _f32(), "host_weight"),
        _dev_or_mapped(host_count, _i32(), "host_count"), _dev(route_counts, _u32(), "route_counts"),
        _dev(ws, None, "ws"), ws_bytes, _stream(stream)))


def moe_count_routes(topk_ids, E: int, counts, stream=None):
    """counts[e] += pairs of topk_ids [T, k] routed to e (device, int32/uint32 [E])."""
    T, k = topk_ids.shape
    if counts is None:
        raise ValueError("counts must be a device tensor")
    _check(lib().moe_count_routes(_dev(topk_ids, _i32(), "topk_ids"), T, k, E, _dev(counts, _u32(), "counts"),
                                  _stream(stream)))


def moe_expert_blob_bytes(fmt: int, H: int, I: int) -> int:
    return int(lib().moe_expert_blob_bytes(fmt, H, I))


def moe_packed_blob_bytes(fmt: int, H: int, I: int) -> int:
    """Bytes of a packed blob (a slot's minimum size)."""
    return int(lib().moe_packed_blob_bytes(fmt, H, I))


def moe_pack_expert(fmt: int, canonical: np.ndarray, H: int, I: int, out: np.ndarray | None = None) -> np.ndarray:
    n = moe_expert_blob_bytes(fmt, H, I)
    canonical = np.ascontiguousarray(canonical, dtype=np.uint8)
    if canonical.nbytes != n:
        raise ValueError(f"canonical blob has {canonical.nbytes} bytes, expected {n}")
    npk = moe_packed_blob_bytes(fmt, H, I)
    if out is None:
        out = np.empty(npk, dtype=np.uint8)
    if out.nbytes != npk or not out.flags.c_contiguous:
        raise ValueError(f"out must be a contiguous {npk}-byte array")
    _check(lib().moe_pack_expert(fmt, canonical.ctypes.data, out.ctypes.data, H, I))
    return out


def moe_unpack_expert(fmt: int, packed: np.ndarray, H: int, I: int) -> np.ndarray:
    n, npk = moe_expert_blob_bytes(fmt, H, I), moe_packed_blob_bytes(fmt, H, I)
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    if packed.nbytes != npk:
        raise ValueError(f"packed blob has {packed.nbytes} bytes, expected {npk}")
    out = np.empty(n, dtype=np.uint8)
    _check(lib().moe_unpack_expert(fmt, packed.ctypes.data, out.ctypes.data, H, I))
    return out


def _pack_matrix(fn, block_w: int, block_b: int, canonical: np.ndarray, rows: int, cols: int,
                 gate_up_interleave: bool) -> np.ndarray:
    n = rows * cols * (2 if gate_up_interleave else 1) // block_w * block_b
    canonical = np.ascontiguousarray(canonical, dtype=np.uint8)
    if canonical.nbytes != n:
        raise ValueError(f"canonical matrix data has {canonical.nbytes} bytes, expected {n}")
    out = np.empty(n, dtype=np.uint8)
    _check(fn(canonical.ctypes.data, out.ctypes.data, rows, cols, int(bool(gate_up_interleave))))
    return out


def moe_pack_q4k(canonical: np.ndarray, rows: int, cols: int, gate_up_interleave: bool) -> np.ndarray:
    """Device layout of one Q4_K matrix [rows, cols] (or of W_gate | W_up with gate_up_interleave)."""
    return _pack_matrix(lib().moe_pack_q4k, 256, 144, canonical, rows, cols, gate_up_interleave)


def moe_pack_q8_0(canonical: np.ndarray, rows: int, cols: int, gate_up_interleave: bool) -> np.ndarray:
    """Device layout of one Q8_0 matrix [rows, cols] (or of W_gate | W_up with gate_up_interleave)."""
    return _pack_matrix(lib().moe_pack_q8_0, 32, 34, canonical, rows, cols, gate_up_interleave)


def moe_validate_slot_map(slot_of_expert: np.ndarray, S: int) -> None:
    soe = np.ascontiguousarray(slot_of_expert, dtype=np.int32)
    _check(lib().moe_validate_slot_map(soe.ctypes.data, soe.size, S))


def moe_ffn_workspace_size(fmt: int, T: int, k: int, H: int, I: int, path: int) -> int:
    return int(lib().moe_ffn_workspace_size(fmt, T, k, H, I, path))


def _ffn(fn, slot_pool, slot_stride: int, S: int, H: int, I: int, x, k: int, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path: int, ws, stream):
    T = x.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    pool_ptr = slot_pool if isinstance(slot_pool, int) else _dev(slot_pool, None, "slot_pool")
    _check(fn(pool_ptr, slot_stride, S, H, I, _dev(x, _fb(), "x"), _dtype_code(x), T, k,
              _dev(slot_offsets, _i32(), "slot_offsets"), _dev(active_slots, _i32(), "active_slots"),
              _dev(num_active, _i32(), "num_active"), _dev(perm_pair, _i32(), "perm_pair"),
              _dev(y_pairs, _fb(), "y_pairs"), _dtype_code(y_pairs), path, _dev(ws, None, "ws"), ws_bytes,
              _stream(stream)))


def moe_expert_ffn_q4k(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                       y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_q4k, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn_q4k_noalloc(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
                               perm_pair, y_pairs, path=MOE_PATH_AUTO, stream=None):
    """moe_expert_ffn_q4k with the library's own scratch as its workspace (no allocation)."""
    T = x.shape[0]
    pool_ptr = slot_pool if isinstance(slot_pool, int) else _dev(slot_pool, None, "slot_pool")
    _check(lib().moe_expert_ffn_q4k_noalloc(
        pool_ptr, slot_stride, S, H, I, _dev(x, _fb(), "x"), _dtype_code(x), T, k,
        _dev(slot_offsets, _i32(), "slot_offsets"), _dev(active_slots, _i32(), "active_slots"),
        _dev(num_active, _i32(), "num_active"), _dev(perm_pair, _i32(), "perm_pair"), _dev(y_pairs, _fb(), "y_pairs"),
        _dtype_code(y_pairs), path, _stream(stream)))


MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_expert_ffn_q8_0(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                        y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_q8_0, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn_mxfp4(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                         y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_mxfp4, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn_q3k_q4k(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                           y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_q3k_q4k, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn_q5k(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                       y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_q5k, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn_q6k(slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active, perm_pair,
                       y_pairs, path=MOE_PATH_AUTO, ws=None, stream=None):
    _ffn(lib().moe_expert_ffn_q6k, slot_pool, slot_stride, S, H, I, x, k, slot_offsets, active_slots, num_active,
         perm_pair, y_pairs, path, ws, stream)


def moe_expert_ffn(fmt: int):
    """The expert-FFN call of a block format."""
    return {MOE_FMT_Q8_0: moe_expert_ffn_q8_0, MOE_FMT_Q4K: moe_expert_ffn_q4k, MOE_FMT_MXFP4: moe_expert_ffn_mxfp4,
            MOE_FMT_Q3K_Q4K: moe_expert_ffn_q3k_q4k, MOE_FMT_Q5K: moe_expert_ffn_q5k,
            MOE_FMT_Q6K: moe_expert_ffn_q6k}[fmt]


def moe_combine(y_pairs, topk_ids, topk_w, slot_of_expert, S: int, y_shared, y, stream=None):
    T, k = topk_ids.shape
    H = y.shape[1]
    E = slot_of_expert.numel()
    _check(lib().moe_combine(_dev(y_pairs, _fb(), "y_pairs"), _dtype_code(y_pairs), _dev(topk_ids, _i32(), "topk_ids"),
                             _dev(topk_w, _f32(), "topk_w"), _dev(slot_of_expert, _i32(), "slot_of_expert"), E, S,
                             _dev(y_shared, _f32(), "y_shared"), T, k, H, _dev(y, _fb(), "y"), _dtype_code(y),
                             _stream(stream)))


def moe_layer_decode_workspace_size(fmt: int, T: int, k: int, E: int, S: int, H: int, I: int, I_shared: int) -> int:
    return int(lib().moe_layer_decode_workspace_size(fmt, T, k, E, S, H, I, I_shared))


def moe_layer_decode(fmt: int, logits, x, k: int, score: int, renormalize: bool, scale: float, slot_of_expert, S: int,
                     slot_pool, slot_stride: int, I: int, shared_pool, I_shared: int, topk_ids, topk_w, slot_offsets,
                     active_slots, num_active, perm_pair, host_token, host_expert, host_weight, host_count, y_pairs, y,
                     ws, stream=None, route_counts=None):
    """The whole decode layer (routing, batching, routed and shared expert FFN, combine) in one call."""
    T, E = logits.shape
    H = x.shape[1]
    pool_ptr = slot_pool if isinstance(slot_pool, int) else _dev(slot_pool, None, "slot_pool")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_layer_decode(
        fmt, _dev(logits, _f32(), "logits"), _dev(x, _fb(), "x"), _dtype_code(x), T, E, k, score, int(bool(renormalize)),
        float(scale), _dev(slot_of_expert, _i32(), "slot_of_expert"), S, pool_ptr, slot_stride, H, I,
        _dev(shared_pool, None, "shared_pool"), I_shared if shared_pool is not None else 0,
        _dev(topk_ids, _i32(), "topk_ids"), _dev(topk_w, _f32(), "topk_w"), _dev(slot_offsets, _i32(), "slot_offsets"),
        _dev(active_slots, _i32(), "active_slots"), _dev(num_active, _i32(), "num_active"),
        _dev(perm_pair, _i32(), "perm_pair"), _dev_or_mapped(host_token, _i32(), "host_token"),
        _dev_or_mapped(host_expert, _i32(), "host_expert"), _dev_or_mapped(host_weight, _f32(), "host_weight"),
        _dev_or_mapped(host_count, _i32(), "host_count"), _dev(route_counts, _u32(), "route_counts"),
        _dev(y_pairs, _f32(), "y_pairs"), _dev(y, _f32(), "y"), _dev(ws, None, "ws"), ws_bytes, _stream(stream)))


# ------------------------------------- expert products, block norms, SwiGLU
# These calls take their sizes from the tensors' shapes and check every shape
# that a kernel relies on.  All tensors live on the current device, on whose
# current stream (or `stream`) the call is enqueued.  No call records itself for
# autograd: with gradients enabled a tensor that requires one is refused (call
# under torch.no_grad(), or from a torch.autograd.Function whose backward makes
# the gradient calls).

MOE_F16 = 2
MOE_ROWS_POSITION, MOE_ROWS_PAIR, MOE_ROWS_TOKEN = 0, 1, 2
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN = 0, 1, 2

_torch = None
_raw_stream = None  # device -> its current stream's handle, without building a Stream object
_CODES = {}  # torch dtype -> moe_dtype
_I32 = _U8 = _F32 = _Tensor = None


def _op_types() -> None:
    global _torch, _raw_stream, _I32, _U8, _F32, _Tensor
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _CODES.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16})
    _I32, _U8, _F32, _Tensor = torch.int32, torch.uint8, torch.float32, torch.Tensor
    _torch = torch


def _op_code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, expected float32, bfloat16 or float16")
    return code


def _op_ptrs(device: int, names: str, *tensors) -> list:
    """Addresses of the tensors (0 for None), each contiguous and on the device.  names: theirs, for a refusal."""
    out, grad = [], _torch.is_grad_enabled()
    for t in tensors:
        if t is None:
            out.append(0)
        elif isinstance(t, _Tensor) and t.get_device() == device and t.is_contiguous() and not (grad and t.requires_grad):
            out.append(t.data_ptr())
        else:
            _op_refuse(device, names.split()[len(out)], t)
    return out


def _op_refuse(device: int, name: str, t):
    if not isinstance(t, _Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a tensor on the current device (cuda:{device})")
    if t.requires_grad and _torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: call it under torch.no_grad() or "
                         "from a torch.autograd.Function")
    raise ValueError(f"{name} must be contiguous")


def _op_device() -> int:
    if _torch is None:
        _op_types()
    return _torch.cuda.current_device()


def _op_stream(device: int, stream) -> int:
    if stream is None:
        return _raw_stream(device)
    if getattr(stream, "device_index", device) != device:
        raise ValueError(f"stream must belong to the current device (cuda:{device})")
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _op_rows(slot_offsets, S: int, perm_pair, x, modes, k: int) -> int:
    """Batch positions of a product: perm_pair's length, or x's rows without one."""
    if slot_offsets is not None and (slot_offsets.dtype != _I32 or slot_offsets.shape != (S + 1,)):
        raise ValueError(f"slot_offsets must be int32 [{S + 1}]")
    if perm_pair is None:
        if any(m != MOE_ROWS_POSITION for m in modes):
            raise ValueError("the row modes need perm_pair")
        return x.shape[0]
    if perm_pair.dtype != _I32 or perm_pair.dim() != 1:
        raise ValueError("perm_pair must be int32 [R]")
    return perm_pair.shape[0]


def _op_matrix(t, cols: int, R: int, mode: int, k: int, name: str) -> None:
    need = -(-R // max(k, 1)) if mode == MOE_ROWS_TOKEN else R
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or shape[0] < need:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected at least {need} rows of {cols}")


def moe_expert_gemm(x, w, slot_offsets, y, perm_pair=None, k: int = 1, x_rows: int = MOE_ROWS_POSITION,
                    y_rows: int = MOE_ROWS_POSITION, transpose: bool = False, act: int = MOE_ACT_NONE, stream=None):
    """y rows = x rows times their slot's matrix of w [S, N, K] (transposed unless `transpose`)."""
    dev = _op_device()
    shape, strides = w.shape, w.stride()
    if len(shape) != 3 or strides[2] != 1 or (strides[1] != shape[2] and shape[1] != 1):
        raise ValueError("w must be [S, N, K] with contiguous matrices")
    S, N, K = shape
    wide_in, wide_out = (N, K) if transpose else (K, N // 2 if act else N)
    R = _op_rows(slot_offsets, S, perm_pair, x, (x_rows, y_rows), k)
    _op_matrix(x, wide_in, R, x_rows, k, "x")
    _op_matrix(y, wide_out, R, y_rows, k, "y")
    if w.dtype != x.dtype:
        raise TypeError(f"w has dtype {w.dtype}, x {x.dtype}")
    xp, op, pp, yp = _op_ptrs(dev, "x slot_offsets perm_pair y", x, slot_offsets, perm_pair, y)
    if w.get_device() != dev or (w.requires_grad and _torch.is_grad_enabled()):
        _op_refuse(dev, "w", w)
    _check(lib().moe_expert_gemm(xp, _op_code(x, "x"), w.data_ptr(), 2 * (strides[0] if S > 1 else N * K), S, N, K,
                                 int(bool(transpose)), op, R, pp, k, x_rows, y_rows, act, yp, _op_code(y, "y"),
                                 _op_stream(dev, stream)))


def moe_expert_gemm_wgrad_workspace_size(S: int, N: int, K: int, R: int) -> int:
    return int(lib().moe_expert_gemm_wgrad_workspace_size(S, N, K, R))


def moe_expert_gemm_wgrad(dy, x, slot_offsets, dw, perm_pair=None, k: int = 1, dy_rows: int = MOE_ROWS_POSITION,
                          x_rows: int = MOE_ROWS_POSITION, ws=None, stream=None):
    """dw [S, N, K] = per slot, the sum over its positions of dy row (outer) x row."""
    dev = _op_device()
    shape = dw.shape
    if len(shape) != 3:
        raise ValueError("dw must be [S, N, K]")
    S, N, K = shape
    R = _op_rows(slot_offsets, S, perm_pair, x, (dy_rows, x_rows), k)
    _op_matrix(dy, N, R, dy_rows, k, "dy")
    _op_matrix(x, K, R, x_rows, k, "x")
    if dy.dtype != x.dtype:
        raise TypeError(f"dy has dtype {dy.dtype}, x {x.dtype}")
    dp, xp, op, pp, wp, sp = _op_ptrs(dev, "dy x slot_offsets perm_pair dw ws", dy, x, slot_offsets, perm_pair, dw, ws)
    _check(lib().moe_expert_gemm_wgrad(dp, xp, _op_code(x, "x"), S, N, K, op, R, pp, k, dy_rows, x_rows, wp,
                                       _op_code(dw, "dw"), sp, 0 if ws is None else ws.numel() * ws.element_size(),
                                       _op_stream(dev, stream)))


def moe_expert_gemv_w4(x, q, scales, zeros, group: int, slot_offsets, y, perm_pair=None, k: int = 1,
                       x_rows: int = MOE_ROWS_POSITION, y_rows: int = MOE_ROWS_POSITION, act: int = MOE_ACT_NONE,
                       stream=None):
    """y rows = x rows times their slot's 4-bit matrix: codes q [S, N, K / 2], scales (and zeros) [S, N, K / group]."""
    dev = _op_device()
    shape = q.shape
    if len(shape) != 3 or q.dtype != _U8:
        raise ValueError("q must be uint8 [S, N, K / 2]")
    S, N, K = shape[0], shape[1], 2 * shape[2]
    if group < 1 or scales.shape != (S, N, K // group):
        raise ValueError(f"scales have shape {tuple(scales.shape)}, expected [{S}, {N}, K / group]")
    if zeros is not None and (zeros.dtype != _U8 or zeros.shape != scales.shape):
        raise ValueError("zeros must be uint8 with the shape of scales")
    R = _op_rows(slot_offsets, S, perm_pair, x, (x_rows, y_rows), k)
    _op_matrix(x, K, R, x_rows, k, "x")
    _op_matrix(y, N // 2 if act else N, R, y_rows, k, "y")
    xp, qp, sp, zp, op, pp, yp = _op_ptrs(dev, "x q scales zeros slot_offsets perm_pair y", x, q, scales, zeros,
                                          slot_offsets, perm_pair, y)
    _check(lib().moe_expert_gemv_w4(xp, _op_code(x, "x"), qp, sp, _op_code(scales, "scales"), zp, group, S, N, K, op,
                                    R, pp, k, x_rows, y_rows, act, yp, _op_code(y, "y"), _op_stream(dev, stream)))


def _norm_shapes(x, y, w_post, gate, w_pre) -> tuple:
    """(shape, gate mode, weight type) of a block norm's tensors."""
    shape = x.shape
    if len(shape) != 2 or (y is not None and y.shape != shape):
        raise ValueError("x and y must be [T, H] of one shape")
    T, H = shape
    vector, first = (H,), None
    for name, w in (("w_post", w_post), ("w_pre", w_pre), ("gate", gate)):
        if w is None:
            continue
        if first is None:
            first = w.dtype
        elif w.dtype != first:
            raise TypeError("w_post, gate and w_pre must have one dtype")
        if name != "gate" and w.shape != vector:
            raise ValueError(f"{name} must be [{H}]")
    mode = MOE_GATE_NONE
    if gate is not None:
        if gate.shape == vector:
            mode = MOE_GATE_CHANNEL
        elif gate.shape == (T, 1):
            mode = MOE_GATE_TOKEN
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected [{H}] (a channel's) or [{T}, 1] (a token's)")
    w = w_post if w_post is not None else w_pre if w_pre is not None else gate
    return shape, mode, MOE_F32 if w is None else _op_code(w, "weights")


def _norm_like(t, shape, dtype, name: str) -> None:
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}")


def moe_block_norm(x, y, w_post, gate, w_pre, x_out, h, eps: float, res_scale: float = 1.0, stream=None):
    """x_out = res_scale x + gate norm(y) w_post and h = norm(x_out) w_pre in one pass over the rows.  gate: [H] (one
    for each channel), [T, 1] (one for each token) or None; y, w_post, w_pre, x_out and h may be None."""
    dev = _op_device()
    shape, mode, w_code = _norm_shapes(x, y, w_post, gate, w_pre)
    T, H = shape
    dtype = x.dtype
    _norm_like(x_out, shape, dtype, "x_out")
    _norm_like(h, shape, dtype, "h")
    xp, yp, wp, gp, np_, op, hp = _op_ptrs(dev, "x y w_post gate w_pre x_out h", x, y, w_post, gate, w_pre, x_out, h)
    _check(lib().moe_block_norm(xp, _op_code(x, "x"), yp, MOE_F32 if y is None else _op_code(y, "y"), wp, gp, mode, np_,
                                w_code, T, H, eps, res_scale, op, hp, _op_stream(dev, stream)))


def moe_block_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(lib().moe_block_norm_backward_workspace_size(T, H))


def moe_block_norm_backward(x, y, w_post, gate, w_pre, dx_out, dh, dx, dy, dw_post, dgate, dw_pre, eps: float,
                            res_scale: float = 1.0, ws=None, stream=None):
    """The gradients of moe_block_norm's outputs with respect to x, y and the channel vectors (fp32)."""
    dev = _op_device()
    shape, mode, w_code = _norm_shapes(x, y, w_post, gate, w_pre)
    T, H = shape
    for name, d in (("dx_out", dx_out), ("dh", dh), ("dx", dx)):
        _norm_like(d, shape, x.dtype, name)
    if y is not None:
        _norm_like(dy, shape, y.dtype, "dy")
    for name, d, w in (("dw_post", dw_post, w_post), ("dgate", dgate, gate), ("dw_pre", dw_pre, w_pre)):
        if (d is None) != (w is None) or (d is not None and (d.dtype != _F32 or d.shape != w.shape)):
            raise ValueError(f"{name} must be float32 with the shape of its weight, and None without one")
    xp, yp, wp, gp, np_, op, hp, dxp, dyp, d0, d1, d2, sp = _op_ptrs(
        dev, "x y w_post gate w_pre dx_out dh dx dy dw_post dgate dw_pre ws", x, y, w_post, gate, w_pre, dx_out, dh, dx,
        dy, dw_post, dgate, dw_pre, ws)
    _check(lib().moe_block_norm_backward(
        xp, _op_code(x, "x"), yp, MOE_F32 if y is None else _op_code(y, "y"), wp, gp, mode, np_, w_code, T, H, eps,
        res_scale, op, hp, dxp, dyp, d0, d1, d2, sp, 0 if ws is None else ws.numel() * ws.element_size(),
        _op_stream(dev, stream)))


def _swiglu_shapes(gu, slot_offsets, **halves) -> tuple:
    shape, dtype = gu.shape, gu.dtype
    if len(shape) != 2 or shape[1] % 2:
        raise ValueError("gu must be [R, 2 I]")
    R, I = shape[0], shape[1] // 2
    for name, t in halves.items():
        if t is not None and (t.dtype != dtype or t.shape != (R, I)):
            raise ValueError(f"{name} must be [{R}, {I}] of dtype {dtype}")
    S = 0
    if slot_offsets is not None:
        if slot_offsets.dtype != _I32 or slot_offsets.dim() != 1:
            raise ValueError("slot_offsets must be int32 [S + 1]")
        S = slot_offsets.shape[0] - 1
    return R, I, S


def moe_swiglu(gu, h, slot_offsets=None, stream=None):
    """h [R, I] = silu(g) u of rows gu = [g | u]; with slot_offsets only the rows that a slot owns."""
    dev = _op_device()
    R, I, S = _swiglu_shapes(gu, slot_offsets, h=h)
    gp, op, hp = _op_ptrs(dev, "gu slot_offsets h", gu, slot_offsets, h)
    _check(lib().moe_swiglu(gp, _op_code(gu, "gu"), R, I, op, S, hp, _op_stream(dev, stream)))


def moe_swiglu_backward(gu, dh, dgu, h=None, slot_offsets=None, stream=None):
    """dgu [R, 2 I] for given dh [R, I]; h is written again unless None."""
    dev = _op_device()
    R, I, S = _swiglu_shapes(gu, slot_offsets, dh=dh, h=h)
    _norm_like(dgu, gu.shape, gu.dtype, "dgu")
    gp, dp, op, up, hp = _op_ptrs(dev, "gu dh slot_offsets dgu h", gu, dh, slot_offsets, dgu, h)
    _check(lib().moe_swiglu_backward(gp, dp, _op_code(gu, "gu"), R, I, op, S, up, hp, _op_stream(dev, stream)))


# ------------------------------------------------------------ host leg

HOST_LIB_PATH = os.path.join(_HERE, "libqmoe_host.so")
_host_lib = None


def host_lib() -> ctypes.CDLL:
    """libqmoe_host.so: the CPU expert FFN for the pairs the card does not
    hold, and the adaptive residency policy (include/qmoe_host.h)."""
    global _host_lib
    if _host_lib is None:
        if not os.path.exists(HOST_LIB_PATH):
            raise ImportError(f"{HOST_LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(HOST_LIB_PATH)
        vp = ctypes.c_void_p
        i32 = ctypes.c_int
        L.moe_host_leg.argtypes = [i32, vp, i32, i32, i32, vp, i32, vp, vp, vp, i32, vp, i32]
        L.moe_host_leg.restype = i32
        L.moe_host_last_error.restype = ctypes.c_char_p
        L.moe_residency_update_scores.argtypes = [vp, vp, i32, i32]
        L.moe_residency_update_scores.restype = i32
        L.moe_residency_plan.argtypes = [vp, i32, vp, i32, ctypes.c_uint64, vp, vp, vp]
        L.moe_residency_plan.restype = i32
        _host_lib = L
    return _host_lib


def moe_host_leg(fmt: int, expert_blobs, H: int, I: int, x: np.ndarray, host_token, host_expert, host_weight,
                 threads: int = 0, out: np.ndarray | None = None) -> np.ndarray:
    """y_host [T, H] fp32 of the listed (token, expert, weight) pairs.
    expert_blobs: E entries, each a canonical blob (uint8 array) or None."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    T = x.shape[0]
    tok = np.ascontiguousarray(host_token, dtype=np.int32)
    exp = np.ascontiguousarray(host_expert, dtype=np.int32)
    wt = np.ascontiguousarray(host_weight, dtype=np.float32)
    if not (tok.shape == exp.shape == wt.shape) or tok.ndim != 1:
        raise ValueError("host_token, host_expert and host_weight must be 1-D of equal length")
    E = len(expert_blobs)
    keep = []
    ptrs = (ctypes.c_void_p * max(E, 1))()
    for e, b in enumerate(expert_blobs):
        if b is not None:
            b = np.ascontiguousarray(b, dtype=np.uint8)
            keep.append(b)
            ptrs[e] = b.ctypes.data
    y = np.empty((T, H), dtype=np.float32) if out is None else out
    if y.shape != (T, H) or y.dtype != np.float32 or not y.flags.c_contiguous:
        raise ValueError("out must be a contiguous float32 [T, H] array")
    st = host_lib().moe_host_leg(fmt, ctypes.cast(ptrs, ctypes.c_void_p), E, H, I, x.ctypes.data, T,
                                 tok.ctypes.data, exp.ctypes.data, wt.ctypes.data, int(tok.size), y.ctypes.data,
                                 int(threads))
    if st != 0:
        raise QmoeError(st, host_lib().moe_host_last_error().decode())
    return y


RESIDENCY_FRAC_BITS = 16  # MOE_RESIDENCY_FRAC_BITS


def moe_residency_update_scores(score: np.ndarray, window, decay_shift: int) -> np.ndarray:
    """score (uint64 [E], updated in place) <- score - (score >> decay_shift)
    + (window << 16); window: uint32 [E] pairs routed since the last update."""
    if score.dtype != np.uint64 or score.ndim != 1 or not score.flags.c_contiguous:
        raise ValueError("score must be a contiguous uint64 [E] array")
    win = np.ascontiguousarray(window, dtype=np.uint32)
    if win.shape != score.shape:
        raise ValueError("window must have the shape of score")
    st = host_lib().moe_residency_update_scores(score.ctypes.data, win.ctypes.data, int(score.size), int(decay_shift))
    if st != 0:
        raise QmoeError(st, host_lib().moe_host_last_error().decode())
    return score


def moe_residency_plan(score, slot_of_expert, max_swaps: int, margin: int = 0) -> tuple[list, list]:
    """(incoming, outgoing) experts of one layer's swap plan."""
    sc = np.ascontiguousarray(score, dtype=np.uint64)
    soe = np.ascontiguousarray(slot_of_expert, dtype=np.int32)
    if sc.ndim != 1 or soe.shape != sc.shape:
        raise ValueError("score and slot_of_expert must be 1-D of equal length")
    m = max(int(max_swaps), 0)
    inc = np.zeros(max(m, 1), dtype=np.int32)
    out = np.zeros(max(m, 1), dtype=np.int32)
    n = ctypes.c_int(0)
    st = host_lib().moe_residency_plan(sc.ctypes.data, int(sc.size), soe.ctypes.data, int(max_swaps), int(margin),
                                       inc.ctypes.data, out.ctypes.data, ctypes.byref(n))
    if st != 0:
        raise QmoeError(st, host_lib().moe_host_last_error().decode())
    return inc[:n.value].tolist(), out[:n.value].tolist()


def moe_timer_begin(stage: int, capacity: int) -> None:
    _check(lib().moe_timer_begin(stage, capacity))


def moe_timer_read(stage: int, capacity: int) -> np.ndarray:
    """Kernel milliseconds of each launch timed so far (the timer stays armed)."""
    out = np.zeros(max(int(capacity), 1), dtype=np.float32)
    n = ctypes.c_int(0)
    _check(lib().moe_timer_read(stage, out.ctypes.data, int(capacity), ctypes.byref(n)))
    return out[:min(n.value, int(capacity))].copy()


def moe_hbm_read_probe(buf, waves: int, depth: int, sink, stream=None) -> int:
    """One pass of the streaming-read probe over the device tensor buf; returns the bytes read."""
    if sink.numel() * sink.element_size() < 256 * int(waves):
        raise ValueError(f"sink holds fewer than waves x 64 words ({waves} waves)")
    n = ctypes.c_size_t(0)
    _check(lib().moe_hbm_read_probe(_dev(buf, name="buf"), buf.numel() * buf.element_size(), int(waves), int(depth),
                                    _dev(sink, name="sink"), ctypes.byref(n),
                                    _stream(stream)))
    return n.value


PREFILL_PROBE_OUT_FLOATS = 131072  # MOE_PREFILL_PROBE_OUT_FLOATS


def moe_prefill_inner_probe(variant: int, sub_blocks: int, out, stream=None) -> float:
    """One launch of the prefill inner-loop probe (variant 0: bf16
    dequantization + bf16 MFMA; 1: int8 MFMA + fp32 rescaling per
    sub-block; 2: variant 1 with two int8 activation planes); returns the
    flops the launch stands for."""
    import torch
    ptr = _dev(out, (torch.float32,), name="out")
    _check(lib().moe_prefill_inner_probe(int(variant), int(sub_blocks), ptr, out.numel(), _stream(stream)))
    return 1024.0 * int(sub_blocks) * 2 * 256 * 64 * 32


def moe_timer_end(stage: int) -> tuple[float, int]:
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int(0)
    _check(lib().moe_timer_end(stage, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
