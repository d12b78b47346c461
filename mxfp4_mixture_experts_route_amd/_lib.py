"""ctypes binding of libmoe_mx4.so: the C ABI declared in include/moe_mx4.h, same names.

Argument marshalling only: each function checks tensor dtypes/devices, allocates missing
outputs with torch (device memory is PyTorch's job), and calls the C entry point on the current
HIP stream. Every step of the chain runs in the library's kernels; there is no fallback — if the
library is missing, loading fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# the in-tree build; MOE_MX4_LIB names another build of the same sources (e.g. a sanitized one)
LIB_PATH = os.environ.get("MOE_MX4_LIB") or os.path.join(PKG, "libmoe_mx4.so")

MOE_OK, MOE_EINVAL, MOE_ESHAPE, MOE_EALIGN, MOE_ELAUNCH = 0, 1, 2, 3, 4
MOE_ACT_NONE, MOE_ACT_SWIGLU_OAI, MOE_ACT_SWIGLU_OAI_MX8 = 0, 1, 2
MOE_MAX_K, MOE_MAX_E, MOE_MAX_TILE_M = 16, 1024, 256

EXPORTS = ("moe_strerror", "moe_mpad_max", "moe_route_topk", "moe_bucket", "mx4_pack_experts",
           "mx4_moe_gemv", "mx4_moe_gemm", "moe_combine", "mx4_moe_decode", "moe_timing_arm",
           "moe_timing_read", "mx8_quantize", "mx4_moe_gemm_mx8", "moe_router",
           "mx4_moe_decode_persistent", "mx4_moe_decode_persistent_static", "moe_probe_read",
           "moe_probe_mfma_bf16", "i8_packed_bytes", "i8_pack_experts", "i8_quantize", "i8_gemm",
           "i8_linear", "i8_moe_gemm", "i8_moe_decode")
MOE_BF16, MOE_F16, MOE_F32 = 0, 1, 2
MOE_I8_MAX_K = 65536
MOE_DECODE_WS_WORDS = 544
MOE_ROUTER_MAX_ROUTED = 16384
MOE_ROUTER_WS_WORDS = 67584
MOE_MX8_GEMM_MAX_K = 4096


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({strerror(status)})")


class Mx4ExpertsC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("E", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int)]


class I8ExpertsC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("E", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("glu", ctypes.c_int)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library once; raises if it has not been built."""
    global _lib
    if _lib is None:
        # torch first: the library and torch must share one HIP runtime. Both runtimes carry the
        # soname libamdhip64.so.7, and the process keeps whichever is loaded first; loaded
        # first, the library (RUNPATH: the system ROCm) would put torch on a runtime other than
        # the one it ships with, and launches then fail (launches rejected, then a crash in
        # torch's own copies)
        _torch()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mxfp4_mixture_experts_route_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_strerror.argtypes = [ci]
        L.moe_mpad_max.restype = i64
        L.moe_mpad_max.argtypes = [i64, ci, ci, ci]
        L.moe_route_topk.restype = ci
        L.moe_route_topk.argtypes = [vp, i64, ci, ci, vp, vp, vp]
        L.moe_bucket.restype = ci
        L.moe_bucket.argtypes = [vp, i64, ci, ci, ci, i64, vp, vp, vp, vp, vp]
        L.mx4_pack_experts.restype = ci
        L.mx4_pack_experts.argtypes = [vp, vp, ci, ci, ci, vp, vp, vp]
        proj = [vp, vp, i64, ctypes.POINTER(Mx4ExpertsC), vp, vp, ci, i64, ci, cf, cf, vp, vp]
        for name in ("mx4_moe_gemv", "mx4_moe_gemm"):
            getattr(L, name).restype = ci
            getattr(L, name).argtypes = proj
        L.moe_combine.restype = ci
        L.moe_combine.argtypes = [vp, i64, vp, vp, i64, ci, ci, vp, vp]
        L.moe_timing_arm.restype = ci
        L.moe_timing_arm.argtypes = [ci]
        L.moe_timing_read.restype = ci
        L.moe_timing_read.argtypes = [ctypes.POINTER(ctypes.c_float), ci]
        pe = ctypes.POINTER(Mx4ExpertsC)
        L.mx4_moe_decode.restype = ci
        L.mx4_moe_decode.argtypes = [vp, vp, i64, ci, ci, pe, pe, cf, cf,
                                     vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.mx4_moe_decode_persistent.restype = ci
        L.mx4_moe_decode_persistent.argtypes = [vp, vp, i64, ci, ci, pe, pe, cf, cf, vp, vp, vp,
                                                vp, vp, vp, vp, vp, vp, vp, ci, vp]
        L.mx4_moe_decode_persistent_static.restype = ci
        L.mx4_moe_decode_persistent_static.argtypes = [vp, vp, i64, ci, ci, pe, pe, cf, cf, vp,
                                                       vp, vp, vp, vp, vp, vp, vp, vp, ci, vp]
        L.moe_router.restype = ci
        L.moe_router.argtypes = [vp, vp, vp, i64, ci, ci, ci, ci, i64, vp, vp, vp, vp, vp, vp,
                                 vp, vp, vp]
        L.mx8_quantize.restype = ci
        L.mx8_quantize.argtypes = [vp, vp, i64, ci, vp, vp, vp]
        L.mx4_moe_gemm_mx8.restype = ci
        L.mx4_moe_gemm_mx8.argtypes = [vp, vp, vp, i64, ctypes.POINTER(Mx4ExpertsC), vp, vp, ci,
                                       i64, ci, cf, cf, vp, vp, vp]
        L.moe_probe_read.restype = ci
        L.moe_probe_read.argtypes = [vp, i64, vp, ci, vp]
        L.moe_probe_mfma_bf16.restype = ci
        L.moe_probe_mfma_bf16.argtypes = [ci, ci, vp, vp]
        p8 = ctypes.POINTER(I8ExpertsC)
        L.i8_packed_bytes.restype = i64
        L.i8_packed_bytes.argtypes = [ci, ci, ci, ci]
        L.i8_pack_experts.restype = ci
        L.i8_pack_experts.argtypes = [vp, ci, ci, ci, ci, vp, vp]
        L.i8_quantize.restype = ci
        L.i8_quantize.argtypes = [vp, ci, i64, vp, i64, ci, vp, vp, vp]
        L.i8_gemm.restype = ci
        L.i8_gemm.argtypes = [vp, vp, i64, p8, vp, ci, i64, vp]
        L.i8_linear.restype = ci
        L.i8_linear.argtypes = [vp, ci, i64, i64, p8, vp, vp, vp, ci, i64, vp]
        L.i8_moe_gemm.restype = ci
        L.i8_moe_gemm.argtypes = [vp, vp, vp, i64, p8, vp, vp, ci, i64, ci, cf, cf, vp, vp]
        L.i8_moe_decode.restype = ci
        L.i8_moe_decode.argtypes = [vp, vp, i64, ci, ci, p8, p8, cf, cf, vp, vp, vp, vp, vp, vp, vp,
                                    ci, vp]
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().moe_strerror(int(status)).decode()


def moe_mpad_max(T: int, k: int, E: int, tile_m: int) -> int:
    return int(lib().moe_mpad_max(int(T), int(k), int(E), int(tile_m)))


# ---------------------------------------------------------------------------------------------
# torch-facing wrappers
# ---------------------------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, dtype, name):
    torch = _torch()
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise TypeError(f"{name}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    del torch


def _call(fn: str, *args):
    st = getattr(lib(), fn)(*args)
    if st != MOE_OK:
        raise MoeError(fn, st)


class MX4Experts:
    """A device-resident MXFP4 expert stack in the chunked layout the projections read.

    Built from the checkpoint (row-major) layout — q u8 [E][N][K/2], s u8 [E][N][K/32] — with one
    mx4_pack_experts call on the current stream; bias f32 [E][N] or None. Holds the tensors alive
    and the C descriptor."""

    def __init__(self, q, s, bias=None, stream=None):
        torch = _torch()
        _check(q, torch.uint8, "q")
        _check(s, torch.uint8, "s")
        E, N, half_k = q.shape
        K = half_k * 2
        if tuple(s.shape) != (E, N, K // 32):
            raise ValueError(f"s: expected shape {(E, N, K // 32)}, got {tuple(s.shape)}")
        if bias is not None:
            _check(bias, torch.float32, "bias")
            if tuple(bias.shape) != (E, N):
                raise ValueError(f"bias: expected shape {(E, N)}")
        qp = torch.empty_like(q)
        sp = torch.empty((E, scale_row_bytes(K) // 16, N, 16), dtype=torch.uint8, device=q.device)
        _call("mx4_pack_experts", _ptr(q), _ptr(s), E, N, K, _ptr(qp), _ptr(sp), _stream(stream))
        self.q, self.s, self.bias = qp, sp, bias
        self.E, self.N, self.K = E, N, K
        self.c = Mx4ExpertsC(qp.data_ptr(), sp.data_ptr(),
                             None if bias is None else bias.data_ptr(), E, N, K)

    @classmethod
    def from_numpy(cls, d: dict, device="cuda"):
        torch = _torch()
        q = torch.from_numpy(np_contig(d["q"])).to(device)
        s = torch.from_numpy(np_contig(d["s"])).to(device)
        b = None if d.get("bias") is None else torch.from_numpy(np_contig(d["bias"])).to(device)
        return cls(q, s, b)

    @property
    def nbytes(self) -> int:
        return self.q.numel() + self.s.numel()


def np_contig(a):
    import numpy as np
    a = np.ascontiguousarray(a)
    return a if a.flags.writeable else a.copy()


def scale_row_bytes(K: int) -> int:
    """K/32 padded to a multiple of 16: the scale bytes per row of the chunked layout (in
    groups of 16) and the pitch of MXFP8 scale rows."""
    return (K // 32 + 15) // 16 * 16


def mx4_pack_experts(q, s, q_dst=None, s_dst=None, stream=None):
    """Checkpoint-layout MXFP4 stack -> chunked layout: q_dst like q, s_dst u8 [E][SP/16][N][16]
    (scale groups of 16 blocks, all rows of a group together)."""
    torch = _torch()
    _check(q, torch.uint8, "q")
    _check(s, torch.uint8, "s")
    E, N, half_k = q.shape
    q_dst = torch.empty_like(q) if q_dst is None else q_dst
    if s_dst is None:
        s_dst = torch.empty((E, scale_row_bytes(half_k * 2) // 16, N, 16), dtype=torch.uint8,
                            device=q.device)
    _call("mx4_pack_experts", _ptr(q), _ptr(s), E, N, half_k * 2, _ptr(q_dst), _ptr(s_dst),
          _stream(stream))
    return q_dst, s_dst


def moe_route_topk(logits, k: int, ids=None, w=None, stream=None):
    """ids i32 [T][k], w f32 [T][k] = top-k routing of f32 logits [T][E]."""
    torch = _torch()
    _check(logits, torch.float32, "logits")
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device) if ids is None else ids
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device) if w is None else w
    _call("moe_route_topk", _ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream(stream))
    return ids, w


def moe_router(x, w_r, b_r, k: int, tile_m: int, ws, mpad_max: int | None = None,
               want_logits: bool = True, out=None, stream=None):
    """Router projection + top-k + bucket in one launch. x bf16 [T][D], w_r bf16 [E][D], b_r f32
    [E] or None, ws an int32/uint32 device tensor of MOE_ROUTER_WS_WORDS elements, zero before
    its first use and then left to the library (word 0 is left zero). Returns a dict: logits (if
    want_logits), ids, w, counts, basep, row_tok, pos, mpad."""
    torch = _torch()
    _check(x, torch.bfloat16, "x")
    _check(w_r, torch.bfloat16, "w_r")
    if b_r is not None:
        _check(b_r, torch.float32, "b_r")
    T, D = x.shape
    E = w_r.shape[0]
    if mpad_max is None:
        mpad_max = moe_mpad_max(T, k, E, tile_m)
    dev = x.device
    o = dict(out or {})
    shapes = {"ids": ((T, k), torch.int32), "w": ((T, k), torch.float32),
              "counts": ((E,), torch.int32), "basep": ((E + 1,), torch.int32),
              "row_tok": ((mpad_max,), torch.int32), "pos": ((T, k), torch.int32)}
    if want_logits:
        shapes["logits"] = ((T, E), torch.float32)
    for key, (shape, dt) in shapes.items():
        if key not in o:
            o[key] = torch.empty(shape, dtype=dt, device=dev)
    _call("moe_router", _ptr(x), _ptr(w_r), _ptr(b_r), T, D, E, k, tile_m, mpad_max,
          _ptr(o.get("logits")), _ptr(o["ids"]), _ptr(o["w"]), _ptr(o["counts"]), _ptr(o["basep"]),
          _ptr(o["row_tok"]), _ptr(o["pos"]), _ptr(ws), _stream(stream))
    o["mpad"] = mpad_max
    return o


def moe_bucket(ids, E: int, tile_m: int, mpad_max: int | None = None, out=None, stream=None):
    """(counts [E], basep [E+1], row_tok [mpad_max], pos [T][k]) of i32 ids [T][k]."""
    torch = _torch()
    _check(ids, torch.int32, "ids")
    T, k = ids.shape
    if mpad_max is None:
        mpad_max = moe_mpad_max(T, k, E, tile_m)
    if out is None:
        dev = ids.device
        out = (torch.empty(E, dtype=torch.int32, device=dev),
               torch.empty(E + 1, dtype=torch.int32, device=dev),
               torch.empty(mpad_max, dtype=torch.int32, device=dev),
               torch.empty((T, k), dtype=torch.int32, device=dev))
    counts, basep, row_tok, pos = out
    _call("moe_bucket", _ptr(ids), T, k, E, tile_m, mpad_max, _ptr(counts), _ptr(basep),
          _ptr(row_tok), _ptr(pos), _stream(stream))
    return counts, basep, row_tok, pos


def _projection(fn, a, a_row, w: MX4Experts, counts, basep, tile_m, mpad_max, act, alpha, limit,
                out, stream):
    torch = _torch()
    _check(a, torch.int16 if a.dtype == torch.int16 else torch.bfloat16, "a")
    if a_row is not None:
        _check(a_row, torch.int32, "a_row")
    _check(counts, torch.int32, "counts")
    _check(basep, torch.int32, "basep")
    if out is None:
        if act == MOE_ACT_SWIGLU_OAI:
            out = torch.empty((mpad_max, w.N // 2), dtype=torch.bfloat16, device=a.device)
        else:
            out = torch.empty((mpad_max, w.N), dtype=torch.float32, device=a.device)
    _call(fn, _ptr(a), _ptr(a_row), a.shape[0], ctypes.byref(w.c), _ptr(counts), _ptr(basep),
          tile_m, mpad_max, act, float(alpha), float(limit), _ptr(out), _stream(stream))
    return out


def mx4_moe_gemv(a, a_row, w, counts, basep, tile_m, mpad_max, act=MOE_ACT_NONE, alpha=1.702,
                 limit=7.0, out=None, stream=None):
    return _projection("mx4_moe_gemv", a, a_row, w, counts, basep, tile_m, mpad_max, act, alpha,
                       limit, out, stream)


def mx4_moe_gemm(a, a_row, w, counts, basep, tile_m, mpad_max, act=MOE_ACT_NONE, alpha=1.702,
                 limit=7.0, out=None, stream=None):
    return _projection("mx4_moe_gemm", a, a_row, w, counts, basep, tile_m, mpad_max, act, alpha,
                       limit, out, stream)


def mx8_quantize(a, live=None, out=None, stream=None):
    """MXFP8 rows of bf16 rows a [rows][K]: (q u8 [rows][K] E4M3, s u8 [rows][SP] e8m0 with
    SP = roundup(K/32, 16), padding 0). Rows with live[r] < 0 are left unwritten."""
    torch = _torch()
    _check(a, torch.bfloat16, "a")
    if live is not None:
        _check(live, torch.int32, "live")
    rows, K = a.shape
    if out is None:
        out = (torch.empty((rows, K), dtype=torch.uint8, device=a.device),
               torch.empty((rows, scale_row_bytes(K)), dtype=torch.uint8, device=a.device))
    q, s = out
    _call("mx8_quantize", _ptr(a), _ptr(live), rows, K, _ptr(q), _ptr(s), _stream(stream))
    return q, s


def mx4_moe_gemm_mx8(aq, as_, a_row, w, counts, basep, tile_m, mpad_max, act=MOE_ACT_NONE,
                     alpha=1.702, limit=7.0, out=None, out_scale=None, stream=None):
    """mx4_moe_gemm over MXFP8 activation rows (aq, as_) from mx8_quantize. With
    MOE_ACT_SWIGLU_OAI_MX8 the SwiGLU rows come out as MXFP8 rows: returns (q, s)."""
    torch = _torch()
    _check(aq, torch.uint8, "aq")
    _check(as_, torch.uint8, "as")
    if a_row is not None:
        _check(a_row, torch.int32, "a_row")
    _check(counts, torch.int32, "counts")
    _check(basep, torch.int32, "basep")
    if act == MOE_ACT_SWIGLU_OAI_MX8:
        F = w.N // 2
        if out is None:
            out = torch.empty((mpad_max, F), dtype=torch.uint8, device=aq.device)
        if out_scale is None:
            out_scale = torch.empty((mpad_max, scale_row_bytes(F)), dtype=torch.uint8,
                                    device=aq.device)
    elif out is None:
        if act == MOE_ACT_SWIGLU_OAI:
            out = torch.empty((mpad_max, w.N // 2), dtype=torch.bfloat16, device=aq.device)
        else:
            out = torch.empty((mpad_max, w.N), dtype=torch.float32, device=aq.device)
    _call("mx4_moe_gemm_mx8", _ptr(aq), _ptr(as_), _ptr(a_row), aq.shape[0], ctypes.byref(w.c),
          _ptr(counts), _ptr(basep), tile_m, mpad_max, act, float(alpha), float(limit),
          _ptr(out), _ptr(out_scale), _stream(stream))
    return (out, out_scale) if act == MOE_ACT_SWIGLU_OAI_MX8 else out


def moe_combine(d, pos, w, out=None, stream=None):
    """y f32 [T][D] = slot-order routing-weighted sum of d rows."""
    torch = _torch()
    _check(d, torch.float32, "d")
    _check(pos, torch.int32, "pos")
    _check(w, torch.float32, "w")
    T, k = pos.shape
    D = d.shape[1]
    y = torch.empty((T, D), dtype=torch.float32, device=d.device) if out is None else out
    _call("moe_combine", _ptr(d), d.shape[0], _ptr(pos), _ptr(w), T, k, D, _ptr(y),
          _stream(stream))
    return y


def mx4_moe_decode(logits, x, gate_up: MX4Experts, down: MX4Experts, k: int,
                   alpha: float = 1.702, limit: float = 7.0, want_d: bool = False, out=None,
                   stream=None):
    """Fused decode chain of a few tokens (two launches). Returns a dict with ids, w, counts,
    basep, row_tok, pos (CSR with tile_m = 1), h [T*k][F] and d [T*k][D] in routed-row order
    (d only with want_d), and y [T][D]. `out` may hold preallocated tensors under those keys."""
    torch = _torch()
    _check(logits, torch.float32, "logits")
    _check(x, torch.bfloat16, "x")
    T, E = logits.shape
    D, F = gate_up.K, gate_up.N // 2
    dev = logits.device
    o = dict(out or {})
    shapes = {"ids": ((T, k), torch.int32), "w": ((T, k), torch.float32),
              "counts": ((E,), torch.int32), "basep": ((E + 1,), torch.int32),
              "row_tok": ((T * k,), torch.int32), "pos": ((T, k), torch.int32),
              "h": ((T * k, F), torch.bfloat16), "y": ((T, D), torch.float32)}
    if want_d:
        shapes["d"] = ((T * k, D), torch.float32)
    for key, (shape, dt) in shapes.items():
        if key not in o:
            o[key] = torch.empty(shape, dtype=dt, device=dev)
    _call("mx4_moe_decode", _ptr(logits), _ptr(x), T, E, k, ctypes.byref(gate_up.c),
          ctypes.byref(down.c), float(alpha), float(limit), _ptr(o["ids"]), _ptr(o["w"]),
          _ptr(o["counts"]), _ptr(o["basep"]), _ptr(o["row_tok"]), _ptr(o["pos"]), _ptr(o["h"]),
          _ptr(o.get("d")), _ptr(o["y"]), _stream(stream))
    return o


def mx4_moe_decode_persistent(logits, x, gate_up: MX4Experts, down: MX4Experts, k: int, ws,
                              alpha: float = 1.702, limit: float = 7.0, want_d: bool = False,
                              out=None, max_workgroups: int = 0, stream=None):
    """mx4_moe_decode in one launch. ws: an int32 device tensor of MOE_DECODE_WS_WORDS words,
    zero before its first use and then left to the library (word 3 is the error flag). Same
    outputs as mx4_moe_decode."""
    torch = _torch()
    _check(logits, torch.float32, "logits")
    _check(x, torch.bfloat16, "x")
    T, E = logits.shape
    D, F = gate_up.K, gate_up.N // 2
    dev = logits.device
    o = dict(out or {})
    shapes = {"ids": ((T, k), torch.int32), "w": ((T, k), torch.float32),
              "counts": ((E,), torch.int32), "basep": ((E + 1,), torch.int32),
              "row_tok": ((T * k,), torch.int32), "pos": ((T, k), torch.int32),
              "h": ((T * k, F), torch.bfloat16), "y": ((T, D), torch.float32)}
    if want_d:
        shapes["d"] = ((T * k, D), torch.float32)
    for key, (shape, dt) in shapes.items():
        if key not in o:
            o[key] = torch.empty(shape, dtype=dt, device=dev)
    _call("mx4_moe_decode_persistent", _ptr(logits), _ptr(x), T, E, k, ctypes.byref(gate_up.c),
          ctypes.byref(down.c), float(alpha), float(limit), _ptr(o["ids"]), _ptr(o["w"]),
          _ptr(o["counts"]), _ptr(o["basep"]), _ptr(o["row_tok"]), _ptr(o["pos"]), _ptr(o["h"]),
          _ptr(o.get("d")), _ptr(o["y"]), _ptr(ws), int(max_workgroups), _stream(stream))
    return o


def mx4_moe_decode_persistent_static(logits, x, gate_up: MX4Experts, down: MX4Experts, k: int,
                                     out: dict, alpha: float = 1.702, limit: float = 7.0,
                                     max_workgroups: int = 0, stream=None):
    """mx4_moe_decode_persistent with the library's own workspace (allocates nothing). out: the
    caller's output tensors, keys ids, w, counts, basep, row_tok, pos, h, y and optionally d."""
    torch = _torch()
    _check(logits, torch.float32, "logits")
    _check(x, torch.bfloat16, "x")
    T, E = logits.shape
    _call("mx4_moe_decode_persistent_static", _ptr(logits), _ptr(x), T, E, k,
          ctypes.byref(gate_up.c), ctypes.byref(down.c), float(alpha), float(limit),
          _ptr(out["ids"]), _ptr(out["w"]), _ptr(out["counts"]), _ptr(out["basep"]),
          _ptr(out["row_tok"]), _ptr(out["pos"]), _ptr(out["h"]), _ptr(out.get("d")),
          _ptr(out["y"]), int(max_workgroups), _stream(stream))
    return out


# ---------------------------------------------------------------------------------------------
# 8-bit integer projections
# ---------------------------------------------------------------------------------------------

# These calls take a few microseconds on the GPU, so that the host's share shows: what they need on
# every call is kept in module names, and a check looks into its details when it has failed.
_i8_torch = None
_i8_codes = {}   # torch dtype -> moe_dtype
_i8_fns = {}     # C entry points by name


def _i8_load():
    global _i8_torch
    torch = _torch()
    _i8_codes.update({torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32})
    _i8_torch = torch
    return torch


def _i8_dtype(dtype, name: str) -> int:
    if _i8_torch is None:
        _i8_load()
    code = _i8_codes.get(dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {dtype}")
    return code


def _i8_call(fn: str, dev: int, *args) -> None:
    """The C entry point on the current stream of device `dev`, with that device current: tensors of
    another device than the current one are worked on there."""
    torch = _i8_torch
    f = _i8_fns.get(fn)
    if f is None:
        f = _i8_fns[fn] = getattr(lib(), fn)
    raw = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != MOE_OK:
        raise MoeError(fn, st)


def _i8_on(stream, t):
    """Context of a call on a stream other than the current one. Everything in it belongs to that
    stream, what the call allocates included: scratch that goes back to the allocator when the call
    returns may then only be handed out to work behind it."""
    if stream.device != t.device:
        raise ValueError(f"stream: on {stream.device}, the tensors on {t.device}")
    return _torch().cuda.stream(stream)


def _i8_rows(x, name: str):
    """Checks a device matrix of rows whose elements are contiguous; returns its rows, their
    length and their pitch in elements."""
    if not x.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a matrix of rows, got shape {tuple(shape)}")
    rows, n = shape
    ld, one = x.stride()
    if one != 1 and n > 1:
        raise ValueError(f"{name}: expected rows of contiguous elements")
    if rows < 2:
        return rows, n, n
    if ld < n:
        raise ValueError(f"{name}: rows overlap (stride {ld} of {n} elements)")
    return rows, n, ld


def _i8_check(t, shape, dtype, name: str, dev: int) -> None:
    """Checks a contiguous tensor of this shape and type on device number `dev`."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()
            and t.is_cuda):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError(f"{name}: on device {t.get_device()}, the others on {dev}")


def _i8_weights(w, name: str, dev: int) -> None:
    if not isinstance(w, I8Experts):
        raise TypeError(f"{name}: expected I8Experts, got {type(w).__name__}")
    if w.dev != dev:
        raise ValueError(f"{name}: on device {w.dev}, the others on {dev}")


def i8_pitch(K: int) -> int:
    """Row pitch in bytes of quantized rows of K values: K padded to a multiple of 128."""
    return (K + 127) // 128 * 128


def i8_row_buffers(rows: int, K: int, device="cuda"):
    """Buffers for `rows` quantized rows of K values: (q int8 [rows][i8_pitch(K)], s f32 [rows])."""
    torch = _torch()
    return (torch.empty((rows, i8_pitch(K)), dtype=torch.int8, device=device),
            torch.empty(rows, dtype=torch.float32, device=device))


class I8Experts:
    """A device-resident stack of 8-bit integer matrices with a scale per output channel, in the
    tiled layout that the projections read; a dense projection is a stack of one.

    q int8 [E][N][K] (or [N][K]), s f32 [E][N] (or [N]), bias like s or None. glu: the rows are
    the gate rows, then the up rows of a SwiGLU projection. Built with one i8_pack_experts call
    on the current stream; holds its tensors alive."""

    def __init__(self, q, s, bias=None, glu: bool = False, stream=None):
        torch = _i8_torch or _i8_load()
        if stream is not None:
            with _i8_on(stream, q):
                return self.__init__(q, s, bias, glu)
        _check(q, torch.int8, "q")
        if q.dim() == 2:
            q = q.unsqueeze(0)
        if q.dim() != 3:
            raise ValueError(f"q: expected shape [E][N][K] or [N][K], got {tuple(q.shape)}")
        E, N, K = q.shape
        dev = q.get_device()
        if s.dim() == 1:
            s = s.unsqueeze(0)
        _i8_check(s, (E, N), torch.float32, "s", dev)
        if bias is not None:
            if bias.dim() == 1:
                bias = bias.unsqueeze(0)
            _i8_check(bias, (E, N), torch.float32, "bias", dev)
        glu = int(bool(glu))
        nbytes = int(lib().i8_packed_bytes(E, N, K, glu))
        if nbytes < 0:
            raise MoeError("i8_pack_experts", MOE_ESHAPE)
        qp = torch.empty(nbytes, dtype=torch.int8, device=q.device)
        _i8_call("i8_pack_experts", dev, q.data_ptr(), E, N, K, glu, qp.data_ptr())
        self.q, self.s, self.bias, self.dev = qp, s, bias, dev
        self.E, self.N, self.K, self.glu = E, N, K, glu
        self.c = I8ExpertsC(qp.data_ptr(), s.data_ptr(),
                            None if bias is None else bias.data_ptr(), E, N, K, glu)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def quantized(cls, w, bias=None, glu: bool = False, stream=None):
        """The stack of bf16 / f16 / f32 weights w [E][N][K] (or [N][K]): every output channel is
        quantized as i8_quantize does a row."""
        if stream is not None:
            with _i8_on(stream, w):
                return cls.quantized(w, bias, glu)
        N, K = w.shape[-2], w.shape[-1]
        q, s = i8_quantize(w.reshape(-1, K))
        q = q[:, :K].contiguous().reshape(-1, N, K)
        return cls(q, s.reshape(-1, N), bias, glu)

    @property
    def nbytes(self) -> int:
        return self.q.numel() + 4 * self.s.numel()


def i8_quantize(x, live=None, out=None, stream=None):
    """Quantized rows of bf16 / f16 / f32 rows x [rows][K] (any row stride from K on): (q int8
    [rows][i8_pitch(K)], s f32 [rows]). Rows with live[r] < 0 are left unwritten."""
    if stream is not None:
        with _i8_on(stream, x):
            return i8_quantize(x, live, out)
    rows, K, ld = _i8_rows(x, "x")
    code = _i8_dtype(x.dtype, "x")
    torch = _i8_torch
    dev = x.get_device()
    if live is not None:
        _i8_check(live, (rows,), torch.int32, "live", dev)
    if out is None:
        out = i8_row_buffers(rows, K, x.device)
    else:
        _i8_check(out[0], (rows, i8_pitch(K)), torch.int8, "q", dev)
        _i8_check(out[1], (rows,), torch.float32, "s", dev)
    q, s = out
    _i8_call("i8_quantize", dev, x.data_ptr(), code, ld,
             None if live is None else live.data_ptr(), rows, K, q.data_ptr(), s.data_ptr())
    return q, s


def _i8_dense_out(out, rows: int, w, out_dtype, x, dev: int):
    if out is None:
        out = _torch().empty((rows, w.N), dtype=out_dtype, device=x.device)
        return out, _i8_dtype(out_dtype, "out"), w.N
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    n_rows, n, ld = _i8_rows(out, "out")
    if n_rows != rows or n != w.N:
        raise ValueError(f"out: expected shape {(rows, w.N)}, got {(n_rows, n)}")
    if out.get_device() != dev:
        raise ValueError(f"out: on device {out.get_device()}, the others on {dev}")
    return out, _i8_dtype(out.dtype, "out"), ld


def i8_gemm(aq, as_, w: I8Experts, out_dtype=None, out=None, stream=None):
    """Dense product of quantized rows (aq, as_) with the one matrix of w: out [rows][N] in
    out_dtype (bf16 by default) or in `out` (any row stride)."""
    if stream is not None:
        with _i8_on(stream, aq):
            return i8_gemm(aq, as_, w, out_dtype, out)
    torch = _i8_torch or _i8_load()
    rows, dev = aq.shape[0], aq.get_device()
    _i8_weights(w, "w", dev)
    _i8_check(aq, (rows, i8_pitch(w.K)), torch.int8, "aq", dev)
    _i8_check(as_, (rows,), torch.float32, "as", dev)
    if out is None and out_dtype is None:
        out_dtype = torch.bfloat16
    out, code, ld = _i8_dense_out(out, rows, w, out_dtype, aq, dev)
    _i8_call("i8_gemm", dev, aq.data_ptr(), as_.data_ptr(), rows, w.ref, out.data_ptr(),
             code, ld)
    return out


def i8_linear(x, w: I8Experts, out_dtype=None, out=None, ws=None, stream=None):
    """Dense projection of bf16 / f16 / f32 rows x [rows][K] (any row stride from K on),
    quantized per row on the way: out [rows][N] in out_dtype (x's by default) or in `out`, which
    must not overlap x. ws: scratch of i8_row_buffers(rows, K) (allocated if None); concurrent
    calls need distinct scratch."""
    if stream is not None:
        with _i8_on(stream, x):
            return i8_linear(x, w, out_dtype, out, ws)
    rows, K, ld = _i8_rows(x, "x")
    code = _i8_dtype(x.dtype, "x")
    torch = _i8_torch
    dev = x.get_device()
    _i8_weights(w, "w", dev)
    if K != w.K:
        raise ValueError(f"x: expected rows of {w.K} values, got {K}")
    if ws is None:
        ws = i8_row_buffers(rows, K, x.device)
    else:
        _i8_check(ws[0], (rows, i8_pitch(K)), torch.int8, "ws[0]", dev)
        _i8_check(ws[1], (rows,), torch.float32, "ws[1]", dev)
    if out is None and out_dtype is None:
        out_dtype = x.dtype
    out, ocode, ldo = _i8_dense_out(out, rows, w, out_dtype, x, dev)
    _i8_call("i8_linear", dev, x.data_ptr(), code, ld, rows, w.ref, ws[0].data_ptr(),
             ws[1].data_ptr(), out.data_ptr(), ocode, ldo)
    return out


def i8_moe_gemm(aq, as_, a_row, w: I8Experts, counts, basep, tile_m: int, mpad_max: int,
                act=MOE_ACT_NONE, alpha: float = 1.702, limit: float = 7.0, out=None,
                stream=None):
    """mx4_moe_gemm in 8-bit integers over quantized rows (aq, as_) from i8_quantize: f32
    [mpad_max][N], or with MOE_ACT_SWIGLU_OAI (w built with glu) bf16 [mpad_max][N/2]."""
    if stream is not None:
        with _i8_on(stream, aq):
            return i8_moe_gemm(aq, as_, a_row, w, counts, basep, tile_m, mpad_max, act, alpha,
                               limit, out)
    torch = _i8_torch or _i8_load()
    rows, dev = aq.shape[0], aq.get_device()
    _i8_weights(w, "w", dev)
    _i8_check(aq, (rows, i8_pitch(w.K)), torch.int8, "aq", dev)
    _i8_check(as_, (rows,), torch.float32, "as", dev)
    if a_row is not None:
        _i8_check(a_row, (mpad_max,), torch.int32, "a_row", dev)
    _i8_check(counts, (w.E,), torch.int32, "counts", dev)
    _i8_check(basep, (w.E + 1,), torch.int32, "basep", dev)
    swiglu = act == MOE_ACT_SWIGLU_OAI
    shape = (mpad_max, w.N // 2 if swiglu else w.N)
    dtype = torch.bfloat16 if swiglu else torch.float32
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=aq.device)
    else:
        _i8_check(out, shape, dtype, "out", dev)
    _i8_call("i8_moe_gemm", dev, aq.data_ptr(), as_.data_ptr(),
             None if a_row is None else a_row.data_ptr(), rows, w.ref, counts.data_ptr(),
             basep.data_ptr(), tile_m, mpad_max, act, float(alpha), float(limit), out.data_ptr())
    return out


def i8_moe_decode(logits, x, gate_up: I8Experts, down: I8Experts, k: int, alpha: float = 1.702,
                  limit: float = 7.0, want_d: bool = False, y_dtype=None, out=None, ws=None,
                  stream=None):
    """The whole 8-bit layer of a few tokens (two launches; three for T*k > 16). Returns a dict with
    ids, w [T][k], h bf16 [T*k][F] and d f32 [T*k][D] in routed-row order (d only with want_d), and
    y [T][D] in y_dtype (f32 by default). `out` may hold preallocated tensors under those keys. ws:
    scratch of i8_row_buffers(T*k, F) (allocated if needed); concurrent calls need distinct
    scratch."""
    if stream is not None:
        with _i8_on(stream, x):
            return i8_moe_decode(logits, x, gate_up, down, k, alpha, limit, want_d, y_dtype, out,
                                 ws)
    torch = _i8_torch or _i8_load()
    dev = x.get_device()
    _i8_weights(gate_up, "gate_up", dev)
    _i8_weights(down, "down", dev)
    D, F = gate_up.K, gate_up.N // 2
    if logits.dim() != 2:
        raise ValueError(f"logits: expected shape [T][E], got {tuple(logits.shape)}")
    T, E = logits.shape
    _i8_check(logits, (T, E), torch.float32, "logits", dev)
    _i8_check(x, (T, D), torch.bfloat16, "x", dev)
    o = dict(out) if out else {}
    if y_dtype is None:
        y_dtype = o["y"].dtype if "y" in o else torch.float32
    code = _i8_dtype(y_dtype, "y")
    R = T * k
    new = functools.partial(torch.empty, device=x.device)
    for key, shape, dt in (("ids", (T, k), torch.int32), ("w", (T, k), torch.float32),
                           ("h", (R, F), torch.bfloat16), ("y", (T, D), y_dtype),
                           ("d", (R, D), torch.float32)):
        if key in o:
            _i8_check(o[key], shape, dt, key, dev)
        elif key != "d" or want_d:
            o[key] = new(shape, dtype=dt)
    q = s = None
    if ws is not None:
        _i8_check(ws[0], (R, i8_pitch(F)), torch.int8, "ws[0]", dev)
        _i8_check(ws[1], (R,), torch.float32, "ws[1]", dev)
    elif R > 16 or F > 4096:
        ws = i8_row_buffers(R, F, x.device)
    if ws is not None:
        q, s = ws[0].data_ptr(), ws[1].data_ptr()
    _i8_call("i8_moe_decode", dev, logits.data_ptr(), x.data_ptr(), T, E, k, gate_up.ref,
             down.ref, float(alpha), float(limit), o["ids"].data_ptr(), o["w"].data_ptr(),
             o["h"].data_ptr(), q, s, o["d"].data_ptr() if "d" in o else None, o["y"].data_ptr(),
             code)
    return o


def moe_timing_arm(n: int) -> None:
    """Time the library's next n kernel launches (kernel execution only); 0 disarms."""
    _call("moe_timing_arm", int(n))


def moe_timing_read(n: int) -> list:
    """Durations in ms of the first n launches timed since moe_timing_arm (waits for them)."""
    buf = (ctypes.c_float * max(1, n))()
    _call("moe_timing_read", buf, int(n))
    return [float(buf[i]) for i in range(n)]


def moe_layer(x, logits, gate_up, down, k: int, tile_m: int,
              alpha: float = 1.702, limit: float = 7.0, projection: str = "gemm", stream=None):
    """One routed-expert MoE layer: route -> bucket -> gate_up+SwiGLU -> down -> combine.
    projection: "gemm" or "gemv" (bf16 activations), or "gemm_mx8" (MXFP8 activations on the
    MX-scaled MFMA: x quantized once, h written as MXFP8 rows by the gate_up epilogue; returns
    xq/xs/hq/hs and no bf16 h); these take MX4Experts. "i8" takes I8Experts (gate_up with glu):
    x and h quantized per row (xq/xs/hq/hs are returned too), a stream argument covering
    everything the call does, what it allocates included.
    Returns a dict of every intermediate (device tensors)."""
    if projection not in ("gemm", "gemv", "gemm_mx8", "i8"):
        raise ValueError(f"unknown projection {projection!r}")
    for name, stack in (("gate_up", gate_up), ("down", down)):
        if isinstance(stack, I8Experts) != (projection == "i8"):
            raise TypeError(f"{name}: {type(stack).__name__} in projection {projection!r}")
    if projection == "i8" and stream is not None:   # routing and sums belong to the stream too
        with _i8_on(stream, x):
            return moe_layer(x, logits, gate_up, down, k, tile_m, alpha, limit, projection)
    T, E = logits.shape
    ids, w = moe_route_topk(logits, k, stream=stream)
    mpad = moe_mpad_max(T, k, E, tile_m)
    counts, basep, row_tok, pos = moe_bucket(ids, E, tile_m, mpad, stream=stream)
    extra = {}
    if projection == "gemm_mx8":
        xq, xs = mx8_quantize(x, stream=stream)
        hq, hs = mx4_moe_gemm_mx8(xq, xs, row_tok, gate_up, counts, basep, tile_m, mpad,
                                  MOE_ACT_SWIGLU_OAI_MX8, alpha, limit, stream=stream)
        d = mx4_moe_gemm_mx8(hq, hs, None, down, counts, basep, tile_m, mpad, MOE_ACT_NONE,
                             alpha, limit, stream=stream)
        h = None
        extra = {"xq": xq, "xs": xs, "hq": hq, "hs": hs}
    elif projection == "i8":
        xq, xs = i8_quantize(x, stream=stream)
        h = i8_moe_gemm(xq, xs, row_tok, gate_up, counts, basep, tile_m, mpad,
                        MOE_ACT_SWIGLU_OAI, alpha, limit, stream=stream)
        hq, hs = i8_quantize(h, live=row_tok, stream=stream)
        d = i8_moe_gemm(hq, hs, None, down, counts, basep, tile_m, mpad, MOE_ACT_NONE, alpha,
                        limit, stream=stream)
        extra = {"xq": xq, "xs": xs, "hq": hq, "hs": hs}
    else:
        fn = mx4_moe_gemm if projection == "gemm" else mx4_moe_gemv
        h = fn(x, row_tok, gate_up, counts, basep, tile_m, mpad, MOE_ACT_SWIGLU_OAI, alpha,
               limit, stream=stream)
        d = fn(h, None, down, counts, basep, tile_m, mpad, MOE_ACT_NONE, alpha, limit,
               stream=stream)
    y = moe_combine(d, pos, w, stream=stream)
    return {"ids": ids, "w": w, "mpad": mpad, "counts": counts, "basep": basep,
            "row_tok": row_tok, "pos": pos, "h": h, "d": d, "y": y, **extra}


# ---------------------------------------------------------------------------------------------
# attained-peak probes (measurement only)
# ---------------------------------------------------------------------------------------------

def moe_probe_read(buf, workgroups: int, sink=None, stream=None):
    """Read every byte of the device tensor `buf` once (moe_probe_read); returns the sink."""
    torch = _torch()
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=buf.device)
    _call("moe_probe_read", _ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
          int(workgroups), _stream(stream))
    return sink


def moe_probe_mfma_bf16(workgroups: int, iters: int, sink=None, stream=None):
    """workgroups * 4 * iters * 4 bf16 MFMAs of 32768 flops each (moe_probe_mfma_bf16)."""
    torch = _torch()
    if sink is None:
        sink = torch.zeros(1, dtype=torch.float32, device="cuda")
    _call("moe_probe_mfma_bf16", int(workgroups), int(iters), _ptr(sink), _stream(stream))
    return sink
