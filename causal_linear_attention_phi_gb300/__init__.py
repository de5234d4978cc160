"""Causal linear attention with phi(x) = elu(x) + 1 on GB300 (sm_103a).

A thin ctypes binding over the C ABI of ``libla.so`` (declared in
``include/la.h``).  It only marshals arguments: every step of the computation
runs in the library's CUDA kernels.  PyTorch supplies device memory (outputs
and the workspace come from its caching allocator) and the current stream.  A
call with ``stream=`` runs on that stream and allocates there; ordering it after
the work that made its inputs, and later work after it, is the caller's.
There is no CPU fallback: if the library is not built, importing works but
every call raises ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

__all__ = [
    "LaError", "noncausal_fwd", "noncausal_bwd", "causal_fwd", "causal_bwd", "causal_step_host", "host_step_bytes",
    "recurrent_step", "retention_fwd", "retention_step", "gated_delta_fwd", "gated_delta_bwd", "gated_delta_step",
    "layer_norm_fwd", "layer_norm_bwd", "layer_norm_workspace_bytes", "selftest_bounded_wait", "workspace_bytes",
    "last_error", "clear_error", "timing_enable", "timing_reset", "timing_read", "library", "version",
    "OP_NONCAUSAL_FWD", "OP_CAUSAL_FWD", "OP_CAUSAL_BWD", "OP_NONCAUSAL_BWD", "OP_RETENTION_FWD",
    "OP_GATED_DELTA_FWD", "OP_GATED_DELTA_BWD",
]

OP_NONCAUSAL_FWD, OP_CAUSAL_FWD, OP_CAUSAL_BWD, OP_NONCAUSAL_BWD, OP_RETENTION_FWD = 0, 1, 2, 3, 4
OP_GATED_DELTA_FWD, OP_GATED_DELTA_BWD = 5, 6
LA_F32, LA_BF16 = 0, 1
_STATUS = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_WORKSPACE",
           4: "LA_ERR_CUDA", 5: "LA_ERR_TIMEOUT", 6: "LA_ERR_BOUNDS"}


class LaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__("%s failed: %s%s" % (where, _STATUS.get(status, str(status)),
                                               (" (%s)" % detail) if detail else ""))


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("Dk", ctypes.c_int),
                ("Dv", ctypes.c_int), ("dtype", ctypes.c_int)]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("C", ctypes.c_int), ("dtype", ctypes.c_int)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


_lib = None
_lock = threading.Lock()
_vp = ctypes.c_void_p


def _declare(lib):
    lib.la_workspace_bytes.argtypes = [ctypes.c_int, Shape]
    lib.la_workspace_bytes.restype = ctypes.c_size_t
    lib.la_noncausal_fwd.argtypes = [_vp, _vp, _vp, _vp, Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_causal_fwd.argtypes = [_vp, _vp, _vp, _vp, Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_causal_fwd_fused.argtypes = [_vp, _vp, _vp, _vp, Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_causal_bwd.argtypes = [_vp] * 7 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_host_step_bytes.argtypes = [Shape, ctypes.c_int]
    lib.la_host_step_bytes.restype = ctypes.c_size_t
    lib.la_causal_step_host.argtypes = [_vp] * 8 + [Shape, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    lib.la_noncausal_bwd.argtypes = [_vp] * 7 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_causal_fwd_with_state.argtypes = [_vp] * 6 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_causal_bwd_after_fwd.argtypes = [_vp] * 7 + [Shape, _vp, ctypes.c_size_t, _vp, ctypes.c_size_t, _vp]
    lib.la_recurrent_step.argtypes = [_vp] * 6 + [Shape, _vp]
    lib.la_retention_fwd.argtypes = [_vp] * 6 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_retention_step.argtypes = [_vp] * 6 + [Shape, _vp]
    lib.la_gated_delta_fwd.argtypes = [_vp] * 8 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_gated_delta_bwd.argtypes = [_vp] * 11 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_gated_delta_bwd_with_state.argtypes = [_vp] * 14 + [Shape, _vp, ctypes.c_size_t, _vp]
    lib.la_gated_delta_step.argtypes = [_vp] * 7 + [Shape, _vp]
    lib.la_layer_norm_fwd.argtypes = [_vp] * 6 + [NormShape, ctypes.c_float, _vp]
    lib.la_layer_norm_workspace_bytes.argtypes = [NormShape]
    lib.la_layer_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.la_layer_norm_bwd.argtypes = [_vp] * 8 + [NormShape, _vp, ctypes.c_size_t, _vp]
    lib.la_selftest_bounded_wait.argtypes = [_vp]
    lib.la_selftest_lookback_timeout.argtypes = [_vp] * 4 + [Shape, _vp, ctypes.c_size_t, _vp]
    for f in ("la_causal_step_host", "la_noncausal_fwd", "la_noncausal_bwd", "la_causal_fwd",
              "la_causal_fwd_with_state", "la_causal_bwd", "la_causal_bwd_after_fwd", "la_recurrent_step",
              "la_retention_fwd", "la_retention_step", "la_gated_delta_fwd", "la_gated_delta_bwd",
              "la_gated_delta_bwd_with_state", "la_gated_delta_step", "la_layer_norm_fwd", "la_layer_norm_bwd",
              "la_selftest_bounded_wait", "la_selftest_lookback_timeout", "la_last_error", "la_causal_fwd_fused",
              "la_clear_error", "la_timing_enable", "la_timing_reset"):
        getattr(lib, f).restype = ctypes.c_int
    lib.la_last_error.argtypes = []
    lib.la_clear_error.argtypes = []
    lib.la_status_string.argtypes = [ctypes.c_int]
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_error_detail.argtypes = []
    lib.la_error_detail.restype = ctypes.c_char_p
    lib.la_version.argtypes = []
    lib.la_version.restype = ctypes.c_char_p
    lib.la_timing_enable.argtypes = [ctypes.c_int]
    lib.la_timing_reset.argtypes = []
    lib.la_timing_read.argtypes = [ctypes.POINTER(KernelTime), ctypes.c_int]
    lib.la_timing_read.restype = ctypes.c_int
    return lib


def library(path: str | None = None):
    """The loaded libla (ctypes.CDLL).  Raises RuntimeError if it is not built.

    With LA_DEBUG=1 in the environment the debug build (device-side index checks,
    _lib/libla_debug.so) is loaded instead of the regular one."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or _build.lib_path(os.environ.get("LA_DEBUG", "0") == "1")
            if not os.path.exists(p):
                raise RuntimeError("libla.so is not built (%s); run causal_linear_attention_phi_gb300.build."
                                   "build_library() or __graft_entry__.build()" % p)
            _lib = _declare(ctypes.CDLL(p))
    return _lib


def version() -> str:
    return library().la_version().decode()


def _check(st: int, where: str):
    if st != 0:
        raise LaError(st, where, library().la_error_detail().decode(errors="replace"))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)


def _need_cuda(*ts):
    for t in ts:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("expected CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("expected contiguous tensors")


# The handle of the current stream without building a torch.cuda.Stream for it (3 us of a 20 us call), where
# this PyTorch has that entry.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_ptr(stream=None) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is not None and _get_device is not None:
        return _raw_stream(_get_device())
    return int(torch.cuda.current_stream().cuda_stream)


# What a call allocates comes from the pool of the stream that it runs on: the current stream, or the one given.  Memory of
# the current stream's pool may still be in use by work queued there, which another stream does not wait for, and a
# workspace dropped on return would be handed to the current stream's next tensor under the kernels that use it.
def _elsewhere(stream):
    """`stream` as a torch stream where it is another than the current one, else None."""
    if stream is None or int(stream.cuda_stream) == _stream_ptr():
        return None
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream.cuda_stream))


def _scratch(nbytes, device, stream):
    """Memory that only the call's kernels use."""
    side = _elsewhere(stream)
    if side is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(side):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _handed_out(make, stream):
    """The tensor `make` allocates, which the caller gets: once the caller lets go of it, its memory waits for the current
    stream too."""
    side = _elsewhere(stream)
    if side is None:
        return make()
    with torch.cuda.stream(side):
        t = make()
    t.record_stream(torch.cuda.current_stream())
    return t


def _new_like(t, stream):
    if stream is None:
        return torch.empty_like(t)
    return _handed_out(lambda: torch.empty_like(t), stream)


def _new_f32(shape, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    return _handed_out(lambda: torch.empty(shape, dtype=torch.float32, device=device), stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else ctypes.c_void_p(0)


def _shape4(q, k, v):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k [B,H,N,Dk] and v [B,H,N,Dv]; got %s %s %s" %
                         (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    B, H, N, Dk = q.shape
    return Shape(B, H, N, Dk, v.shape[3], _dtype_code(q))


def workspace_bytes(op: int, B: int, H: int, N: int, Dk: int, Dv: int, dtype: torch.dtype) -> int:
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    code = LA_BF16 if dtype == torch.bfloat16 else LA_F32
    return int(library().la_workspace_bytes(op, Shape(B, H, N, Dk, Dv, code)))


def _workspace(op, s: Shape, device, workspace, stream):
    need = int(library().la_workspace_bytes(op, s))
    if workspace is not None:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a device tensor")
        return workspace, workspace.numel() * workspace.element_size()  # its real size: the library checks it
    if need == 0:
        return None, 0
    return _scratch(need, device, stream), need


def noncausal_fwd(q, k, v, out=None, workspace=None, stream=None):
    """o_i = phi(q_i)^T S / phi(q_i)^T z with S = phi(K)^T V, z = phi(K)^T 1 over all positions."""
    _need_cuda(q, k, v)
    s = _shape4(q, k, v)
    if out is None:
        out = _new_like(v, stream)
    ws, nb = _workspace(OP_NONCAUSAL_FWD, s, q.device, workspace, stream)
    _check(library().la_noncausal_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, _ptr(ws), nb, _stream_ptr(stream)),
           "la_noncausal_fwd")
    return out


def causal_fwd(q, k, v, out=None, workspace=None, stream=None, return_state=False, one_launch=False):
    """Causal linear attention (j <= i) in the chunked form; returns o [B,H,N,Dv].

    With return_state, returns (o, S, z): the fp32 state after the last position
    (S [B,H,Dk,Dv], z [B,H,Dk]), from which recurrent_step continues.  With
    one_launch, runs la_causal_fwd_fused (the same results from one kernel launch
    with a chained scan; bf16 heads of 64 or 128).
    """
    _need_cuda(q, k, v)
    s = _shape4(q, k, v)
    if out is None:
        out = _new_like(v, stream)
    ws, nb = _workspace(OP_CAUSAL_FWD, s, q.device, workspace, stream)
    if not return_state:
        fn = library().la_causal_fwd_fused if one_launch else library().la_causal_fwd
        _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, _ptr(ws), nb, _stream_ptr(stream)),
               "la_causal_fwd_fused" if one_launch else "la_causal_fwd")
        return out
    B, H, _, Dk = q.shape
    S = _new_f32((B, H, Dk, v.shape[-1]), q.device, stream)
    z = _new_f32((B, H, Dk), q.device, stream)
    _check(library().la_causal_fwd_with_state(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), _ptr(z), s, _ptr(ws),
                                              nb, _stream_ptr(stream)), "la_causal_fwd_with_state")
    return out, S, z


def causal_bwd(q, k, v, dout, dq=None, dk=None, dv=None, workspace=None, stream=None, fwd_workspace=None):
    """Gradients (dq, dk, dv) of the causal form for upstream gradient dout.

    With fwd_workspace (the workspace of the causal_fwd call on the same q, k,
    v, unchanged since), the per-segment forward states are read from it
    (la_causal_bwd_after_fwd); otherwise they are recomputed (la_causal_bwd).
    """
    _need_cuda(q, k, v, dout)
    s = _shape4(q, k, v)
    if dout.shape != v.shape or dout.dtype != v.dtype:
        raise ValueError("dout must match v in shape and dtype")
    dq = _new_like(q, stream) if dq is None else dq
    dk = _new_like(k, stream) if dk is None else dk
    dv = _new_like(v, stream) if dv is None else dv
    ws, nb = _workspace(OP_CAUSAL_BWD, s, q.device, workspace, stream)
    if fwd_workspace is None:
        _check(library().la_causal_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), s,
                                       _ptr(ws), nb, _stream_ptr(stream)), "la_causal_bwd")
    else:
        if not fwd_workspace.is_cuda:
            raise ValueError("fwd_workspace must be the device workspace of the forward call")
        fnb = fwd_workspace.numel() * fwd_workspace.element_size()
        _check(library().la_causal_bwd_after_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                                 s, _ptr(fwd_workspace), fnb, _ptr(ws), nb, _stream_ptr(stream)),
               "la_causal_bwd_after_fwd")
    return dq, dk, dv


def noncausal_bwd(q, k, v, dout, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of the non-causal form for upstream gradient dout."""
    _need_cuda(q, k, v, dout)
    s = _shape4(q, k, v)
    if dout.shape != v.shape or dout.dtype != v.dtype:
        raise ValueError("dout must match v in shape and dtype")
    dq = _new_like(q, stream) if dq is None else dq
    dk = _new_like(k, stream) if dk is None else dk
    dv = _new_like(v, stream) if dv is None else dv
    ws, nb = _workspace(OP_NONCAUSAL_BWD, s, q.device, workspace, stream)
    _check(library().la_noncausal_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), s,
                                      _ptr(ws), nb, _stream_ptr(stream)), "la_noncausal_bwd")
    return dq, dk, dv


def host_step_bytes(B: int, H: int, N: int, Dk: int, Dv: int, dtype: torch.dtype, group_heads: int) -> int:
    code = LA_BF16 if dtype == torch.bfloat16 else LA_F32
    return int(library().la_host_step_bytes(Shape(B, H, N, Dk, Dv, code), group_heads))


def causal_step_host(q, k, v, dout, o, dq, dk, dv, group_heads=2, dev_buf=None, stream=None):
    """One causal forward + backward on pinned host tensors (la_causal_step_host).

    q, k, v, dout are read and o, dq, dk, dv written, all pinned CPU tensors of
    the [B,H,N,D] shapes; transfers and kernels are pipelined over groups of
    `group_heads` heads.  Returns after queueing: synchronise the stream before
    reading the outputs.
    """
    for t in (q, k, v, dout, o, dq, dk, dv):
        if t.is_cuda or not t.is_pinned():
            raise ValueError("causal_step_host takes pinned host tensors")
    s = _shape4(q, k, v)
    if dout.shape != v.shape or o.shape != v.shape or dv.shape != v.shape or dq.shape != q.shape or \
            dk.shape != k.shape:
        raise ValueError("output and gradient shapes must match the inputs")
    need = int(library().la_host_step_bytes(s, group_heads))
    if dev_buf is None:
        dev_buf = _scratch(need, torch.device("cuda", torch.cuda.current_device()), stream)
    nb = dev_buf.numel() * dev_buf.element_size()
    _check(library().la_causal_step_host(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(dq), _ptr(dk), _ptr(dv),
                                         s, group_heads, _ptr(dev_buf), nb, _stream_ptr(stream)),
           "la_causal_step_host")
    return o, dq, dk, dv


def recurrent_step(q, k, v, S, z, out=None, stream=None):
    """One decode step: S += phi(k) v^T, z += phi(k) (in place), out = phi(q)^T S / phi(q)^T z."""
    _need_cuda(q, k, v, S, z)
    if q.dim() != 3 or k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("expected q, k [B,H,Dk] and v [B,H,Dv]")
    B, H, Dk = q.shape
    Dv = v.shape[2]
    if S.dtype != torch.float32 or z.dtype != torch.float32 or S.shape != (B, H, Dk, Dv) or z.shape != (B, H, Dk):
        raise ValueError("S must be fp32 [B,H,Dk,Dv] and z fp32 [B,H,Dk]")
    if out is None:
        out = _new_like(v, stream)
    s = Shape(B, H, 1, Dk, Dv, _dtype_code(q))
    _check(library().la_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out), s, _stream_ptr(stream)),
           "la_recurrent_step")
    return out


def _gamma(gamma, H):
    _need_cuda(gamma)
    if gamma.dtype != torch.float32 or gamma.shape != (H,):
        raise ValueError("gamma must be an fp32 CUDA tensor of shape [H] (one decay per head)")
    return gamma


def retention_fwd(q, k, v, gamma, out=None, workspace=None, stream=None, return_state=False):
    """Retention with a constant decay per head: o_t = sum_{j<=t} gamma^(t-j) (q_t . k_j) v_j.

    No feature map and no normaliser; gamma is fp32 [H] on the device.  With
    return_state, returns (o, S): S [B,H,Dk,Dv] fp32 is the state after the
    last position, from which retention_step continues.
    """
    _need_cuda(q, k, v)
    s = _shape4(q, k, v)
    _gamma(gamma, q.shape[1])
    if out is None:
        out = _new_like(v, stream)
    S = None
    if return_state:
        B, H, _, Dk = q.shape
        S = _new_f32((B, H, Dk, v.shape[-1]), q.device, stream)
    ws, nb = _workspace(OP_RETENTION_FWD, s, q.device, workspace, stream)
    _check(library().la_retention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(out), _ptr(S), s, _ptr(ws), nb,
                                      _stream_ptr(stream)), "la_retention_fwd")
    return (out, S) if return_state else out


def retention_step(q, k, v, gamma, S, out=None, stream=None):
    """One retention decode step: S <- gamma S + k v^T (in place), out = S^T q."""
    _need_cuda(q, k, v, S)
    if q.dim() != 3 or k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("expected q, k [B,H,Dk] and v [B,H,Dv]")
    B, H, Dk = q.shape
    Dv = v.shape[2]
    _gamma(gamma, H)
    if S.dtype != torch.float32 or S.shape != (B, H, Dk, Dv):
        raise ValueError("S must be fp32 [B,H,Dk,Dv]")
    if out is None:
        out = _new_like(v, stream)
    s = Shape(B, H, 1, Dk, Dv, _dtype_code(q))
    _check(library().la_retention_step(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(S), _ptr(out), s,
                                       _stream_ptr(stream)), "la_retention_step")
    return out


# The entry points below are called once per decoded token, where the time of the call itself counts: the checks
# are written out over plain attributes, pointers go to ctypes as integers.
_DTYPE_CODE = {torch.float32: LA_F32, torch.bfloat16: LA_BF16}


def _p(t):
    return None if t is None else t.data_ptr()


def _result(t, like, what, stream):
    """A caller's output tensor, checked against what it receives; a new one if None."""
    if t is None:
        return _new_like(like, stream)
    _need_cuda(t)
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError("%s must be %s of shape %s" % (what, like.dtype, tuple(like.shape)))
    return t


def _delta_args(q, k, v, g, beta):
    """Checks the inputs of a gated delta call; returns their leading sizes, Dk, Dv and the dtype code."""
    _need_cuda(q, k, v, g, beta)
    qs, vs, dt = q.shape, v.shape, q.dtype
    lead = qs[:-1]
    if k.shape != qs or len(vs) != len(qs) or vs[:-1] != lead:
        raise ValueError("expected q, k [..., Dk] and v [..., Dv]; got %s %s %s" %
                         (tuple(qs), tuple(k.shape), tuple(vs)))
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k, v must share a dtype")
    if g.shape != lead or beta.shape != lead or g.dtype != dt or beta.dtype != dt:
        raise ValueError("g and beta must have the leading sizes %s and the dtype of q" % (tuple(lead),))
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % dt)
    return lead, qs[-1], vs[-1], code


def _state(S, shape, what):
    _need_cuda(S)
    if S.dtype != torch.float32 or S.shape != shape:
        raise ValueError("%s must be fp32 [B,H,Dk,Dv]" % what)


def gated_delta_fwd(q, k, v, g, beta, S0=None, out=None, workspace=None, stream=None, return_state=False):
    """The gated delta rule: S_t = a_t S_(t-1) + k_t u_t^T with a_t = exp(g_t) and
    u_t = beta_t (v_t - a_t S_(t-1)^T k_t); returns o_t = S_t^T q_t, [B,H,N,Dv].

    q, k [B,H,N,Dk], v [B,H,N,Dv], g (log decays) and beta (write strengths) [B,H,N], one dtype.  A g of
    -inf starts the state anew (packed sequences).  S0: the fp32 [B,H,Dk,Dv] state before the first
    position (zero if None).  With return_state, returns (o, S): the fp32 state after the last position, from
    which gated_delta_step or another gated_delta_fwd continues.
    """
    lead, Dk, Dv, code = _delta_args(q, k, v, g, beta)
    if len(lead) != 3:
        raise ValueError("expected q, k [B,H,N,Dk] and v [B,H,N,Dv]")
    B, H, N = lead
    s = Shape(B, H, N, Dk, Dv, code)
    if S0 is not None:
        _state(S0, (B, H, Dk, Dv), "S0")
    out = _result(out, v, "out", stream)
    S = _new_f32((B, H, Dk, Dv), q.device, stream) if return_state else None
    ws, nb = _workspace(OP_GATED_DELTA_FWD, s, q.device, workspace, stream)
    _check(library().la_gated_delta_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(out), _p(S), s, _p(ws), nb,
                                        _stream_ptr(stream)), "la_gated_delta_fwd")
    return (out, S) if return_state else out


def gated_delta_bwd(q, k, v, g, beta, dout, dq=None, dk=None, dv=None, dg=None, dbeta=None, workspace=None,
                    stream=None, S0=None, dS=None, return_dS0=False):
    """Gradients (dq, dk, dv, dg, dbeta) of gated_delta_fwd for upstream gradient dout.

    For a piece of a longer sequence: S0 is the state that the forward was given, dS the gradient of the state
    that it returned (fp32 [B,H,Dk,Dv]; zero if None), and with return_dS0 the gradient of S0 is returned as well,
    last: the dS of the piece before.
    """
    lead, Dk, Dv, code = _delta_args(q, k, v, g, beta)
    if len(lead) != 3:
        raise ValueError("expected q, k [B,H,N,Dk] and v [B,H,N,Dv]")
    _need_cuda(dout)
    if dout.shape != v.shape or dout.dtype != v.dtype:
        raise ValueError("dout must match v in shape and dtype")
    s = Shape(*lead, Dk, Dv, code)
    dq = _result(dq, q, "dq", stream)
    dk = _result(dk, k, "dk", stream)
    dv = _result(dv, v, "dv", stream)
    dg = _result(dg, g, "dg", stream)
    dbeta = _result(dbeta, beta, "dbeta", stream)
    state = (lead[0], lead[1], Dk, Dv)
    for t, what in ((S0, "S0"), (dS, "dS")):
        if t is not None:
            _state(t, state, what)
    dS0 = _new_f32(state, q.device, stream) if return_dS0 else None
    ws, nb = _workspace(OP_GATED_DELTA_BWD, s, q.device, workspace, stream)
    _check(library().la_gated_delta_bwd_with_state(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(dout), _p(dS), _p(dq),
                                                   _p(dk), _p(dv), _p(dg), _p(dbeta), _p(dS0), s, _p(ws), nb,
                                                   _stream_ptr(stream)), "la_gated_delta_bwd_with_state")
    return (dq, dk, dv, dg, dbeta, dS0) if return_dS0 else (dq, dk, dv, dg, dbeta)


def gated_delta_step(q, k, v, g, beta, S, out=None, stream=None):
    """One decode step of the gated delta rule: u = beta (v - a S^T k), S <- a S + k u^T (in place),
    out = S^T q, with a = exp(g).  q, k [B,H,Dk], v [B,H,Dv], g, beta [B,H], S fp32 [B,H,Dk,Dv]."""
    lead, Dk, Dv, code = _delta_args(q, k, v, g, beta)
    if len(lead) != 2:
        raise ValueError("expected q, k [B,H,Dk] and v [B,H,Dv]")
    B, H = lead
    _state(S, (B, H, Dk, Dv), "S")
    out = _result(out, v, "out", stream)
    _check(library().la_gated_delta_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S), _p(out),
                                         Shape(B, H, 1, Dk, Dv, code), _stream_ptr(stream)), "la_gated_delta_step")
    return out


def _norm_args(x, *params):
    """Checks x and its [C] parameters (None: not given); returns the call's shape."""
    _need_cuda(x)
    xs, dt = x.shape, x.dtype
    if not xs:
        raise ValueError("expected x of shape [..., C]")
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % dt)
    C = xs[-1]
    for p in params:
        if p is not None:
            _need_cuda(p)
            if p.shape != xs[-1:] or p.dtype != dt:
                raise ValueError("weight and bias must be [C] of the dtype of x")
    return NormShape(x.numel() // C if C else 0, C, code)


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, stream=None, return_stats=False):
    """Layer norm over the last dimension of x: (x - mean) rstd weight + bias.

    weight and bias are [C] of x's dtype, or None (1 and 0).  With return_stats, returns
    (y, mean, rstd): the fp32 statistics of shape x.shape[:-1] that layer_norm_bwd takes.
    """
    s = _norm_args(x, weight, bias)
    out = _result(out, x, "out", stream)
    mean = rstd = None
    if return_stats:
        mean = _new_f32(x.shape[:-1], x.device, stream)
        rstd = _new_like(mean, stream)
    _check(library().la_layer_norm_fwd(_p(x), _p(weight), _p(bias), _p(out), _p(mean), _p(rstd), s, eps,
                                       _stream_ptr(stream)), "la_layer_norm_fwd")
    return (out, mean, rstd) if return_stats else out


def layer_norm_workspace_bytes(rows: int, C: int, dtype: torch.dtype) -> int:
    if dtype not in _DTYPE_CODE:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    return int(library().la_layer_norm_workspace_bytes(NormShape(rows, C, _DTYPE_CODE[dtype])))


def layer_norm_bwd(x, weight, mean, rstd, dout, dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm_fwd for upstream gradient dout, from its
    statistics.  With weight None (1), dweight and dbias are formed where the caller gives the
    tensor that receives them ([C] of x's dtype; dbias for a norm with a bias alone), else None."""
    s = _norm_args(x, weight)
    _need_cuda(mean, rstd, dout)
    if dout.shape != x.shape or dout.dtype != x.dtype:
        raise ValueError("dout must match x in shape and dtype")
    stats = x.shape[:-1]
    if mean.dtype != torch.float32 or rstd.dtype != torch.float32 or mean.shape != stats or rstd.shape != stats:
        raise ValueError("mean and rstd must be fp32 of shape x.shape[:-1]")
    dx = _result(dx, x, "dx", stream)
    lib = library()
    ws, nb = None, 0
    if weight is not None:
        dweight = _result(dweight, weight, "dweight", stream)
        dbias = _result(dbias, weight, "dbias", stream)
    else:
        for t, what in ((dweight, "dweight"), (dbias, "dbias")):
            if t is None:
                continue
            _need_cuda(t)
            if t.shape != x.shape[-1:] or t.dtype != x.dtype:
                raise ValueError("%s must be %s of shape %s" % (what, x.dtype, tuple(x.shape[-1:])))
    if dweight is not None or dbias is not None:
        if workspace is not None:
            if not workspace.is_cuda:
                raise ValueError("workspace must be a device tensor")
            ws, nb = workspace, workspace.numel() * workspace.element_size()
        else:
            nb = int(lib.la_layer_norm_workspace_bytes(s))
            ws = _scratch(nb, x.device, stream)
    _check(lib.la_layer_norm_bwd(_p(x), _p(weight), _p(mean), _p(rstd), _p(dout), _p(dx), _p(dweight), _p(dbias), s,
                                 _p(ws), nb, _stream_ptr(stream)), "la_layer_norm_bwd")
    return dx, dweight, dbias


def selftest_bounded_wait(stream=None):
    """Launch the bounded-wait self-test (a wait that runs out after about a second and
    records LA_ERR_TIMEOUT in the sticky status word); read it with last_error()."""
    _check(library().la_selftest_bounded_wait(_stream_ptr(stream)), "la_selftest_bounded_wait")


def selftest_lookback_timeout(q, k, v, out=None, workspace=None, stream=None):
    """The one-launch causal forward with segment 0 of head 0 withholding its sums: the
    later segments of that head time out (about a second) and record LA_ERR_TIMEOUT; read
    it with last_error().  Other heads' outputs are complete."""
    _need_cuda(q, k, v)
    s = _shape4(q, k, v)
    if out is None:
        out = _new_like(v, stream)
    ws, nb = _workspace(OP_CAUSAL_FWD, s, q.device, workspace, stream)
    _check(library().la_selftest_lookback_timeout(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, _ptr(ws), nb,
                                                  _stream_ptr(stream)), "la_selftest_lookback_timeout")
    return out


def last_error() -> int:
    """Sticky device-side status (0 = LA_OK); synchronises the device."""
    return int(library().la_last_error())


def clear_error():
    _check(library().la_clear_error(), "la_clear_error")


def timing_enable(on: bool = True):
    _check(library().la_timing_enable(1 if on else 0), "la_timing_enable")


def timing_reset():
    _check(library().la_timing_reset(), "la_timing_reset")


def timing_read() -> dict:
    """{kernel name: (launches, total_ms)} since the last reset."""
    lib = library()
    n = lib.la_timing_read(None, 0)
    buf = (KernelTime * max(n, 1))()
    n = lib.la_timing_read(buf, n)
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n)}
