"""Thin Python binding of the C ABI in include/gla.h (ctypes; argument marshalling only).

Every step of the computation runs in the CUDA library ``libgla_b200.so`` built
in-tree from ``csrc/``.  There is no fallback: if the library is missing or a
call fails, an exception is raised.  PyTorch is used only to own device memory
(inputs, outputs and the workspace) and to name the CUDA stream.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgla_b200.so")

GLA_OK = 0
STATUS = {
    0: "GLA_OK", -1: "GLA_ERR_INVALID_ARG", -2: "GLA_ERR_UNSUPPORTED_SHAPE", -3: "GLA_ERR_MISALIGNED",
    -4: "GLA_ERR_WORKSPACE_TOO_SMALL", -5: "GLA_ERR_CUDA", -6: "GLA_ERR_TIMEOUT", -7: "GLA_ERR_GATE_RANGE",
    -8: "GLA_ERR_NO_DEVICE", -9: "GLA_ERR_INDEX",
}
DTYPE = {torch.bfloat16: 0, torch.float32: 1}
GATE = {"vector": 0, "scalar": 1, "none": 2}
VARIANT = {"auto": 0, "fused": 1, "materialized": 2}
NOALLOC_SCRATCH_BYTES = 64 << 20  # GLA_NOALLOC_SCRATCH_BYTES in include/gla.h

# Every exported symbol of include/gla.h.
EXPORTS = ["gla_workspace_size", "gla_check", "gla_fwd", "gla_bwd", "gla_poll_status", "gla_status_string",
           "gla_timing_enable", "gla_timing_collect", "gla_kernel_name", "gla_build_info", "gla_fwd_noalloc",
           "gla_decode_step", "gla_selftest_timeout", "gla_epilogue_workspace_size", "gla_epilogue_fwd",
           "gla_epilogue_bwd", "gla_fwd_state", "gla_bwd_state", "gla_state_scan", "gla_general_workspace_size",
           "gla_fwd_general", "gla_bwd_general", "gla_poll_status_noalloc", "gla_last_cuda_error",
           "gla_fwd_epilogue", "gla_decay_workspace_size", "gla_decay_fwd", "gla_decay_bwd", "gla_decay_step",
           "gla_layernorm_workspace_size", "gla_layernorm_fwd", "gla_layernorm_bwd"]


class GLAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        extra = ""
        if code == -5:  # GLA_ERR_CUDA: name the CUDA error behind it
            extra = f"; CUDA: {load().gla_last_cuda_error().decode()}"
        super().__init__(f"{where} failed: {STATUS.get(code, code)} ({status_string(code)}{extra})")


class gla_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int), ("dk", ctypes.c_int),
                ("dv", ctypes.c_int), ("dtype", ctypes.c_int), ("gate", ctypes.c_int), ("subchunk", ctypes.c_int),
                ("variant", ctypes.c_int), ("segments", ctypes.c_int), ("flags", ctypes.c_int),
                ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class gla_view(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong),
                ("st", ctypes.c_longlong)]


class gla_decay_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int), ("max_len", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("dtype", ctypes.c_int), ("slots0", ctypes.c_int),
                ("slots1", ctypes.c_int), ("segments", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgla_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} (run chunkwise_linear_rnn_fwd_b200/build.py)")
    lib = ctypes.CDLL(path)
    vp, i, dp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(gla_desc)
    lib.gla_workspace_size.argtypes = [dp, i, i]
    lib.gla_workspace_size.restype = ctypes.c_size_t
    lib.gla_check.argtypes = [dp, i]
    lib.gla_check.restype = i
    lib.gla_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_fwd.restype = i
    lib.gla_fwd_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_fwd_noalloc.restype = i
    lib.gla_poll_status_noalloc.argtypes = [vp]
    lib.gla_poll_status_noalloc.restype = i
    lib.gla_decode_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp]
    lib.gla_decode_step.restype = i
    lib.gla_selftest_timeout.argtypes = [vp, ctypes.c_uint, vp]
    lib.gla_selftest_timeout.restype = i
    f = ctypes.c_float
    lib.gla_epilogue_workspace_size.argtypes = [dp]
    lib.gla_epilogue_workspace_size.restype = ctypes.c_size_t
    lib.gla_epilogue_fwd.argtypes = [dp, vp, vp, vp, vp, f, vp, vp]
    lib.gla_epilogue_fwd.restype = i
    lib.gla_fwd_epilogue.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, i, vp]
    lib.gla_fwd_epilogue.restype = i
    lib.gla_epilogue_bwd.argtypes = [dp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp]
    lib.gla_epilogue_bwd.restype = i
    lib.gla_fwd_state.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_fwd_state.restype = i
    lib.gla_bwd_state.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_bwd_state.restype = i
    lib.gla_state_scan.argtypes = [dp, i, i, i, vp, vp, vp, vp, vp]
    lib.gla_state_scan.restype = i
    lib.gla_general_workspace_size.argtypes = [dp, i, i]
    lib.gla_general_workspace_size.restype = ctypes.c_size_t
    lib.gla_fwd_general.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_fwd_general.restype = i
    lib.gla_bwd_general.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_bwd_general.restype = i
    dd, vw, ll = ctypes.POINTER(gla_decay_desc), vp, ctypes.c_longlong  # vw: a gla_view's address
    lib.gla_decay_workspace_size.argtypes = [dd, i]
    lib.gla_decay_workspace_size.restype = ctypes.c_size_t
    lib.gla_decay_fwd.argtypes = [dd, vw, vw, vw, vp, vp, vp, vp, vw, vp, vp, vp]
    lib.gla_decay_fwd.restype = i
    lib.gla_decay_bwd.argtypes = [dd, vw, vw, vw, vp, vp, vp, vw, vp, vw, vw, vw, vp, vp]
    lib.gla_decay_bwd.restype = i
    lib.gla_decay_step.argtypes = [dd, vw, vw, vw, vp, vp, vp, vw, vp]
    lib.gla_decay_step.restype = i
    lib.gla_layernorm_workspace_size.argtypes = [ll, i]
    lib.gla_layernorm_workspace_size.restype = ctypes.c_size_t
    lib.gla_layernorm_fwd.argtypes = [i, ll, i, vp, ll, vp, vp, f, vp, ll, vp, vp, vp]
    lib.gla_layernorm_fwd.restype = i
    lib.gla_layernorm_bwd.argtypes = [i, ll, i, vp, ll, vp, ll, vp, vp, vp, vp, ll, vp, vp, vp, ctypes.c_size_t, vp]
    lib.gla_layernorm_bwd.restype = i
    lib.gla_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, vp]
    lib.gla_bwd.restype = i
    lib.gla_poll_status.argtypes = [dp, vp]
    lib.gla_poll_status.restype = i
    lib.gla_status_string.argtypes = [i]
    lib.gla_status_string.restype = ctypes.c_char_p
    lib.gla_timing_enable.argtypes = [i]
    lib.gla_timing_enable.restype = i
    lib.gla_timing_collect.argtypes = [i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float)]
    lib.gla_timing_collect.restype = i
    lib.gla_kernel_name.argtypes = [i]
    lib.gla_kernel_name.restype = ctypes.c_char_p
    lib.gla_build_info.argtypes = []
    lib.gla_build_info.restype = ctypes.c_char_p
    lib.gla_last_cuda_error.argtypes = []
    lib.gla_last_cuda_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().gla_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the GLA library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def _on_stream(fn):
    """Run a binding with `stream` (keyword argument) as torch's current stream, so that
    the tensors the binding allocates (outputs the caller did not pass, a temporary
    workspace) belong to the stream the library launches on: the caching allocator
    then cannot hand a temporary workspace to other work while the kernels that use
    it are still queued on that stream."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        stream = kwargs.get("stream")
        if stream is None or stream == torch.cuda.current_stream(stream.device):
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


def _gate_of(log_alpha, gate):
    if gate is not None:
        return gate
    if log_alpha is None:
        return "none"
    return "vector" if log_alpha.dim() == 4 else "scalar"


FLAG_REUSE_PREP = 1
FLAG_SAVE_STATES = 2
FLAG_REUSE_SEGMENTS = 4


def make_desc(B, H, T, dk, dv, dtype, gate, *, subchunk=16, variant="auto", segments=0, flags=0,
              workspace: Optional[torch.Tensor] = None) -> gla_desc:
    d = gla_desc()
    d.B, d.H, d.T, d.dk, d.dv = int(B), int(H), int(T), int(dk), int(dv)
    d.dtype = DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    d.gate = GATE[gate] if isinstance(gate, str) else int(gate)
    d.subchunk = int(subchunk)
    d.variant = VARIANT[variant] if isinstance(variant, str) else int(variant)
    d.segments = int(segments)
    d.flags = int(flags)
    if workspace is not None:
        d.workspace = workspace.data_ptr()
        d.workspace_bytes = workspace.numel() * workspace.element_size()
    return d


def workspace_size(B, H, T, dk, dv, dtype, gate, chunk=64, for_bwd=False, **kw) -> int:
    d = make_desc(B, H, T, dk, dv, dtype, gate, **kw)
    n = load().gla_workspace_size(ctypes.byref(d), int(chunk), int(bool(for_bwd)))
    if n == 0:
        raise GLAError(load().gla_check(ctypes.byref(d), int(chunk)), "gla_workspace_size")
    return int(n)


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A caller-owned workspace (PyTorch memory, 256-byte aligned by the allocator)."""
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device)


@_on_stream
def gla_fwd(q, k, v, log_alpha=None, h0=None, *, chunk=64, gate=None, subchunk=16, variant="auto", segments=0,
            o=None, h_final=None, want_final=True, workspace=None, stream=None, save_states=False,
            reuse_prep=False, reuse_segments=False):
    """Forward.  Returns (o, h_final or None).  See include/gla.h.
    save_states=True: also store the bf16 chunk states in `workspace` (sized for
    the backward) for a following gla_bwd(..., saved_states=True)
    (GLA_FLAG_SAVE_STATES).  reuse_prep / reuse_segments: `workspace` holds the prep
    outputs / segment contributions of a gla_fwd_state call on the same inputs and
    flags (GLA_FLAG_REUSE_PREP, GLA_FLAG_REUSE_SEGMENTS)."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_final is None and want_final:
        h_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    flags = ((FLAG_SAVE_STATES if save_states else 0) | (FLAG_REUSE_PREP if reuse_prep else 0)
             | (FLAG_REUSE_SEGMENTS if reuse_segments else 0))
    if workspace is None:
        workspace = alloc_workspace(workspace_size(B, H, T, dk, dv, q.dtype, gate, chunk, save_states,
                                                   subchunk=subchunk, variant=variant, segments=segments,
                                                   flags=flags), q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, subchunk=subchunk, variant=variant, segments=segments,
                  flags=flags, workspace=workspace)
    r = lib.gla_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(o), _ptr(h_final),
                    int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_fwd")
    return o, h_final


def general_workspace_size(B, H, T, dk, dv, dtype, gate, chunk=64, for_bwd=False) -> int:
    d = make_desc(B, H, T, dk, dv, dtype, gate)
    n = load().gla_general_workspace_size(ctypes.byref(d), int(chunk), int(bool(for_bwd)))
    if n == 0:
        raise GLAError(load().gla_check(ctypes.byref(d), int(chunk)), "gla_general_workspace_size")
    return int(n)


@_on_stream
def gla_fwd_general(q, k, v, log_alpha, log_beta, h0=None, *, chunk=64, gate=None, o=None, h_final=None,
                    want_final=True, workspace=None, stream=None):
    """Forward with the general gate alpha_t^T beta_t (log_beta [B,H,T,d_v]).
    Returns (o, h_final or None).  See include/gla.h."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_final is None and want_final:
        h_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(general_workspace_size(B, H, T, dk, dv, q.dtype, gate, chunk, False), q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, workspace=workspace)
    r = lib.gla_fwd_general(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(log_beta), _ptr(h0),
                            _ptr(o), _ptr(h_final), int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_fwd_general")
    return o, h_final


@_on_stream
def gla_bwd_general(q, k, v, log_alpha, log_beta, do, h0=None, dh_final=None, *, chunk=64, gate=None,
                    want_dh0=True, workspace=None, stream=None):
    """Backward of gla_fwd_general: (dq, dk, dv, dlog_alpha or None, dlog_beta, dh0 or None)."""
    lib = load()
    B, H, T, dk_ = q.shape
    dv_ = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = None if gate == "none" else torch.empty_like(log_alpha)
    dlb = torch.empty_like(log_beta)
    dh0 = torch.empty(B, H, dk_, dv_, dtype=torch.float32, device=q.device) if want_dh0 else None
    if workspace is None:
        workspace = alloc_workspace(general_workspace_size(B, H, T, dk_, dv_, q.dtype, gate, chunk, True), q.device)
    d = make_desc(B, H, T, dk_, dv_, q.dtype, gate, workspace=workspace)
    r = lib.gla_bwd_general(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(log_beta), _ptr(h0),
                            _ptr(do), _ptr(dh_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dla), _ptr(dlb), _ptr(dh0),
                            int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_bwd_general")
    return dq, dk, dv, dla, dlb, dh0


@_on_stream
def gla_fwd_state(q, k, v, log_alpha=None, h0=None, *, chunk=64, gate=None, subchunk=16, segments=0,
                  delta=None, gamma=None, workspace=None, stream=None, save_states=False, reuse_prep=False):
    """Summary of this piece of the sequence: (delta, gamma) = (the state after the
    piece from h0, the product of its gates per key channel).  See include/gla.h.
    save_states: use the workspace layout of gla_fwd(..., save_states=True), so that
    call can reuse the prep outputs and segment contributions left here."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if delta is None:
        delta = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if gamma is None:
        gamma = torch.empty(B, H, dk, dtype=torch.float32, device=q.device)
    flags = (FLAG_SAVE_STATES if save_states else 0) | (FLAG_REUSE_PREP if reuse_prep else 0)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(B, H, T, dk, dv, q.dtype, gate, chunk, bool(flags),
                                                   subchunk=subchunk, segments=segments, flags=flags), q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, subchunk=subchunk, segments=segments, flags=flags,
                  workspace=workspace)
    r = lib.gla_fwd_state(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(delta),
                          _ptr(gamma), int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_fwd_state")
    return delta, gamma


@_on_stream
def gla_bwd_state(q, k, log_alpha, do, dh_final=None, *, chunk=64, gate=None, subchunk=16, segments=0,
                  ddelta=None, gamma=None, want_gamma=True, workspace=None, stream=None, reuse_prep=False):
    """Reverse summary of this piece: (ddelta, gamma or None) = (the state adjoint
    before the piece given dh_final after it, the gate product).  See include/gla.h."""
    lib = load()
    B, H, T, dk = q.shape
    dv = do.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if ddelta is None:
        ddelta = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if gamma is None and want_gamma:
        gamma = torch.empty(B, H, dk, dtype=torch.float32, device=q.device)
    flags = FLAG_REUSE_PREP if reuse_prep else 0
    if workspace is None:
        workspace = alloc_workspace(workspace_size(B, H, T, dk, dv, q.dtype, gate, chunk, True, subchunk=subchunk,
                                                   segments=segments), q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, subchunk=subchunk, segments=segments, flags=flags,
                  workspace=workspace)
    r = lib.gla_bwd_state(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(log_alpha), _ptr(do), _ptr(dh_final), _ptr(ddelta),
                          _ptr(gamma), int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_bwd_state")
    return ddelta, gamma


@_on_stream
def gla_state_scan(gammas, deltas, seg, *, reverse=False, init=None, out=None, stream=None):
    """Fold of gathered piece summaries: gammas [P,B,H,dk], deltas [P,B,H,dk,dv] fp32.
    reverse=False: the state entering piece `seg` (pieces 0 .. seg-1 over init);
    reverse=True: the adjoint leaving piece `seg` (pieces P-1 .. seg+1 over init)."""
    lib = load()
    P, B, H, dk, dv = deltas.shape
    if out is None:
        out = torch.empty(B, H, dk, dv, dtype=torch.float32, device=deltas.device)
    d = make_desc(B, H, 1, dk, dv, torch.bfloat16, "vector")
    r = lib.gla_state_scan(ctypes.byref(d), int(P), int(seg), int(bool(reverse)), _ptr(gammas), _ptr(deltas),
                           _ptr(init), _ptr(out), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_state_scan")
    return out


@_on_stream
def gla_fwd_noalloc(q, k, v, log_alpha=None, h0=None, *, chunk=64, gate=None, subchunk=16, variant="auto",
                    segments=0, o=None, h_final=None, want_final=True, stream=None):
    """Forward without a workspace, for callers that cannot allocate device memory:
    the library uses a fixed scratch array of its own (GLA_NOALLOC_SCRATCH_BYTES,
    shared by all calls; calls must not overlap on the GPU).  Returns (o, h_final)."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_final is None and want_final:
        h_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, subchunk=subchunk, variant=variant, segments=segments)
    r = lib.gla_fwd_noalloc(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(o),
                            _ptr(h_final), int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_fwd_noalloc")
    return o, h_final


def poll_status_noalloc(stream=None) -> int:
    """Synchronise and read/clear the status word of gla_fwd_noalloc's scratch on the
    current device (GLA_OK = 0, GLA_ERR_TIMEOUT = -6, GLA_ERR_GATE_RANGE = -7)."""
    return int(load().gla_poll_status_noalloc(_stream_handle(stream)))


@_on_stream
def gla_decode_step(q, k, v, log_alpha, state, *, gate=None, o=None, stream=None):
    """One recurrent decode step per (batch, head): state <- diag(alpha) state + k^T v
    (in place), o = q state.  q, k [B,H,d_k]; v [B,H,d_v]; log_alpha [B,H,d_k] or
    [B,H] or None; state [B,H,d_k,d_v] fp32.  Returns o [B,H,d_v].  See include/gla.h."""
    lib = load()
    B, H, dk = q.shape
    dv = v.shape[-1]
    if gate is None:
        gate = "none" if log_alpha is None else ("vector" if log_alpha.dim() == 3 else "scalar")
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    d = make_desc(B, H, 1, dk, dv, q.dtype, gate)
    r = lib.gla_decode_step(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(state), _ptr(o),
                            _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_decode_step")
    return o


def epilogue_workspace_size(B, H, T, dv, dtype) -> int:
    """Bytes of the layer epilogue's workspace (status word + dw/db partial sums)."""
    d = make_desc(B, H, T, 1, dv, dtype, "none")
    return int(load().gla_epilogue_workspace_size(ctypes.byref(d)))


@_on_stream
def gla_epilogue_fwd(o, r, w=None, b=None, *, eps=1e-5, y=None, workspace=None, stream=None):
    """y = LayerNorm(o; w, b, eps) * Swish(r) per (batch, head, token) over d_v.
    o, r [B,H,T,d_v]; w, b [d_v] fp32 or None.  See include/gla.h."""
    lib = load()
    B, H, T, dv = o.shape
    if y is None:
        y = torch.empty_like(o)
    if workspace is None:
        workspace = alloc_workspace(256, o.device)
    d = make_desc(B, H, T, 1, dv, o.dtype, "none", workspace=workspace)
    r_ = lib.gla_epilogue_fwd(ctypes.byref(d), _ptr(o), _ptr(r), _ptr(w), _ptr(b), float(eps), _ptr(y),
                              _stream_handle(stream))
    if r_ != GLA_OK:
        raise GLAError(r_, "gla_epilogue_fwd")
    return y


@_on_stream
def gla_fwd_epilogue(q, k, v, log_alpha, r, w=None, b=None, h0=None, *, eps=1e-5, chunk=64, gate=None, subchunk=16,
                     variant="auto", segments=0, o=None, y=None, h_final=None, want_final=True, workspace=None,
                     stream=None, save_states=False, reuse_prep=False):
    """Forward with the layer epilogue fused into its output store.  Returns
    (o, y, h_final or None): o and h_final as gla_fwd, y = LayerNorm(o; w, b, eps)
    * Swish(r).  r [B,H,T,d_v] like v; w, b [d_v] fp32 or None.  See include/gla.h."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if y is None:
        y = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_final is None and want_final:
        h_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    flags = (FLAG_SAVE_STATES if save_states else 0) | (FLAG_REUSE_PREP if reuse_prep else 0)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(B, H, T, dk, dv, q.dtype, gate, chunk, save_states,
                                                   subchunk=subchunk, variant=variant, segments=segments,
                                                   flags=flags), q.device)
    d = make_desc(B, H, T, dk, dv, q.dtype, gate, subchunk=subchunk, variant=variant, segments=segments,
                  flags=flags, workspace=workspace)
    r_ = lib.gla_fwd_epilogue(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(r), _ptr(w),
                              _ptr(b), float(eps), _ptr(o), _ptr(y), _ptr(h_final), int(chunk), _stream_handle(stream))
    if r_ != GLA_OK:
        raise GLAError(r_, "gla_fwd_epilogue")
    return o, y, h_final


@_on_stream
def gla_epilogue_bwd(o, r, dy, w=None, b=None, *, eps=1e-5, want_dwb=True, workspace=None, stream=None):
    """Backward of gla_epilogue_fwd: (do, dr, dw or None, db or None)."""
    lib = load()
    B, H, T, dv = o.shape
    do_, dr = torch.empty_like(o), torch.empty_like(r)
    dw = db = None
    if want_dwb:
        dw = torch.empty(dv, dtype=torch.float32, device=o.device)
        db = torch.empty(dv, dtype=torch.float32, device=o.device)
    if workspace is None:
        workspace = alloc_workspace(epilogue_workspace_size(B, H, T, dv, o.dtype) if want_dwb else 256, o.device)
    d = make_desc(B, H, T, 1, dv, o.dtype, "none", workspace=workspace)
    r_ = lib.gla_epilogue_bwd(ctypes.byref(d), _ptr(o), _ptr(r), _ptr(w), _ptr(b), float(eps), _ptr(dy), _ptr(do_),
                              _ptr(dr), _ptr(dw), _ptr(db), _stream_handle(stream))
    if r_ != GLA_OK:
        raise GLAError(r_, "gla_epilogue_bwd")
    return do_, dr, dw, db


@_on_stream
def gla_bwd(q, k, v, log_alpha, do, h0=None, dh_final=None, *, chunk=64, gate=None, subchunk=16, dq=None, dk=None,
            dv=None, dlog_alpha=None, dh0=None, want_dh0=True, workspace=None, stream=None, reuse_prep=False,
            saved_states=False, reuse_segments=False, segments=0, variant="auto"):
    """Backward.  Returns (dq, dk, dv, dlog_alpha or None, dh0 or None).  See include/gla.h.
    reuse_prep=True: `workspace` holds the prep outputs of a gla_fwd call on the same
    inputs with this workspace (GLA_FLAG_REUSE_PREP).  saved_states=True: it also
    holds the chunk states of a gla_fwd(..., save_states=True) call with the same
    segments and variant (GLA_FLAG_SAVE_STATES).  reuse_segments=True: it holds the
    segment contributions of a gla_bwd_state call (GLA_FLAG_REUSE_SEGMENTS)."""
    lib = load()
    B, H, T, dk_ = q.shape
    dv_ = v.shape[-1]
    gate = _gate_of(log_alpha, gate)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dlog_alpha is None and gate != "none":
        dlog_alpha = torch.empty_like(log_alpha)
    if dh0 is None and want_dh0:
        dh0 = torch.empty(B, H, dk_, dv_, dtype=torch.float32, device=q.device)
    flags = ((FLAG_REUSE_PREP if reuse_prep else 0) | (FLAG_SAVE_STATES if saved_states else 0)
             | (FLAG_REUSE_SEGMENTS if reuse_segments else 0))
    if workspace is None:
        workspace = alloc_workspace(workspace_size(B, H, T, dk_, dv_, q.dtype, gate, chunk, True, subchunk=subchunk,
                                                   segments=segments, variant=variant, flags=flags), q.device)
    d = make_desc(B, H, T, dk_, dv_, q.dtype, gate, subchunk=subchunk, variant=variant, segments=segments,
                  workspace=workspace, flags=flags)
    r = lib.gla_bwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(h0), _ptr(do), _ptr(dh_final),
                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_alpha), _ptr(dh0), int(chunk), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_bwd")
    return dq, dk, dv, dlog_alpha, dh0


def _on_device(fn):
    """_on_stream, on the device of the first tensor: the library launches on the device
    that is current, so a call with tensors of another device makes that one current."""
    on_stream = _on_stream(fn)
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        x = args[0] if args else kwargs.get(first)
        if x is None:
            return fn(*args, **kwargs)  # which names what is missing
        index = x.get_device()
        if index < 0:
            raise ValueError("tensors passed to the GLA library must be on a CUDA device")
        stream = kwargs.get("stream")
        if stream is None and index == torch._C._cuda_getDevice():
            return fn(*args, **kwargs)
        if stream is not None and stream.device != x.device:
            raise ValueError("stream and tensors are on different devices")
        with torch.cuda.device(index):
            return on_stream(*args, **kwargs)
    return wrapper


def _raw_stream(stream, index) -> int:
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _check(t, name, dtype, shape, index):
    """Refuse a tensor of another type, shape or device than the call needs."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{index}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")


def _dense(t, name, dtype, shape, index):
    """Address of a contiguous tensor, None for None."""
    if t is None:
        return None
    _check(t, name, dtype, shape, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(ws, index):
    """(address, bytes) of a workspace: contiguous memory of the device that the call runs on."""
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on cuda:{index}, got strides {ws.stride()} on {ws.device}")
    return ws.data_ptr(), ws.nbytes


def _views(dtype, index, *tensors):
    """gla_view of each (tensor [B,H,T,d] or, one token, [B,H,d], its name, its shape): an array of
    them, and the address of the first (they lie 32 bytes apart)."""
    a = array.array("q")
    for t, name, shape in tensors:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
            _check(t, name, dtype, shape, index)
        s = t.stride()
        if s[-1] != 1 and shape[-1] != 1:
            raise ValueError(f"{name}: the channels of a token must be contiguous")
        a.extend((t.data_ptr(), s[0], s[1], s[2] if len(s) == 4 else 0))
    return a, a.buffer_info()[0]


def _decay_desc(B, H, T, max_len, dk, dv, dtype, slots0=0, slots1=0, segments=0, workspace=None,
                index=0) -> gla_decay_desc:
    code = DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    ws, size = (None, 0) if workspace is None else _workspace(workspace, index)
    return gla_decay_desc(B, H, T, max_len, dk, dv, code, slots0, slots1, segments, ws, size)


def decay_workspace_size(B, H, T, dk, dv, dtype, for_bwd=False, *, max_len=0, segments=0) -> int:
    """Bytes of workspace for gla_decay_fwd / gla_decay_bwd: B sequences of T tokens each
    (dense) or, with max_len, B sequences of at most max_len tokens in T rows (packed)."""
    d = _decay_desc(B, H, T, max_len, dk, dv, dtype, segments=segments)
    n = load().gla_decay_workspace_size(ctypes.byref(d), int(for_bwd))
    if n == 0:
        raise GLAError(-2 if min(B, H, T, dk, dv) >= 1 and segments >= 0 else -1, "gla_decay_workspace_size")
    return int(n)


def alloc_decay_workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace for the decay calls with its status word cleared (read: poll_status)."""
    ws = torch.empty(int(nbytes), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


@functools.lru_cache(maxsize=256)
def _decay_bytes(B, H, T, max_len, dk, dv, dtype, segments, for_bwd) -> int:
    """decay_workspace_size without its refusal: an invalid call needs no workspace to be refused."""
    d = _decay_desc(B, H, T, max_len, dk, dv, dtype, segments=segments)
    return max(load().gla_decay_workspace_size(ctypes.byref(d), for_bwd), 256)


def _decay_setup(q, v, index, cu_seqlens, max_len, slots0, slots1, segments, workspace, for_bwd):
    """(B sequences, cu pointer, descriptor, workspace) of a chunked call.  A workspace the
    caller did not pass lives for this call, and its status word, never cleared, is not read."""
    B, H, T, dk = q.shape
    if cu_seqlens is None:
        if max_len is not None:
            raise ValueError("max_len goes with cu_seqlens")
        cu, max_len = None, 0
    else:
        if B != 1:
            raise ValueError("packed tensors are [1,H,T,d]")
        if max_len is None:
            raise ValueError("packed tensors need max_len, a bound on the longest sequence")
        max_len = 1 if max_len == 0 else max_len  # a batch of empty sequences; the library's 0 means dense
        B = cu_seqlens.numel() - 1
        cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), index)
    d = _decay_desc(B, H, T, max_len, dk, v.shape[-1], q.dtype, B if slots0 is None else slots0,
                    B if slots1 is None else slots1, segments, workspace, index)
    if workspace is None:
        n = _decay_bytes(B, H, T, max_len, dk, v.shape[-1], q.dtype, segments, for_bwd)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
        d.workspace, d.workspace_bytes = workspace.data_ptr(), n
    return B, cu, d, workspace


@_on_device
def gla_decay_fwd(q, k, v, log_decay, *, cu_seqlens=None, max_len=None, h0=None, h0_index=None, o=None, h_final=None,
                  h_final_index=None, want_final=True, segments=0, workspace=None, stream=None):
    """Linear attention whose heads forget at a constant rate: S_t = lambda_h S_{t-1} + k_t^T v_t,
    o_t = q_t S_t, lambda_h = exp(log_decay[h]).  Returns (o, h_final or None).  See include/gla.h.

    q, k [B,H,T,dk], v [B,H,T,dv] with any distances between sequences, heads and tokens (a
    transposed view of token-major rows is fine, and one expanded over heads); log_decay [H] fp32.  Dense: B sequences of T
    tokens.  Packed: cu_seqlens [n+1] int32, B = 1, sequence i owns rows cu[i] .. cu[i+1]-1 and
    none is longer than max_len; rows of no sequence are left as they are in a given `o` and are
    zero in one that the call makes.
    h0 [slots,H,dk,dv] fp32: start states, sequence i from entry h0_index[i] (int32; default i;
    negative: zero).  h_final: where the last states go, by h_final_index (negative: nowhere);
    it may be h0 itself.  Without it, and with want_final, a new [n,H,dk,dv] tensor.
    What the device finds (a bad bound, an index out of range or used twice, a positive decay, a
    wait that ran out) is reported in the status word of a workspace that the caller passes
    (alloc_decay_workspace, poll_status), and nowhere without one."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    index, dt, f32, i32 = q.get_device(), q.dtype, torch.float32, torch.int32
    if o is None:
        # rows of no sequence are not written
        o = (torch.empty if cu_seqlens is None else torch.zeros)(B, H, T, dv, dtype=dt, device=q.device)
    if h_final is None and h_final_index is not None:
        raise ValueError("h_final_index needs h_final")
    slots0, slots1 = (0 if h0 is None else h0.shape[0]), (None if h_final is None else h_final.shape[0])
    n, cu, d, workspace = _decay_setup(q, v, index, cu_seqlens, max_len, slots0, slots1, segments, workspace, 0)
    if h_final is None and want_final:
        h_final, slots1 = torch.empty(n, H, dk, dv, dtype=f32, device=q.device), n
    keep, p = _views(dt, index, (q, "q", q.shape), (k, "k", q.shape), (v, "v", (B, H, T, dv)), (o, "o", (B, H, T, dv)))
    r = lib.gla_decay_fwd(ctypes.byref(d), p, p + 32, p + 64, _dense(log_decay, "log_decay", f32, (H,), index), cu,
                          _dense(h0, "h0", f32, (slots0, H, dk, dv), index),
                          _dense(h0_index, "h0_index", i32, (n,), index), p + 96,
                          _dense(h_final, "h_final", f32, (slots1, H, dk, dv), index),
                          _dense(h_final_index, "h_final_index", i32, (n,), index), _raw_stream(stream, index))
    if r != GLA_OK:
        raise GLAError(r, "gla_decay_fwd")
    return o, h_final


@_on_device
def gla_decay_bwd(q, k, v, log_decay, do, *, cu_seqlens=None, max_len=None, h0=None, dh_final=None, dq=None, dk=None,
                  dv=None, dh0=None, want_dh0=True, segments=0, workspace=None, stream=None):
    """Backward of gla_decay_fwd: (dq, dk, dv, dh0 or None) from do [B,H,T,dv] and dh_final
    [n,H,dk,dv] (None: zero); h0 [n,H,dk,dv] or None, in order.  The decay is a constant.
    An input expanded over heads or sequences gets a gradient for each: sum them.
    Rows of no sequence, and what the device finds: as in gla_decay_fwd.  See include/gla.h."""
    lib = load()
    B, H, T, K = q.shape
    V = v.shape[-1]
    index, dt, f32 = q.get_device(), q.dtype, torch.float32
    n, cu, d, workspace = _decay_setup(q, v, index, cu_seqlens, max_len, 0, 0, segments, workspace, 1)
    made = []
    if dq is None:
        made.append(dq := torch.empty_like(q))
    if dk is None:
        made.append(dk := torch.empty_like(k))
    if dv is None:
        made.append(dv := torch.empty_like(v))
    if cu is not None and made:
        torch._foreach_zero_(made)  # rows of no sequence are not written; one launch for the three
    if dh0 is None and want_dh0:
        dh0 = torch.empty(n, H, K, V, dtype=f32, device=q.device)
    sk, sv, ss = q.shape, (B, H, T, V), (n, H, K, V)
    keep, p = _views(dt, index, (q, "q", sk), (k, "k", sk), (v, "v", sv), (do, "do", sv), (dq, "dq", sk), (dk, "dk", sk),
                     (dv, "dv", sv))
    r = lib.gla_decay_bwd(ctypes.byref(d), p, p + 32, p + 64, _dense(log_decay, "log_decay", f32, (H,), index), cu,
                          _dense(h0, "h0", f32, ss, index), p + 96, _dense(dh_final, "dh_final", f32, ss, index),
                          p + 128, p + 160, p + 192, _dense(dh0, "dh0", f32, ss, index), _raw_stream(stream, index))
    if r != GLA_OK:
        raise GLAError(r, "gla_decay_bwd")
    return dq, dk, dv, dh0


@_on_device
def gla_decay_step(q, k, v, log_decay, state, index=None, *, o=None, workspace=None, stream=None):
    """One token for each of B running sequences of gla_decay_fwd: state [slots,H,dk,dv] fp32 is
    updated in place at entry index[b] (int32; default b; negative: a padding row, left out) and
    o reads it.  q, k [B,H,dk], v [B,H,dv], any distances between rows and heads.  Returns o.
    workspace: only its status word is used (poll_status); without one, what the device finds (an
    index out of range or used twice, a positive decay) is not reported.  See include/gla.h."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    if o is None:
        # a padding row's output is not written
        o = (torch.empty if index is None else torch.zeros)(B, H, dv, dtype=dt, device=q.device)
    d = _decay_desc(B, H, 1, 0, dk, dv, dt, 0, state.shape[0], 0, workspace, dev)
    keep, p = _views(dt, dev, (q, "q", q.shape), (k, "k", q.shape), (v, "v", (B, H, dv)), (o, "o", (B, H, dv)))
    r = load().gla_decay_step(ctypes.byref(d), p, p + 32, p + 64, _dense(log_decay, "log_decay", f32, (H,), dev),
                              _dense(state, "state", f32, (state.shape[0], H, dk, dv), dev),
                              _dense(index, "index", torch.int32, (B,), dev), p + 96, _raw_stream(stream, dev))
    if r != GLA_OK:
        raise GLAError(r, "gla_decay_step")
    return o


def layernorm_workspace_size(rows, d) -> int:
    """Bytes of workspace for a gla_layernorm_bwd that returns dw or db."""
    n = load().gla_layernorm_workspace_size(int(rows), int(d))
    if n == 0:
        raise GLAError(-2 if rows >= 1 and d >= 1 else -1, "gla_layernorm_workspace_size")
    return int(n)


def _row_view(t, name, like, index):
    """(address, distance of rows) of [..., d] whose leading dimensions are evenly spaced rows."""
    _check(t, name, like.dtype, like.shape, index)
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name}: contiguous, or two-dimensional with contiguous rows")
    return t.data_ptr(), t.stride(0)


@_on_device
def gla_layernorm_fwd(x, w=None, b=None, *, eps=1e-5, y=None, want_stats=True, stream=None):
    """y = (x - mean) rstd w + b over the last dimension.  x [...,d] (contiguous, or rows of a
    wider matrix); w, b [d] fp32 or None.  Returns (y, mean, rstd), the statistics [...] in fp32
    (None without want_stats).  y may be x.  See include/gla.h."""
    code, shape, index, f32 = DTYPE.get(x.dtype), x.shape, x.get_device(), torch.float32
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    n = shape[-1]
    rows = x.numel() // max(1, n)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = rstd = pm = pr = None
    if want_stats:
        mean = torch.empty(rows, dtype=f32, device=x.device)
        mean = mean if len(shape) == 2 else mean.view(shape[:-1])
        rstd = torch.empty_like(mean)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
    (px, ldx), (py, ldy) = _row_view(x, "x", x, index), _row_view(y, "y", x, index)
    r = load().gla_layernorm_fwd(code, rows, n, px, ldx, _dense(w, "w", f32, (n,), index),
                                 _dense(b, "b", f32, (n,), index), eps, py, ldy, pm, pr, _raw_stream(stream, index))
    if r != GLA_OK:
        raise GLAError(r, "gla_layernorm_fwd")
    return y, mean, rstd


@_on_device
def gla_layernorm_bwd(x, dy, mean, rstd, w=None, *, dx=None, want_dwb=True, workspace=None, stream=None):
    """Backward of gla_layernorm_fwd: (dx, dw or None, db or None), dw and db [d] fp32 summed
    over all rows in a fixed order.  mean, rstd from the forward.  dx may be dy."""
    lib = load()
    code, shape, index, f32 = DTYPE.get(x.dtype), x.shape, x.get_device(), torch.float32
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    n = shape[-1]
    rows = x.numel() // max(1, n)
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    dw = db = pw = pb = None
    if want_dwb:
        dw = torch.empty(n, dtype=f32, device=x.device)
        db = torch.empty_like(dw)
        pw, pb = dw.data_ptr(), db.data_ptr()
        if workspace is None:
            workspace = torch.empty(lib.gla_layernorm_workspace_size(rows, n), dtype=torch.uint8, device=x.device)
    (px, ldx), (pg, ldg), (po, ldo) = (_row_view(t, m, x, index) for t, m in ((x, "x"), (dy, "dy"), (dx, "dx")))
    ws, size = (None, 0) if workspace is None else _workspace(workspace, index)
    r = lib.gla_layernorm_bwd(code, rows, n, px, ldx, pg, ldg, _dense(mean, "mean", f32, shape[:-1], index),
                              _dense(rstd, "rstd", f32, shape[:-1], index), _dense(w, "w", f32, (n,), index), po, ldo,
                              pw, pb, ws, size, _raw_stream(stream, index))
    if r != GLA_OK:
        raise GLAError(r, "gla_layernorm_bwd")
    return dx, dw, db


def poll_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and read/clear the device status word of a workspace (GLA_OK = 0)."""
    d = gla_desc()
    d.workspace = workspace.data_ptr()
    d.workspace_bytes = workspace.numel()
    return int(load().gla_poll_status(ctypes.byref(d), _stream_handle(stream)))


def selftest_timeout(workspace: torch.Tensor, limit_us: int = 20000, stream=None) -> None:
    """Enqueue the bounded-wait self-test: a kernel whose wait on an mbarrier that
    nothing completes runs out after limit_us and sets the timeout bit of the status
    word at the start of `workspace` (read it with poll_status)."""
    r = load().gla_selftest_timeout(ctypes.c_void_p(workspace.data_ptr()), int(limit_us), _stream_handle(stream))
    if r != GLA_OK:
        raise GLAError(r, "gla_selftest_timeout")


def timing_enable(on: bool = True) -> None:
    load().gla_timing_enable(int(bool(on)))


def timing_collect(max_launches: int = 65536):
    """[(kernel_name, ms), ...] for the launches recorded since the last collect."""
    lib = load()
    ids = (ctypes.c_int * max_launches)()
    ms = (ctypes.c_float * max_launches)()
    n = lib.gla_timing_collect(max_launches, ids, ms)
    return [(lib.gla_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(n)]


def build_info() -> str:
    return load().gla_build_info().decode()
