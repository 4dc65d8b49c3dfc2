"""Python binding of libckda.so: (Complex) Kimi Delta Attention on MI355X.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of ``include/ckda.h``.  Tensors are torch CUDA
(HIP) tensors; calls are asynchronous on the current stream, or on ``stream``:
then the caller orders that stream behind what wrote the inputs, and waits for
it before the results are read.  If the shared library is missing the calls
raise -- there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

__all__ = ["chunk_fwd", "chunk_bwd", "chunk_bwd_workspace_size", "recurrent_step",
           "l2norm_debug", "fwd_supported",
           "library_path", "abi_version", "chunk_fwd_save", "CkdaError", "BF16", "F32", "GATE_KDA",
           "GATE_CKDA", "GATES_F32", "GATES_LOGITS_F32", "GATES_LOGITS_BF16", "ChunkFwdPlan",
           "decay_fwd", "decay_bwd", "decay_step", "decay_supported",
           "block_norm", "block_norm_bwd"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = os.path.join(_HERE, "libckda.so")
_lock = threading.Lock()
_lib = None

BF16, F32 = 0, 1
GATE_KDA, GATE_CKDA = 0, 1
GATES_F32, GATES_LOGITS_F32, GATES_LOGITS_BF16 = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 128 * 1024 * 1024  # CKDA_NOALLOC_SCRATCH_BYTES in include/ckda.h
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small",
           4: "HIP error"}


class CkdaError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__("%s: %s" % (_STATUS.get(status, status), detail))
        self.status = status


class FwdDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("chunk_size", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("gate_range", ctypes.c_int32), ("use_qk_l2norm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("gate_input", ctypes.c_int32),
                ("qk_heads", ctypes.c_int32), ("sign_absorb", ctypes.c_int32)]


class DecayDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("gate_range", ctypes.c_int32),
                ("gate_input", ctypes.c_int32), ("qk_heads", ctypes.c_int32),
                ("alpha_per_head", ctypes.c_int32), ("scale", ctypes.c_float)]


def library_path() -> str:
    return _LIB


def _load():
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB):
            raise ImportError(
                "libckda.so is not built (%s); run `python -m gated_delta_rule_ckda_amd.build` "
                "or __graft_entry__.build()" % _LIB)
        lib = ctypes.CDLL(_LIB)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        lib.ckda_chunk_fwd.restype = i32
        lib.ckda_chunk_fwd.argtypes = [ctypes.POINTER(FwdDesc), vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, ctypes.c_size_t, vp]
        lib.ckda_chunk_fwd_noalloc.restype = i32
        lib.ckda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(FwdDesc), vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp]
        lib.ckda_chunk_fwd_prepare.restype = i32
        lib.ckda_chunk_fwd_prepare.argtypes = [ctypes.POINTER(FwdDesc), vp, vp, vp, vp, vp, vp,
                                               ctypes.c_size_t, vp]
        lib.ckda_chunk_fwd_finish.restype = i32
        lib.ckda_chunk_fwd_finish.argtypes = [ctypes.POINTER(FwdDesc), vp, vp, vp, vp, vp, vp,
                                              ctypes.c_size_t, vp]
        lib.ckda_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        lib.ckda_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(FwdDesc), i32]
        lib.ckda_chunk_bwd.restype = i32
        lib.ckda_chunk_bwd.argtypes = [ctypes.POINTER(FwdDesc)] + [vp] * 16 + [ctypes.c_size_t, vp]
        lib.ckda_chunk_fwd_save.restype = i32
        lib.ckda_chunk_fwd_save.argtypes = [ctypes.POINTER(FwdDesc)] + [vp] * 10 + [ctypes.c_size_t, vp]
        lib.ckda_chunk_bwd_saved.restype = i32
        lib.ckda_chunk_bwd_saved.argtypes = [ctypes.POINTER(FwdDesc)] + [vp] * 16 + [ctypes.c_size_t, vp]
        lib.ckda_chunk_bwd_workspace_size.restype = ctypes.c_size_t
        lib.ckda_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(FwdDesc), i32]
        lib.ckda_fwd_supported.restype = i32
        lib.ckda_fwd_supported.argtypes = [ctypes.POINTER(FwdDesc)]
        lib.ckda_recurrent_step.restype = i32
        lib.ckda_recurrent_step.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp,
                                            vp, vp, vp, vp, vp, vp, vp, vp]
        lib.ckda_l2norm_debug.restype = i32
        lib.ckda_l2norm_debug.argtypes = [vp, vp, ctypes.c_int64, i32, i32, vp]
        dd, sz = ctypes.POINTER(DecayDesc), ctypes.c_size_t
        lib.ckda_decay_supported.restype = i32
        lib.ckda_decay_supported.argtypes = [i32, i32]
        for name in ("ckda_decay_fwd_workspace_size", "ckda_decay_bwd_workspace_size"):
            getattr(lib, name).restype = sz
            getattr(lib, name).argtypes = [dd, i32]
        lib.ckda_decay_fwd.restype = i32
        lib.ckda_decay_fwd.argtypes = [dd] + [vp] * 9 + [sz, vp]
        lib.ckda_decay_bwd.restype = i32
        lib.ckda_decay_bwd.argtypes = [dd] + [vp] * 14 + [sz, vp]
        lib.ckda_decay_step.restype = i32
        lib.ckda_decay_step.argtypes = [i32] * 9 + [f32] + [vp] * 8
        i64 = ctypes.c_int64
        lib.ckda_block_norm.restype = i32
        lib.ckda_block_norm.argtypes = [i64, i32, i32, i32, f32] + [vp] * 9
        lib.ckda_block_norm_bwd_workspace_size.restype = sz
        lib.ckda_block_norm_bwd_workspace_size.argtypes = [i64, i32, i32]
        lib.ckda_block_norm_bwd.restype = i32
        lib.ckda_block_norm_bwd.argtypes = [i64, i32, i32, i32, f32] + [vp] * 15 + [sz, vp]
        lib.ckda_status_string.restype = ctypes.c_char_p
        lib.ckda_status_string.argtypes = [i32]
        lib.ckda_last_error.restype = ctypes.c_char_p
        lib.ckda_last_error.argtypes = []
        lib.ckda_abi_version.restype = i32
        lib.ckda_abi_version.argtypes = []
        _lib = lib
        return lib


def abi_version() -> int:
    return int(_load().ckda_abi_version())


def _check(status):
    if status != 0:
        raise CkdaError(status, _load().ckda_last_error().decode())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _record(tensors, stream):
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _on_stream(call, named):
    """call(**named) on named["stream"]: it runs with that stream current, so what it
    allocates belongs to it, a workspace that is dropped on return among that.
    Tensors that come from or go back to the caller's own stream are recorded on
    the other one, so that their memory is not given out again while either
    still uses it."""
    import torch
    stream = named.pop("stream")
    given = [t for t in named.values() if isinstance(t, torch.Tensor)]
    for t in given:
        if t.device != stream.device:
            raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device, t.device))
    caller = torch.cuda.current_stream(stream.device)
    if stream == caller:
        return call(**named)
    try:
        with torch.cuda.stream(stream):
            got = call(**named)
    finally:
        _record(given, stream)
    _record(got if isinstance(got, tuple) else (got,), caller)
    return got


def _gate_code(gate):
    if gate in ("ckda", GATE_CKDA):
        return GATE_CKDA
    if gate in ("kda", GATE_KDA):
        return GATE_KDA
    raise ValueError("gate must be 'ckda' or 'kda'")


def _gate_input(gates, alpha, beta):
    """ckda_gate_input_t for gates='values' (float32 gates) or gates='logits'
    (float32 or bfloat16 logits, activated in the kernels)."""
    import torch
    _require(alpha.dtype == beta.dtype, "alpha and beta must share a dtype")
    if gates == "values":
        _require(alpha.dtype == torch.float32, "gate values must be float32")
        return GATES_F32
    if gates == "logits":
        if alpha.dtype == torch.float32:
            return GATES_LOGITS_F32
        if alpha.dtype == torch.bfloat16:
            return GATES_LOGITS_BF16
        raise ValueError("gate logits must be float32 or bfloat16")
    raise ValueError("gates must be 'values' or 'logits'")


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _make_desc(q, v, H, dk, dv, chunk_size, gate, use_qk_l2norm, scale, cu_seqlens,
               gate_input=GATES_F32, sign_absorb=False):
    """H: value heads (v.shape[-2]); the q/k heads are q.shape[-2]."""
    if cu_seqlens is not None:
        B, T = 1, q.shape[-3] if q.dim() == 3 else q.shape[1]
        N = cu_seqlens.numel() - 1
    else:
        B, T = q.shape[0], q.shape[1]
        N = B
    return FwdDesc(B, T, H, dk, dv, N, chunk_size, _dtype_code(q), _gate_code(gate),
                   int(bool(use_qk_l2norm)), float(scale), gate_input, q.shape[-2],
                   int(bool(sign_absorb)))


def fwd_supported(chunk_size, dk, dv, dtype) -> bool:
    d = FwdDesc(1, 1, 1, dk, dv, 1, chunk_size, dtype, GATE_CKDA, 1, 1.0, GATES_F32, 0, 0)
    return bool(_load().ckda_fwd_supported(ctypes.byref(d)))


def chunk_fwd_workspace_size(desc: FwdDesc, packed: bool) -> int:
    """Bytes of workspace ckda_chunk_fwd needs for `desc`."""
    return int(_load().ckda_chunk_fwd_workspace_size(ctypes.byref(desc), int(bool(packed))))


def _fwd_call(q, k, v, alpha, beta, h0, cu_seqlens, chunk_size, use_qk_l2norm, gate, scale,
              output_final_state, out, final_state, gates, sign_absorb):
    """Checks shared by chunk_fwd and chunk_fwd_noalloc; returns (desc, o, ht)."""
    import torch
    H, dk, dv = v.shape[-2], q.shape[-1], v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta)):
        _require(t.is_cuda and t.is_contiguous(), "%s must be a contiguous device tensor" % name)
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q, k, v must share a dtype")
    gi = _gate_input(gates, alpha, beta)
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda,
                 "cu_seqlens must be an int32 device tensor")
    desc = _make_desc(q, v, H, dk, dv, chunk_size, gate, use_qk_l2norm, scale, cu_seqlens, gi,
                      sign_absorb)
    _require(q.numel() == desc.B * desc.T * desc.qk_heads * dk, "q has the wrong number of elements")
    _require(k.numel() == q.numel(), "k must match q")
    _require(alpha.numel() == desc.B * desc.T * H * dk, "alpha has the wrong number of elements")
    _require(v.numel() == desc.B * desc.T * H * dv, "v has the wrong number of elements")
    _require(beta.numel() == desc.B * desc.T * H, "beta has the wrong number of elements")
    if h0 is not None:
        _require(h0.dtype == torch.float32 and h0.is_contiguous()
                 and h0.numel() == desc.num_seqs * H * dk * dv, "h0 must be [N,H,dk,dv] float32")
    o = torch.empty_like(v) if out is None else out
    ht = None
    if output_final_state:
        ht = (torch.empty((desc.num_seqs, H, dk, dv), device=q.device, dtype=torch.float32)
              if final_state is None else final_state)
    return desc, o, ht


def chunk_fwd(q, k, v, alpha, beta, *, h0=None, cu_seqlens=None, chunk_size=64,
              use_qk_l2norm=True, gate="ckda", scale=1.0, output_final_state=True,
              out=None, final_state=None, workspace=None, stream=None, gates="values",
              sign_absorb=False):
    """Chunked prefill.  Dense: q,k [B,T,Hk,dk], alpha [B,T,H,dk], v [B,T,H,dv],
    beta [B,T,H]; Hk divides H (grouped value heads: value head h reads q/k
    head h // (H // Hk)).  Packed (cu_seqlens int32 [N+1]): leading [1,T,...]
    or [T,...].
    gates='values': alpha, beta are float32 gates; gates='logits': they are
    float32 or bfloat16 logits that the kernels activate.  sign_absorb=True
    runs the comparison strategy that folds the gates' cumulative signs into
    q and k (same result, more traffic).
    `workspace`: optional uint8 device tensor of at least
    chunk_fwd_workspace_size() bytes (allocated per call when omitted).
    Returns (o, ht) with ht [N,H,dk,dv] float32 (None if not requested)."""
    if stream is not None:
        return _on_stream(chunk_fwd, locals())
    import torch
    lib = _load()
    desc, o, ht = _fwd_call(q, k, v, alpha, beta, h0, cu_seqlens, chunk_size, use_qk_l2norm, gate,
                            scale, output_final_state, out, final_state, gates, sign_absorb)
    need = chunk_fwd_workspace_size(desc, cu_seqlens is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    _require(workspace.is_cuda and workspace.dtype == torch.uint8 and workspace.numel() >= need,
             "workspace must be a uint8 device tensor of at least %d bytes" % need)
    _check(lib.ckda_chunk_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                              _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                              _ptr(workspace), workspace.numel(), _stream()))
    return o, ht


def chunk_fwd_noalloc(q, k, v, alpha, beta, *, h0=None, cu_seqlens=None, chunk_size=64,
                      use_qk_l2norm=True, gate="ckda", scale=1.0, output_final_state=True,
                      out=None, final_state=None, stream=None, gates="values",
                      sign_absorb=False):
    """chunk_fwd through ckda_chunk_fwd_noalloc: no workspace, the library's
    static per-GPU scratch instead (NOALLOC_SCRATCH_BYTES).  The C call
    allocates nothing; pass `out` (and `final_state`) to keep this wrapper
    from allocating them.  Calls on one GPU must not overlap."""
    if stream is not None:
        return _on_stream(chunk_fwd_noalloc, locals())
    lib = _load()
    desc, o, ht = _fwd_call(q, k, v, alpha, beta, h0, cu_seqlens, chunk_size, use_qk_l2norm, gate,
                            scale, output_final_state, out, final_state, gates, sign_absorb)
    _check(lib.ckda_chunk_fwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                      _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                                      _stream()))
    return o, ht


def chunk_fwd_save(q, k, v, alpha, beta, *, h0=None, cu_seqlens=None, chunk_size=64,
                   use_qk_l2norm=True, gate="ckda", scale=1.0, output_final_state=True,
                   out=None, final_state=None, saved=None, stream=None, gates="values"):
    """chunk_fwd through ckda_chunk_fwd_save: the same (o, ht), plus the
    backward's records kept in `saved` (uint8 device tensor of at least
    chunk_bwd_workspace_size() bytes, allocated when omitted) for
    chunk_bwd(..., saved=saved).  Returns (o, ht, saved)."""
    if stream is not None:
        return _on_stream(chunk_fwd_save, locals())
    import torch
    lib = _load()
    desc, o, ht = _fwd_call(q, k, v, alpha, beta, h0, cu_seqlens, chunk_size, use_qk_l2norm, gate,
                            scale, output_final_state, out, final_state, gates, False)
    need = chunk_bwd_workspace_size(desc, cu_seqlens is not None)
    if saved is None:
        saved = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    _require(saved.is_cuda and saved.dtype == torch.uint8 and saved.numel() >= need,
             "saved must be a uint8 device tensor of at least %d bytes" % need)
    _check(lib.ckda_chunk_fwd_save(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                   _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                                   _ptr(saved), saved.numel(), _stream()))
    return o, ht, saved


def chunk_bwd_workspace_size(desc: FwdDesc, packed: bool) -> int:
    """Bytes of workspace ckda_chunk_bwd needs for `desc`."""
    return int(_load().ckda_chunk_bwd_workspace_size(ctypes.byref(desc), int(bool(packed))))


def chunk_bwd(q, k, v, alpha, beta, dout, *, h0=None, dht=None, cu_seqlens=None, chunk_size=64,
              use_qk_l2norm=True, gate="ckda", scale=1.0, output_dh0=True, workspace=None,
              stream=None, gates="values", saved=None):
    """Gradients of chunk_fwd for dL/do = dout (dtype of v) and dL/dht = dht
    ([N,H,dk,dv] float32, None for zero).  Same layouts as chunk_fwd: q, k on
    Hk heads (grouped value heads when Hk < H), gates='values' (float32
    gates) or 'logits' (float32 or bfloat16 logits; the gradients are then
    those of the logits).  With `saved` (from chunk_fwd_save on the same
    inputs) the records are read from it (ckda_chunk_bwd_saved) instead of
    recomputed, and it serves as the workspace.  Returns float32 (dq, dk, dv,
    dalpha, dbeta, dh0) shaped like q, k, v, alpha, beta and [N,H,dk,dv] (dh0
    None unless output_dh0)."""
    if stream is not None:
        return _on_stream(chunk_bwd, locals())
    import torch
    lib = _load()
    H, dk, dv = v.shape[-2], q.shape[-1], v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta),
                    ("dout", dout)):
        _require(t.is_cuda and t.is_contiguous(), "%s must be a contiguous device tensor" % name)
    _require(k.dtype == q.dtype and v.dtype == q.dtype and dout.dtype == q.dtype,
             "q, k, v, dout must share a dtype")
    gi = _gate_input(gates, alpha, beta)
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda,
                 "cu_seqlens must be an int32 device tensor")
    desc = _make_desc(q, v, H, dk, dv, chunk_size, gate, use_qk_l2norm, scale, cu_seqlens,
                      gi, False)
    Hk = desc.qk_heads
    _require(H % Hk == 0, "the q/k heads must divide the value heads")
    _require(q.numel() == desc.B * desc.T * Hk * dk, "q has the wrong number of elements")
    _require(k.numel() == q.numel(), "k must match q")
    _require(alpha.numel() == desc.B * desc.T * H * dk, "alpha has the wrong number of elements")
    _require(v.numel() == desc.B * desc.T * H * dv and dout.numel() == v.numel(),
             "v, dout have the wrong number of elements")
    _require(beta.numel() == desc.B * desc.T * H, "beta has the wrong number of elements")
    for name, t in (("h0", h0), ("dht", dht)):
        if t is not None:
            _require(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda
                     and t.numel() == desc.num_seqs * H * dk * dv,
                     "%s must be [N,H,dk,dv] float32" % name)
    f32 = dict(device=q.device, dtype=torch.float32)
    dq, dkk = (torch.empty(q.shape, **f32) for _ in range(2))
    dal = torch.empty(alpha.shape, **f32)
    dvv = torch.empty(v.shape, **f32)
    dbe = torch.empty(beta.shape, **f32)
    dh0 = torch.empty((desc.num_seqs, H, dk, dv), **f32) if output_dh0 else None
    need = chunk_bwd_workspace_size(desc, cu_seqlens is not None)
    fn = lib.ckda_chunk_bwd
    if saved is not None:
        _require(workspace is None, "pass either workspace or saved")
        workspace, fn = saved, lib.ckda_chunk_bwd_saved
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    _require(workspace.is_cuda and workspace.dtype == torch.uint8 and workspace.numel() >= need,
             "workspace must be a uint8 device tensor of at least %d bytes" % need)
    _check(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
              _ptr(cu_seqlens), _ptr(h0), _ptr(dout), _ptr(dht), _ptr(dq), _ptr(dkk), _ptr(dvv),
              _ptr(dal), _ptr(dbe), _ptr(dh0), _ptr(workspace), workspace.numel(),
              _stream()))
    return dq, dkk, dvv, dal, dbe, dh0


class ChunkFwdPlan:
    """The two passes of chunk_fwd as separate launches on one workspace:
    prepare() runs the transform pass over all chunks, finish() the state
    pass (o and the final state).  Used to time the passes one by one."""

    def __init__(self, q, k, v, alpha, beta, *, h0=None, cu_seqlens=None, chunk_size=64,
                 use_qk_l2norm=True, gate="ckda", scale=1.0, out=None, final_state=None,
                 stream=None, gates="values", sign_absorb=False):
        import torch
        self.lib = _load()
        H, dk, dv = v.shape[-2], q.shape[-1], v.shape[-1]
        self.desc = _make_desc(q, v, H, dk, dv, chunk_size, gate, use_qk_l2norm, scale,
                               cu_seqlens, _gate_input(gates, alpha, beta), sign_absorb)
        self.args = (q, k, v, alpha, beta, h0, cu_seqlens)
        self.stream = stream
        need = chunk_fwd_workspace_size(self.desc, cu_seqlens is not None)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            self.o = torch.empty_like(v) if out is None else out
            self.ht = (torch.empty((self.desc.num_seqs, H, dk, dv), device=q.device,
                                   dtype=torch.float32) if final_state is None else final_state)
            self.ws = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
        if stream is not None and stream != torch.cuda.current_stream(stream.device):
            _record(self.args + (out, final_state), stream)
            _record((self.o, self.ht), torch.cuda.current_stream(stream.device))

    def prepare(self):
        q, k, v, alpha, beta, h0, cu = self.args
        _check(self.lib.ckda_chunk_fwd_prepare(ctypes.byref(self.desc), _ptr(q), _ptr(k),
                                               _ptr(alpha), _ptr(beta), _ptr(cu), _ptr(self.ws),
                                               self.ws.numel(), _stream(self.stream)))

    def finish(self):
        q, k, v, alpha, beta, h0, cu = self.args
        _check(self.lib.ckda_chunk_fwd_finish(ctypes.byref(self.desc), _ptr(v), _ptr(cu),
                                              _ptr(h0), _ptr(self.o), _ptr(self.ht),
                                              _ptr(self.ws), self.ws.numel(),
                                              _stream(self.stream)))
        return self.o, self.ht


def recurrent_step(q, k, v, alpha, beta, state, *, use_qk_l2norm=True, gate="ckda",
                   scale=1.0, out=None, new_state=None, stream=None, gates="values"):
    """One decode token per sequence: q,k [N,Hk,dk], alpha [N,H,dk], v [N,H,dv],
    beta [N,H], state [N,H,dk,dv] float32, updated in place unless new_state
    is given.  `gates` as for chunk_fwd.  Returns o [N,H,dv]."""
    if stream is not None:
        return _on_stream(recurrent_step, locals())
    import torch
    lib = _load()
    N, Hk, dk = q.shape
    H, dv = v.shape[-2], v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta),
                    ("state", state)):
        _require(t.is_cuda and t.is_contiguous(), "%s must be a contiguous device tensor" % name)
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q, k, v must share a dtype")
    gi = _gate_input(gates, alpha, beta)
    _require(state.dtype == torch.float32, "state must be float32")
    _require(k.shape == q.shape and alpha.shape == (N, H, dk) and v.shape == (N, H, dv)
             and beta.shape == (N, H) and state.shape == (N, H, dk, dv), "shape mismatch")
    o = torch.empty_like(v) if out is None else out
    dst = state if new_state is None else new_state
    _check(lib.ckda_recurrent_step(N, H, Hk, dk, dv, _dtype_code(q), _gate_code(gate), gi,
                                   int(bool(use_qk_l2norm)), float(scale), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(dst),
                                   _ptr(o), _stream()))
    return o


def l2norm_debug(x, stream=None):
    """Test export of the in-kernel normalisation over the last axis."""
    import torch
    lib = _load()
    _require(x.is_cuda and x.is_contiguous(), "x must be a contiguous device tensor")
    d = x.shape[-1]
    y = torch.empty(x.shape, device=x.device, dtype=torch.float32)
    _check(lib.ckda_l2norm_debug(_ptr(x), _ptr(y), x.numel() // d, d, _dtype_code(x),
                                 _stream(stream)))
    return y


# ---- linear attention with one decay a head

def _tensors(device, **named):
    """Checks that every given tensor is contiguous on `device` (a GPU)."""
    _require(device.type == "cuda", "tensors must be on a GPU, got %s" % device)
    for name, t in named.items():
        if t is not None:
            if t.device != device:
                raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _launch(device, fn, *args):
    """fn(*args, stream) with the tensors' device current, on that device's
    current stream."""
    import torch
    stream = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        _check(fn(*args, stream))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, stream))


def _sizes_ok(sizes):
    """The library takes 32-bit sizes and would lose the upper half of a longer one;
    `sizes` has the bits of all of a call's."""
    _require(sizes < 1 << 31, "sizes must be below 2^31")


def _state_ok(name, t, shape):
    import torch
    if t is not None:
        _require(t.dtype == torch.float32 and tuple(t.shape) == shape,
                 "%s must be float32 of shape %s" % (name, list(shape)))


@functools.lru_cache(maxsize=256)
def _decay_plan(packed, B, T, H, dk, dv, n, *fields):
    """The descriptor of these sizes and the workspaces it needs (forward, backward)."""
    _sizes_ok(B | T | H | dk | dv | n)
    desc = DecayDesc(B, T, H, dk, dv, n, *fields)
    lib = _load()
    return (desc, int(lib.ckda_decay_fwd_workspace_size(ctypes.byref(desc), packed)),
            int(lib.ckda_decay_bwd_workspace_size(ctypes.byref(desc), packed)))


def _decay_desc(q, k, v, alpha, cu_seqlens, gate, gates, scale):
    """The plan of a decay call, after the checks of its inputs' shapes and types."""
    import torch
    io = _dtype_code(q)
    qs, vs = q.shape, v.shape
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q, k, v must share a dtype")
    lead = 1 if cu_seqlens is not None and len(qs) == 3 else 2
    _require(len(qs) == lead + 2 and len(vs) == lead + 2,
             "q and v must be [B,T,heads,d] (a packed batch may leave B out)")
    _require(k.shape == qs, "k must match q")
    _require(vs[:lead] == qs[:lead], "v must have the tokens of q")
    H, Hk = vs[-2], qs[-2]
    _require(Hk > 0 and H % Hk == 0, "the q/k heads must divide the value heads")
    per_head = alpha.dim() == 1
    _require(alpha.shape == ((H,) if per_head else vs[:-1]),
             "alpha must be [H] or one gate a token and head")
    B, T = (1, qs[0]) if lead == 1 else (qs[0], qs[1])
    n = B
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1,
                 "cu_seqlens must be an int32 vector")
        _require(B == 1, "a packed batch has B = 1")
        n = cu_seqlens.numel() - 1
    return _decay_plan(int(cu_seqlens is not None), B, T, H, qs[-1], vs[-1], n, io, _gate_code(gate),
                       _gate_input(gates, alpha, alpha), Hk, int(per_head), float(scale))


def _workspace(workspace, need, device):
    import torch
    if workspace is None:
        return torch.empty(max(need, 1), device=device, dtype=torch.uint8)
    _require(workspace.device == device and workspace.dtype == torch.uint8
             and workspace.is_contiguous() and workspace.numel() >= need,
             "workspace must be a uint8 tensor of at least %d bytes on %s" % (need, device))
    return workspace


def decay_supported(dk, dv) -> bool:
    return bool(_load().ckda_decay_supported(dk, dv))


def decay_fwd_workspace_size(desc: DecayDesc, packed: bool) -> int:
    """Bytes of workspace ckda_decay_fwd needs for `desc` (0: none)."""
    return int(_load().ckda_decay_fwd_workspace_size(ctypes.byref(desc), int(bool(packed))))


def decay_bwd_workspace_size(desc: DecayDesc, packed: bool) -> int:
    """Bytes of workspace ckda_decay_bwd needs for `desc`."""
    return int(_load().ckda_decay_bwd_workspace_size(ctypes.byref(desc), int(bool(packed))))


def decay_fwd(q, k, v, alpha, *, h0=None, cu_seqlens=None, gate="ckda", gates="values", scale=1.0,
              output_final_state=True, out=None, final_state=None, workspace=None, stream=None):
    """Linear attention with one decay a head, S_t = a_t S_{t-1} + k_t v_t^T and
    o_t = scale S_t^T q_t, over whole prompts.  Dense: q, k [B,T,Hk,dk], v
    [B,T,H,dv] (Hk divides H); packed (cu_seqlens int32 [N+1]): [1,T,...] or
    [T,...].  alpha: [B,T,H], or [H] for a fixed decay; gates='values'
    (float32) or 'logits' (float32 or bfloat16, activated by `gate`).
    Returns (o, ht) with ht [N,H,dk,dv] float32 (None if not requested).  A
    workspace that the caller passes must not be shared by calls that overlap."""
    if stream is not None:
        return _on_stream(decay_fwd, locals())
    import torch
    lib = _load()
    desc, need, _ = _decay_desc(q, k, v, alpha, cu_seqlens, gate, gates, scale)
    dev = q.device
    _tensors(dev, q=q, k=k, v=v, alpha=alpha, h0=h0, cu_seqlens=cu_seqlens, out=out,
             final_state=final_state)
    shape = (desc.num_seqs, desc.H, desc.dk, desc.dv)
    _state_ok("h0", h0, shape)
    _state_ok("final_state", final_state, shape)
    if out is not None:
        _require(out.dtype == v.dtype and out.shape == v.shape, "out must match v")
    o = torch.empty_like(v) if out is None else out
    ht = final_state
    if output_final_state and ht is None:
        ht = torch.empty(shape, device=dev, dtype=torch.float32)
    ws = _workspace(workspace, need, dev) if need else None
    _launch(dev, lib.ckda_decay_fwd, ctypes.byref(desc), _addr(q), _addr(k), _addr(v),
            _addr(alpha), _addr(cu_seqlens), _addr(h0), _addr(o), _addr(ht), _addr(ws),
            0 if ws is None else ws.numel())
    return o, ht


def decay_bwd(q, k, v, alpha, dout, *, h0=None, dht=None, cu_seqlens=None, gate="ckda",
              gates="values", scale=1.0, output_dalpha=True, output_dh0=True, workspace=None,
              stream=None):
    """Gradients of decay_fwd for dL/do = dout and dL/dht = dht (None for zero).
    Returns (dq, dk, dv, dalpha, dh0): the first four in q's dtype, shaped like
    q, k, v and alpha (with logits, the gradient of the logits; with [H], the
    sum over all tokens), dh0 [N,H,dk,dv] float32; dalpha and dh0 None unless
    requested."""
    if stream is not None:
        return _on_stream(decay_bwd, locals())
    import torch
    lib = _load()
    desc, _, need = _decay_desc(q, k, v, alpha, cu_seqlens, gate, gates, scale)
    dev = q.device
    _tensors(dev, q=q, k=k, v=v, alpha=alpha, dout=dout, h0=h0, dht=dht, cu_seqlens=cu_seqlens)
    shape = (desc.num_seqs, desc.H, desc.dk, desc.dv)
    _state_ok("h0", h0, shape)
    _state_ok("dht", dht, shape)
    _require(dout.dtype == v.dtype and dout.shape == v.shape, "dout must match v")
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dal = torch.empty(alpha.shape, device=dev, dtype=q.dtype) if output_dalpha else None
    dh0 = torch.empty(shape, device=dev, dtype=torch.float32) if output_dh0 else None
    ws = _workspace(workspace, need, dev)
    _launch(dev, lib.ckda_decay_bwd, ctypes.byref(desc), _addr(q), _addr(k), _addr(v),
            _addr(alpha), _addr(cu_seqlens), _addr(h0), _addr(dout), _addr(dht), _addr(dq),
            _addr(dkk), _addr(dvv), _addr(dal), _addr(dh0), _addr(ws), ws.numel())
    return dq, dkk, dvv, dal, dh0


def decay_step(q, k, v, alpha, state, *, gate="ckda", gates="values", scale=1.0, out=None,
               new_state=None, stream=None):
    """One token a sequence of decay_fwd's recurrence: q, k [N,Hk,dk], v
    [N,H,dv], alpha [N,H] or [H], state [N,H,dk,dv] float32, updated in place
    unless new_state is given.  Returns o [N,H,dv]."""
    if stream is not None:
        return _on_stream(decay_step, locals())
    import torch
    lib = _load()
    _require(q.dim() == 3 and v.dim() == 3, "q and v must be [N,heads,d]")
    N, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q, k, v must share a dtype")
    _require(k.shape == q.shape and v.shape[0] == N, "shape mismatch")
    per_head = alpha.dim() == 1
    _require(tuple(alpha.shape) == ((H,) if per_head else (N, H)), "alpha must be [N,H] or [H]")
    _sizes_ok(N | H | Hk | dk | dv)
    dev = q.device
    _tensors(dev, q=q, k=k, v=v, alpha=alpha, state=state, out=out, new_state=new_state)
    _state_ok("state", state, (N, H, dk, dv))
    _state_ok("new_state", new_state, (N, H, dk, dv))
    if out is not None:
        _require(out.dtype == v.dtype and out.shape == v.shape, "out must match v")
    o = torch.empty_like(v) if out is None else out
    dst = state if new_state is None else new_state
    _launch(dev, lib.ckda_decay_step, N, H, Hk, dk, dv, _dtype_code(q), _gate_code(gate),
            _gate_input(gates, alpha, alpha), int(per_head), float(scale), _addr(q), _addr(k),
            _addr(v), _addr(alpha), _addr(state), _addr(dst), _addr(o))
    return o


# ---- the norms around a block, with its gate and residual scale

_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}


def _norm_args(y, weight, gate, act, residual, scale, next_weight, **more):
    """Checks of the norm calls' tensors; returns (rows, d, activation code)."""
    import torch
    _require(y.dim() >= 1 and y.shape[-1] > 0, "y must be [..., d]")
    _require(act in _ACTS, "act must be 'none', 'sigmoid' or 'silu'")
    d = y.shape[-1]
    _sizes_ok(d)
    _tensors(y.device, y=y, weight=weight, gate=gate, residual=residual, scale=scale,
             next_weight=next_weight, **more)
    for name, t in dict(gate=gate, residual=residual, **more).items():
        if t is not None and (t.dtype != y.dtype or t.shape != y.shape):
            raise ValueError("%s must match y" % name)
    for name, t in (("weight", weight), ("scale", scale), ("next_weight", next_weight)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (d,)):
            raise ValueError("%s must be float32 [%d]" % (name, d))
    return y.numel() // d, d, 0 if gate is None else _ACTS[act]


def block_norm(y, weight, *, gate=None, act="sigmoid", residual=None, scale=None,
               next_weight=None, eps=1e-6, out=None, next_out=None, stream=None):
    """The norm after a block, its output gate, the residual stream and the norm
    before the next block, over the last axis of y [..., d]:
        u = rmsnorm(y) * weight        (y itself if weight is None)
        v = u * act(gate)              (act 'sigmoid' or 'silu'; gate shaped like y)
        h = residual + scale * v       (scale a channel)
        n = rmsnorm(h) * next_weight
    y, gate and residual in bfloat16 or float32, weight, scale and next_weight
    float32 [d].  Any part may be left out.  Returns (h, n), n None without
    next_weight.  out may be the residual itself (updated in place)."""
    if stream is not None:
        return _on_stream(block_norm, locals())
    import torch
    lib = _load()
    io = _dtype_code(y)
    rows, d, code = _norm_args(y, weight, gate, act, residual, scale, next_weight, out=out,
                               next_out=next_out)
    _require(gate is None or code != 0, "a gate needs act 'sigmoid' or 'silu'")
    _require(next_out is None or next_weight is not None, "next_out needs next_weight")
    h = torch.empty_like(y) if out is None else out
    n = next_out
    if next_weight is not None and n is None:
        n = torch.empty_like(y)
    _launch(y.device, lib.ckda_block_norm, rows, d, io, code, float(eps), _addr(y),
            _addr(weight), _addr(gate), _addr(residual), _addr(scale), _addr(next_weight), _addr(h),
            _addr(n))
    return h, n


def block_norm_bwd(y, weight, dh, *, dnext=None, gate=None, act="sigmoid", residual=None,
                   scale=None, next_weight=None, eps=1e-6, workspace=None, stream=None):
    """Gradients of block_norm for dL/dh = dh and dL/dn = dnext (given exactly
    with next_weight).  Returns (dy, dweight, dgate, dresidual, dscale,
    dnext_weight), None where the input was left out; dy, dgate and dresidual
    in y's dtype, the others float32 [d].  Without next_weight dresidual is dh
    itself."""
    if stream is not None:
        return _on_stream(block_norm_bwd, locals())
    import torch
    lib = _load()
    io = _dtype_code(y)
    rows, d, code = _norm_args(y, weight, gate, act, residual, scale, next_weight, dh=dh, dnext=dnext)
    _require(gate is None or code != 0, "a gate needs act 'sigmoid' or 'silu'")
    _require((dnext is None) == (next_weight is None), "dnext is given exactly with next_weight")
    new = lambda like: None if like is None else torch.empty_like(like)
    dy, dw, dg, ds, dw2 = (new(t) for t in (y, weight, gate, scale, next_weight))
    if rows == 0:
        for t in (dw, ds, dw2):
            if t is not None:
                t.zero_()
        return dy, dw, dg, None if residual is None else dh, ds, dw2
    dx = dh if residual is not None and next_weight is None else new(residual)
    need = int(lib.ckda_block_norm_bwd_workspace_size(rows, d, io))
    ws = _workspace(workspace, need, y.device)
    _launch(y.device, lib.ckda_block_norm_bwd, rows, d, io, code, float(eps), _addr(y),
            _addr(weight), _addr(gate), _addr(residual), _addr(scale), _addr(next_weight),
            _addr(dh), _addr(dnext), _addr(dy), _addr(dw), _addr(dg),
            None if dx is dh else _addr(dx), _addr(ds), _addr(dw2), _addr(ws), ws.numel())
    return dy, dw, dg, dx, ds, dw2
