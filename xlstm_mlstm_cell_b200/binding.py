"""Thin ctypes binding of libmlstm (argument marshalling only).

The functions take torch tensors that already live on the GPU, pass their
device pointers, sizes and the current CUDA stream to the C ABI declared in
``include/*.h``, and raise ``MlstmError`` on a non-zero status.  Every step
of the computation runs in the library's CUDA kernels; there is no other code
path.  A call runs on the current stream, or as one on ``stream`` where that is
given.  If the library cannot be loaded the import of the functions fails
loudly (``load()`` raises).
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmlstm.so")

MLSTM_F32, MLSTM_BF16 = 0, 1
STATUS = {0: "MLSTM_OK", 1: "MLSTM_ERR_INVALID_ARG", 2: "MLSTM_ERR_UNSUPPORTED", 3: "MLSTM_ERR_WORKSPACE",
          4: "MLSTM_ERR_CUDA", 5: "MLSTM_ERR_TIMEOUT"}


class _Strides(ctypes.Structure):
    """qknorm_strides of include/qknorm.h."""
    _fields_ = [("batch", ctypes.c_longlong), ("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


# Every symbol the headers under include/ declare, with its ctypes signature.
_vp, _fp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "mlstm_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "mlstm_fwd": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _fp, _fp, _fp, _vp, _sz,
                       _vp]),
    "mlstm_fwd_state": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp, _fp, _fp,
                             _fp, _vp, _sz, _vp]),
    "mlstm_fwd_profiled": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _fp, _fp, _fp,
                                _vp, _sz, _vp, ctypes.POINTER(ctypes.c_void_p)]),
    "mlstm_fwd_status": (_i, [_vp, _vp]),
    "mlstm_fwd_noalloc": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _fp, _fp, _fp,
                               _vp]),
    "mlstm_fwd_noalloc_status": (_i, [_vp]),
    "mlstm_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "mlstm_bwd": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _fp, _fp, _vp,
                       _vp, _sz, _vp]),
    "mlstm_fwd_kernel_launches": (_i, [_i, _i, _i, _i, _i, _i, _i]),
    "mlstm_fwd_tensor_path": (_i, [_i, _i, _i, _i]),
    "mlstm_fwd_paired_walk": (_i, [_i, _i, _i, _i]),
    "mlstm_bwd_tensor_path": (_i, [_i, _i, _i, _i]),
    "mlstm_fwd_segments": (_i, [_i, _i, _i, _i, _i, _i, _i]),
    "mlstm_step": (_i, [_fp, _fp, _fp, _vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "mlstm_status_string": (ctypes.c_char_p, [_i]),
    "mlstm_fwd_final_state": (_i, [_vp, _vp, _fp, _fp, _i, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp, _sz, _vp]),
    "mlstm_log_decay_sum": (_i, [_fp, _i, _i, _i, _fp, _vp]),
    "mlstm_state_prefix": (_i, [_fp, _fp, _fp, _fp, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp]),
    "mlstm_selftest_wait_timeout": (_i, [_vp, _vp]),
    "slstm_fwd": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _fp, _vp, _vp, _vp]),
    "slstm_batch_per_cluster": (_i, [_i, _i, _i, _i]),
    "gdelta_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "gdelta_fwd": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _fp, _vp, _fp, _vp, _sz, _vp]),
    "gdelta_fwd_tensor_path": (_i, [_i, _i, _i]),
    "gdelta_step": (_i, [_fp, _vp, _vp, _vp, _fp, _fp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "gdelta_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "gdelta_bwd": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _fp, _vp, _fp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp,
                        _fp, _fp, _fp, _vp, _sz, _vp]),
    "qknorm_fwd": (_i, [_vp, _Strides, _vp, _Strides, _fp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                        _vp, _vp]),
    "qknorm_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "qknorm_bwd": (_i, [_vp, _vp, _vp, _Strides, _vp, _Strides, _fp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                        _i, _vp, _Strides, _vp, _Strides, _fp, _fp, _vp, _sz, _vp]),
}

_lib = None


class MlstmError(RuntimeError):
    def __init__(self, fn: str, status: int, lib=None):
        text = lib.mlstm_status_string(status).decode() if lib is not None else ""
        super().__init__("%s returned %s (%s)" % (fn, STATUS.get(status, status), text))
        self.status = status


def load(path: str | None = None):
    """Loads libmlstm.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libmlstm.so not found at %s; build it with `python -m xlstm_mlstm_cell_b200.build`" % p)
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MLSTM_F32
    if t.dtype == torch.bfloat16:
        return MLSTM_BF16
    raise TypeError("q, k, v must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, status):
    if status != 0:
        raise MlstmError(fn, status, _lib)


def _on_stream(stream, fn, tensor, *args, **kwargs):
    """``fn(tensor, *args, **kwargs)`` as a call on ``stream``.

    The stream is the current one meanwhile, so that what the call allocates comes from its memory: a block of the
    caller's stream could still be in use by work queued there, for which the call's kernels do not wait.  The results
    are recorded on the caller's stream, where it goes on to use them, so that a block is not handed on before that is
    done either.
    """
    if tensor.get_device() != stream.device_index:
        raise ValueError("the tensors are on %s, the stream on %s" % (tensor.device, stream.device))
    device, caller = torch._C._cuda_getDevice(), torch.cuda.current_stream(stream.device_index)
    torch.cuda.set_stream(stream)
    try:
        out = fn(tensor, *args, **kwargs)
    finally:
        torch.cuda.set_stream(caller)
        if device != stream.device_index:   # selecting a stream selects its device
            torch.cuda.set_device(device)
    if caller != stream:
        _record(out, caller)
    return out


def _record(out, stream):
    if isinstance(out, torch.Tensor):
        out.record_stream(stream)
    elif out is not None:
        for x in out:
            _record(x, stream)


def workspace_size(B, NH, S, DHQK, DHV, chunk, dtype) -> int:
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_fwd_workspace_size(B, NH, S, DHQK, DHV, chunk, dt))


def fwd_kernel_launches(B, NH, S, DHQK, DHV, chunk, dtype) -> int:
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_fwd_kernel_launches(B, NH, S, DHQK, DHV, chunk, dt))


def fwd_tensor_path(DHQK, DHV, chunk, dtype) -> int:
    """1: tensor-core path, 0: fp32 CUDA-core path, -1: unsupported (mlstm_fwd_tensor_path)."""
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_fwd_tensor_path(DHQK, DHV, chunk, dt))


def fwd_paired_walk(DHQK, DHV, chunk, dtype) -> int:
    """1: the walk runs as CTA pairs, 0: one CTA per value tile, -1: off the tensor-core path
    (mlstm_fwd_paired_walk)."""
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_fwd_paired_walk(DHQK, DHV, chunk, dt))


def fwd_segments(B, NH, S, DHQK, DHV, chunk, dtype) -> int:
    """Segments per head of the tensor-core path for this shape (0 off that path)."""
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_fwd_segments(B, NH, S, DHQK, DHV, chunk, dt))


def alloc_workspace(B, NH, S, DHQK, DHV, chunk, dtype, device="cuda") -> torch.Tensor:
    n = workspace_size(B, NH, S, DHQK, DHV, chunk, dtype)
    if n == 0:
        raise MlstmError("mlstm_fwd_workspace_size", 2)
    return torch.empty(n, dtype=torch.uint8, device=device)


FWD_PHASES = 4
PHASE_NAMES = ("gate_prep", "state_contributions", "state_scan", "outputs")


def fwd(q, k, v, igate, fgate, ogate=None, chunk: int = 64, h_out=None, C_final=None, n_final=None,
        m_final=None, workspace=None, return_state: bool = True, stream=None, events=None, state=None):
    """mlstm_fwd on device tensors; returns ``(h, C, n, m)`` (states None unless requested).

    ``state=(C0, n0, m0)`` starts from that state (mlstm_fwd_state) instead of the zero state.
    With ``events`` (FWD_PHASES + 1 ``torch.cuda.Event`` or None) the call goes through
    mlstm_fwd_profiled, which records them around its phases on the stream; ``events[FWD_PHASES
    - 1]`` completes once the final state is written.
    """
    if stream is not None:
        return _on_stream(stream, fwd, q, k, v, igate, fgate, ogate, chunk, h_out, C_final, n_final, m_final,
                          workspace, return_state, events=events, state=state)
    lib = load()
    B, NH, S, DHQK = q.shape
    DHV = v.shape[-1]
    dt = _dt(q)
    if h_out is None:
        h_out = torch.empty((B, NH, S, DHV), dtype=q.dtype, device=q.device)
    if return_state:
        if C_final is None:
            C_final = torch.empty((B, NH, DHQK, DHV), dtype=torch.float32, device=q.device)
        if n_final is None:
            n_final = torch.empty((B, NH, DHQK), dtype=torch.float32, device=q.device)
        if m_final is None:
            m_final = torch.empty((B, NH), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, NH, S, DHQK, DHV, chunk, q.dtype, q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(igate), _ptr(fgate), _ptr(ogate), dt, B, NH, S, DHQK, DHV, chunk,
            _ptr(h_out), _ptr(C_final), _ptr(n_final), _ptr(m_final), _ptr(workspace), workspace.numel(),
            _stream())
    if state is not None:
        assert events is None
        C0, n0, m0 = state
        sargs = args[:13] + (_ptr(C0), _ptr(n0), _ptr(m0)) + args[13:]
        _check("mlstm_fwd_state", lib.mlstm_fwd_state(*sargs))
    elif events is None:
        _check("mlstm_fwd", lib.mlstm_fwd(*args))
    else:
        assert len(events) == FWD_PHASES + 1
        for e in events:            # torch creates the CUDA event lazily, on its first record
            if e is not None and not e.cuda_event:
                e.record()
        arr = (ctypes.c_void_p * (FWD_PHASES + 1))(*[None if e is None else e.cuda_event for e in events])
        _check("mlstm_fwd_profiled", lib.mlstm_fwd_profiled(*args, arr))
    return h_out, C_final, n_final, m_final


def bwd_tensor_path(DHQK, DHV, chunk, dtype) -> int:
    """mlstm_bwd_tensor_path: 1 for the tensor-core gradient products, 0 for the CUDA cores, -1 unsupported."""
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_bwd_tensor_path(DHQK, DHV, chunk, dt))


def bwd_workspace_size(B, NH, S, DHQK, DHV, chunk, dtype) -> int:
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().mlstm_bwd_workspace_size(B, NH, S, DHQK, DHV, chunk, dt))


def bwd(q, k, v, igate, fgate, ogate, dh, chunk: int = 64, workspace=None, stream=None, out=None):
    """mlstm_bwd on device tensors: gradients of sum(dh * h) for the forward pass from the zero
    state.  Returns ``(dq, dk, dv, digate, dfgate, dogate)`` (dogate None without an output gate);
    ``out`` may give those six tensors to write into."""
    if stream is not None:
        return _on_stream(stream, bwd, q, k, v, igate, fgate, ogate, dh, chunk, workspace, out=out)
    lib = load()
    B, NH, S, DHQK = q.shape
    DHV = v.shape[-1]
    dt = _dt(q)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(igate),
               torch.empty_like(fgate), None if ogate is None else torch.empty_like(ogate))
    dq, dk, dv, dig, dfg, dog = out
    if workspace is None:
        n = bwd_workspace_size(B, NH, S, DHQK, DHV, chunk, q.dtype)
        if n == 0:
            raise MlstmError("mlstm_bwd_workspace_size", 2)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check("mlstm_bwd", lib.mlstm_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(igate), _ptr(fgate), _ptr(ogate), _ptr(dh), dt,
                                      B, NH, S, DHQK, DHV, chunk, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dig), _ptr(dfg),
                                      _ptr(dog), _ptr(workspace), workspace.numel(), _stream()))
    return dq, dk, dv, dig, dfg, dog


def fwd_final_state(k, v, igate, fgate, chunk: int = 64, workspace=None, stream=None):
    """mlstm_fwd_final_state: ``(C, n, m)`` of the sequence from the zero state, no outputs."""
    if stream is not None:
        return _on_stream(stream, fwd_final_state, k, v, igate, fgate, chunk, workspace)
    lib = load()
    B, NH, S, DHQK = k.shape
    DHV = v.shape[-1]
    C = torch.empty((B, NH, DHQK, DHV), dtype=torch.float32, device=k.device)
    n = torch.empty((B, NH, DHQK), dtype=torch.float32, device=k.device)
    m = torch.empty((B, NH), dtype=torch.float32, device=k.device)
    if workspace is None:
        workspace = alloc_workspace(B, NH, S, DHQK, DHV, chunk, k.dtype, k.device)
    _check("mlstm_fwd_final_state",
           lib.mlstm_fwd_final_state(_ptr(k), _ptr(v), _ptr(igate), _ptr(fgate), _dt(k), B, NH, S, DHQK, DHV, chunk,
                                     _ptr(C), _ptr(n), _ptr(m), _ptr(workspace), workspace.numel(), _stream()))
    return C, n, m


def log_decay_sum(fgate, stream=None):
    """mlstm_log_decay_sum: per (b, h) the sum over tokens of logsigmoid(f~), ``[B, NH]``."""
    if stream is not None:
        return _on_stream(stream, log_decay_sum, fgate)
    lib = load()
    B, NH, S = fgate.shape
    g = torch.empty((B, NH), dtype=torch.float32, device=fgate.device)
    _check("mlstm_log_decay_sum", lib.mlstm_log_decay_sum(_ptr(fgate), B, NH, S, _ptr(g), _stream()))
    return g


def state_prefix(C_parts, n_parts, m_parts, g_parts, rank: int, stream=None):
    """mlstm_state_prefix: the start state ``(C0, n0, m0)`` of slice ``rank`` from the gathered
    summaries ``C_parts [R, B, NH, DHQK, DHV]``, ``n_parts [R, B, NH, DHQK]``, ``m_parts`` and
    ``g_parts [R, B, NH]``."""
    if stream is not None:
        return _on_stream(stream, state_prefix, C_parts, n_parts, m_parts, g_parts, rank)
    lib = load()
    R, B, NH, DHQK, DHV = C_parts.shape
    C0 = torch.empty((B, NH, DHQK, DHV), dtype=torch.float32, device=C_parts.device)
    n0 = torch.empty((B, NH, DHQK), dtype=torch.float32, device=C_parts.device)
    m0 = torch.empty((B, NH), dtype=torch.float32, device=C_parts.device)
    _check("mlstm_state_prefix",
           lib.mlstm_state_prefix(_ptr(C_parts), _ptr(n_parts), _ptr(m_parts), _ptr(g_parts), R, rank, B, NH, DHQK,
                                  DHV, _ptr(C0), _ptr(n0), _ptr(m0), _stream()))
    return C0, n0, m0


NOALLOC_MAX_BYTES = 32 * 1024 * 1024


def fwd_noalloc(q, k, v, igate, fgate, ogate=None, chunk: int = 64, h_out=None, C_final=None, n_final=None,
                m_final=None, stream=None):
    """mlstm_fwd_noalloc: the forward pass with the library's built-in scratch array.

    For callers that may not allocate device memory for a workspace (the outputs are still
    the caller's).  Returns ``(h, C, n, m)``.
    """
    if stream is not None:
        return _on_stream(stream, fwd_noalloc, q, k, v, igate, fgate, ogate, chunk, h_out, C_final, n_final, m_final)
    lib = load()
    B, NH, S, DHQK = q.shape
    DHV = v.shape[-1]
    if h_out is None:
        h_out = torch.empty((B, NH, S, DHV), dtype=q.dtype, device=q.device)
    if C_final is None:
        C_final = torch.empty((B, NH, DHQK, DHV), dtype=torch.float32, device=q.device)
    if n_final is None:
        n_final = torch.empty((B, NH, DHQK), dtype=torch.float32, device=q.device)
    if m_final is None:
        m_final = torch.empty((B, NH), dtype=torch.float32, device=q.device)
    st = lib.mlstm_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(igate), _ptr(fgate), _ptr(ogate), _dt(q), B, NH,
                               S, DHQK, DHV, chunk, _ptr(h_out), _ptr(C_final), _ptr(n_final), _ptr(m_final),
                               _stream())
    _check("mlstm_fwd_noalloc", st)
    return h_out, C_final, n_final, m_final


def fwd_noalloc_status(stream=None) -> int:
    """mlstm_fwd_noalloc_status: 0 when the last mlstm_fwd_noalloc on this device completed, else the
    status code (MLSTM_ERR_TIMEOUT after a bounded wait gave up); synchronizes the stream."""
    return int(load().mlstm_fwd_noalloc_status(_stream(stream)))


def fwd_status(workspace, stream=None) -> int:
    return int(load().mlstm_fwd_status(_ptr(workspace), _stream(stream)))


def step(C, n, m, q, k, v, igate, fgate, ogate=None, h_out=None, stream=None):
    """mlstm_step on device tensors; the state (C, n, m) is updated in place; returns h."""
    if stream is not None:
        return _on_stream(stream, step, C, n, m, q, k, v, igate, fgate, ogate, h_out)
    lib = load()
    B, NH, DHQK = q.shape
    DHV = v.shape[-1]
    if h_out is None:
        h_out = torch.empty((B, NH, DHV), dtype=q.dtype, device=q.device)
    st = lib.mlstm_step(_ptr(C), _ptr(n), _ptr(m), _ptr(q), _ptr(k), _ptr(v), _ptr(igate), _ptr(fgate),
                        _ptr(ogate), _dt(q), B, NH, DHQK, DHV, _ptr(h_out), _stream())
    _check("mlstm_step", st)
    return h_out


def slstm_fwd(wx, R, forget: str = "exp", state=None, h_out=None, want_h: bool = True, status=None, stream=None):
    """slstm_fwd on device tensors: S steps of the sLSTM recurrence.

    wx [B, S, 4, NH, DH] gate pre-activations (i, f, z, o), R [NH, 4, DH, DH], both float32 or
    bfloat16; forget "exp" or "sigmoid"; state (c, n, m, h) fp32 [B, NH, DH] updated in place
    (zeros when None); status: an optional int32 device tensor that a timed-out wait sets to
    MLSTM_ERR_TIMEOUT.  Returns (h_seq [B, S, NH, DH] or None, (c, n, m, h)).
    """
    if forget not in ("exp", "sigmoid"):
        raise ValueError("forget must be 'exp' or 'sigmoid'")
    if stream is not None:
        return _on_stream(stream, slstm_fwd, wx, R, forget, state, h_out, want_h, status)
    lib = load()
    B, S, _, NH, DH = wx.shape
    if state is None:
        state = tuple(torch.zeros((B, NH, DH), dtype=torch.float32, device=wx.device) for _ in range(4))
    c, n, m, h = state
    if want_h and h_out is None:
        h_out = torch.empty((B, S, NH, DH), dtype=wx.dtype, device=wx.device)
    st = lib.slstm_fwd(_ptr(wx), _ptr(R), _dt(wx), B, S, NH, DH, 1 if forget == "sigmoid" else 0, _ptr(c), _ptr(n),
                       _ptr(m), _ptr(h), _ptr(h_out if want_h else None), _ptr(status), _stream())
    _check("slstm_fwd", st)
    return (h_out if want_h else None), (c, n, m, h)


def slstm_batch_per_cluster(B, NH, DH, dtype) -> int:
    dt = MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    return int(load().slstm_batch_per_cluster(B, NH, DH, dt))


# ---------------------------------------------------------------- gated delta rule

def _need(name, t, shape, dtype, index):
    """Checks one tensor argument (device ``index``): the C ABI sees only its address."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))
    raise ValueError("%s must be contiguous" % name)


def _cuda_index(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("the tensors must be on a CUDA device, got %s" % t.device)
    return index


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(index, call):
    """``call(stream address)`` with the arguments' device as the current one, on that device's current stream."""
    current = torch._C._cuda_getDevice()
    s = torch._C._cuda_getCurrentRawStream(index)
    if current == index:
        return call(s)
    torch.cuda.set_device(index)
    try:
        return call(s)
    finally:
        torch.cuda.set_device(current)


def _gdelta_inputs(q, k, v, g, beta, lengths, step=False):
    """Checks the delta rule's inputs; returns (dt, B, NH, NHV, S, DK, DV, device index)."""
    dt, index = _dt(q), _cuda_index(q)
    if q.dim() != (3 if step else 4) or v.dim() != q.dim():
        raise ValueError("q, k and v must be %s" % ("[B, heads, D]" if step else "[B, heads, S, D]"))
    shape, vshape = q.shape, v.shape
    gates = (shape[0], vshape[1]) if step else (shape[0], vshape[1], shape[2])
    _need("q", q, shape, q.dtype, index)
    _need("k", k, shape, q.dtype, index)
    _need("v", v, gates + (vshape[-1],), q.dtype, index)
    _need("g", g, gates, torch.float32, index)
    _need("beta", beta, gates, torch.float32, index)
    if lengths is not None:
        _need("lengths", lengths, (shape[0],), torch.int32, index)
    return dt, shape[0], shape[1], vshape[1], 1 if step else shape[2], shape[-1], vshape[-1], index


def gdelta_fwd_tensor_path(DK, DV, dtype) -> int:
    """gdelta_fwd_tensor_path: 1 tensor cores, 0 fp32 on the CUDA cores, -1 unsupported."""
    return int(load().gdelta_fwd_tensor_path(DK, DV, MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32))


def gdelta_workspace_size(B, NH, NHV, S, DK, DV, dtype, backward: bool = False) -> int:
    """Workspace bytes of gdelta_fwd, or of gdelta_bwd (0: unsupported)."""
    lib, dt = load(), MLSTM_BF16 if dtype == torch.bfloat16 else MLSTM_F32
    size = lib.gdelta_bwd_workspace_size if backward else lib.gdelta_fwd_workspace_size
    return int(size(B, NH, NHV, S, DK, DV, dt))


def _gdelta_workspace(workspace, sizes, device, index, backward):
    if workspace is None:
        lib = load()
        fn = "gdelta_bwd_workspace_size" if backward else "gdelta_fwd_workspace_size"
        n = int(getattr(lib, fn)(*sizes))
        if n == 0:
            raise MlstmError(fn, 2, lib)
        return torch.empty(n, dtype=torch.uint8, device=device)
    _need("workspace", workspace, workspace.shape, torch.uint8, index)
    return workspace


def gdelta_fwd(q, k, v, g, beta, state=None, lengths=None, scale=None, o_out=None, state_out=None,
               return_state: bool = True, workspace=None, stream=None):
    """gdelta_fwd: the gated delta rule over whole sequences; returns ``(o, final state)``.

    q, k ``[B, NH, S, DK]``, v ``[B, NHV, S, DV]`` (float32 or bfloat16; NHV a multiple of NH), the log
    forget gates g and the write strengths beta ``[B, NHV, S]`` float32.  ``state`` ``[B, NHV, DK, DV]``
    float32 is the state to start from (None: zero) and is not changed unless it is ``state_out`` too;
    ``lengths`` int32 ``[B]`` the real tokens of each item (None: all); ``scale`` defaults to
    DK ** -0.5.  The state is None with ``return_state=False``.
    """
    if stream is not None:
        return _on_stream(stream, gdelta_fwd, q, k, v, g, beta, state, lengths, scale, o_out, state_out,
                          return_state, workspace)
    lib = load()
    dt, B, NH, NHV, S, DK, DV, index = _gdelta_inputs(q, k, v, g, beta, lengths)
    if state is not None:
        _need("state", state, (B, NHV, DK, DV), torch.float32, index)
    if o_out is None:
        o_out = torch.empty_like(v)
    else:
        _need("o_out", o_out, v.shape, q.dtype, index)
    if state_out is not None:
        _need("state_out", state_out, (B, NHV, DK, DV), torch.float32, index)
    elif return_state:
        state_out = torch.empty((B, NHV, DK, DV), dtype=torch.float32, device=q.device)
    workspace = _gdelta_workspace(workspace, (B, NH, NHV, S, DK, DV, dt), q.device, index, False)
    _check("gdelta_fwd", _on(index, lambda s: lib.gdelta_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _addr(lengths), dt, B, NH, NHV, S, DK,
        DV, DK ** -0.5 if scale is None else scale, _addr(state), o_out.data_ptr(), _addr(state_out),
        workspace.data_ptr(), workspace.numel(), s)))
    return o_out, state_out


def gdelta_step(state, q, k, v, g, beta, scale=None, o_out=None, stream=None):
    """gdelta_step: one token of the gated delta rule; updates ``state`` ``[B, NHV, DK, DV]`` in place
    and returns o ``[B, NHV, DV]``.  q, k ``[B, NH, DK]``, v ``[B, NHV, DV]``, g, beta ``[B, NHV]``."""
    if stream is not None:
        return _on_stream(stream, gdelta_step, state, q, k, v, g, beta, scale, o_out)
    lib = load()
    dt, B, NH, NHV, _, DK, DV, index = _gdelta_inputs(q, k, v, g, beta, None, step=True)
    _need("state", state, (B, NHV, DK, DV), torch.float32, index)
    if o_out is None:
        o_out = torch.empty_like(v)
    else:
        _need("o_out", o_out, v.shape, q.dtype, index)
    _check("gdelta_step", _on(index, lambda s: lib.gdelta_step(
        state.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), dt, B, NH, NHV, DK,
        DV, DK ** -0.5 if scale is None else scale, o_out.data_ptr(), s)))
    return o_out


def gdelta_bwd(q, k, v, g, beta, do, state=None, dstate=None, lengths=None, scale=None, workspace=None, out=None,
               stream=None):
    """gdelta_bwd: gradients of ``sum(do * o) + sum(dstate * final state)`` for the forward pass from
    ``state`` (None: zero; ``dstate`` None: zero).  Returns ``(dq, dk, dv, dg, dbeta, dstate0)``, dstate0
    None without a ``state``; ``out`` may give those six tensors (the last one or None) to write into."""
    if stream is not None:
        return _on_stream(stream, gdelta_bwd, q, k, v, g, beta, do, state, dstate, lengths, scale, workspace, out)
    lib = load()
    dt, B, NH, NHV, S, DK, DV, index = _gdelta_inputs(q, k, v, g, beta, lengths)
    _need("do", do, v.shape, q.dtype, index)
    for name, t in (("state", state), ("dstate", dstate)):
        if t is not None:
            _need(name, t, (B, NHV, DK, DV), torch.float32, index)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g),
               torch.empty_like(beta), None if state is None else torch.empty_like(state))
    else:
        for name, t, x in zip(("dq", "dk", "dv", "dg", "dbeta"), out, (q, k, v, g, beta)):
            _need(name, t, x.shape, x.dtype, index)
        if out[5] is not None:
            _need("dstate0", out[5], (B, NHV, DK, DV), torch.float32, index)
    dq, dk, dv, dg, dbeta, dstate0 = out
    workspace = _gdelta_workspace(workspace, (B, NH, NHV, S, DK, DV, dt), q.device, index, True)
    _check("gdelta_bwd", _on(index, lambda s: lib.gdelta_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _addr(lengths), _addr(state),
        do.data_ptr(), _addr(dstate), dt, B, NH, NHV, S, DK, DV, DK ** -0.5 if scale is None else scale, dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _addr(dstate0), workspace.data_ptr(),
        workspace.numel(), s)))
    return dq, dk, dv, dg, dbeta, dstate0


# ---------------------------------------------------------------- norms of queries and keys

QKNORM_KINDS = {"rms": 0, "l2": 1}


def _qknorm_inputs(q, k, q_weight, k_weight, norm, inv_freq, positions):
    """Checks the norms' inputs; returns (dt, B, S, NHQ, NHK, D, RD, kind, device index)."""
    dt, index = _dt(q), _cuda_index(q)
    if norm not in QKNORM_KINDS:
        raise ValueError("norm must be one of %s" % ", ".join(map(repr, QKNORM_KINDS)))
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, S, heads, D]")
    B, S, NHQ, D = q.shape
    NHK = k.shape[2]
    if k.shape != (B, S, NHK, D) or k.dtype != q.dtype or k.get_device() != index:
        raise ValueError("k must be [%d, %d, heads, %d] of %s on %s" % (B, S, D, q.dtype, index))
    for name, t in (("q", q), ("k", k)):
        if t.numel() and t.stride(3) != 1:
            raise ValueError("the elements of a head of %s must be contiguous" % name)
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None:
            _need(name, t, (D,), torch.float32, index)
    RD = 0
    if inv_freq is not None:
        RD = 2 * inv_freq.numel()
        _need("inv_freq", inv_freq, (RD // 2,), torch.float32, index)
        if RD > D:
            raise ValueError("inv_freq must have at most D / 2 = %d frequencies, got %d" % (D // 2, RD // 2))
        if positions is not None:
            _need("positions", positions, (B, S), torch.int32, index)
    elif positions is not None:
        raise ValueError("positions without inv_freq")
    return dt, B, S, NHQ, NHK, D, RD, QKNORM_KINDS[norm], index


def qknorm_bwd_workspace_size(B, S, NHQ, NHK, D) -> int:
    """Workspace bytes of a qknorm_bwd with weights (0: unsupported)."""
    return int(load().qknorm_bwd_workspace_size(B, S, NHQ, NHK, D))


def _strides(t):
    b, s, h, _ = t.stride()
    return _Strides(b, s, h)


def qknorm_fwd(q, k, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6, inv_freq=None,
               positions=None, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """qknorm_fwd: norms every head's query and key, weights and rotates them, and lays them out for the
    cells; returns ``(q_out [B, NHQ, S, D], k_out [B, NHK, S, D])``.

    q ``[B, S, NHQ, D]`` and k ``[B, S, NHK, D]`` (float32 or bfloat16) may be slices of a fused projection:
    only the last axis has to be contiguous.  norm "rms" divides by sqrt(mean(x^2) + eps), "l2" by
    sqrt(sum(x^2) + eps); the weights are float32 ``[D]`` or None.  ``inv_freq`` float32 ``[RD / 2]`` rotates the
    first RD elements by position * inv_freq (None: no rotation); ``positions`` int32 ``[B, S]``, None for
    0 .. S-1; pairs are (p, p + RD/2), or neighbours with ``interleaved``.
    """
    if stream is not None:
        return _on_stream(stream, qknorm_fwd, q, k, q_weight, k_weight, norm, eps, inv_freq, positions, interleaved,
                          q_out, k_out)
    lib = load()
    dt, B, S, NHQ, NHK, D, RD, kind, index = _qknorm_inputs(q, k, q_weight, k_weight, norm, inv_freq, positions)
    if q_out is None:
        q_out = torch.empty((B, NHQ, S, D), dtype=q.dtype, device=q.device)
    else:
        _need("q_out", q_out, (B, NHQ, S, D), q.dtype, index)
    if k_out is None:
        k_out = torch.empty((B, NHK, S, D), dtype=q.dtype, device=q.device)
    else:
        _need("k_out", k_out, (B, NHK, S, D), q.dtype, index)
    _check("qknorm_fwd", _on(index, lambda s: lib.qknorm_fwd(
        q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), _addr(q_weight), _addr(k_weight), _addr(inv_freq),
        _addr(positions), dt, B, S, NHQ, NHK, D, RD, kind, eps, 1 if interleaved else 0, q_out.data_ptr(),
        k_out.data_ptr(), s)))
    return q_out, k_out


def qknorm_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6,
               inv_freq=None, positions=None, interleaved: bool = False, out=None, workspace=None, stream=None):
    """qknorm_bwd: the gradients ``(dq, dk, dq_weight, dk_weight)`` of qknorm_fwd's inputs from those of its
    outputs (weight gradients None where the weight is).  ``out`` may give dq ``[B, S, NHQ, D]`` and dk to
    write into, such as slices of a fused projection's gradient (views that share no element), ``workspace`` the
    bytes that qknorm_bwd_workspace_size names."""
    if stream is not None:
        return _on_stream(stream, qknorm_bwd, dq_out, dk_out, q, k, q_weight, k_weight, norm, eps, inv_freq,
                          positions, interleaved, out, workspace)
    lib = load()
    dt, B, S, NHQ, NHK, D, RD, kind, index = _qknorm_inputs(q, k, q_weight, k_weight, norm, inv_freq, positions)
    _need("dq_out", dq_out, (B, NHQ, S, D), q.dtype, index)
    _need("dk_out", dk_out, (B, NHK, S, D), q.dtype, index)
    if out is None:
        dq = torch.empty((B, S, NHQ, D), dtype=q.dtype, device=q.device)
        dk = torch.empty((B, S, NHK, D), dtype=q.dtype, device=q.device)
    else:
        dq, dk = out
        for name, t, x in (("dq", dq, q), ("dk", dk, k)):
            if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != index or (t.numel() and t.stride(3) != 1):
                raise ValueError("%s must be like its input, the elements of a head contiguous" % name)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k_weight is None else torch.empty_like(k_weight)
    if workspace is None:
        n = int(lib.qknorm_bwd_workspace_size(B, S, NHQ, NHK, D)) if (dwq is not None or dwk is not None) else 0
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    else:
        _need("workspace", workspace, workspace.shape, torch.uint8, index)
    _check("qknorm_bwd", _on(index, lambda s: lib.qknorm_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), _addr(q_weight),
        _addr(k_weight), _addr(inv_freq), _addr(positions), dt, B, S, NHQ, NHK, D, RD, kind, eps,
        1 if interleaved else 0, dq.data_ptr(), _strides(dq), dk.data_ptr(), _strides(dk), _addr(dwq), _addr(dwk),
        workspace.data_ptr(), workspace.numel(), s)))
    return dq, dk, dwq, dwk
