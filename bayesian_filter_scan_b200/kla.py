"""Python binding of libkla (include/kla.h): argument marshalling only.

Every step of the forward pass runs in libkla's CUDA kernels; this module
allocates outputs and workspace with torch (device memory and streams are the
only things torch provides), checks dtypes and shapes, and calls the C ABI
through ctypes on the current CUDA stream. There is no fallback: if libkla.so
is missing or a call fails, it raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkla.so")

KLA_OK, KLA_ERR_INVALID_ARG, KLA_ERR_UNSUPPORTED, KLA_ERR_CUDA, KLA_ERR_TIMEOUT, KLA_ERR_RANGE = range(6)
KLA_BF16, KLA_FP32 = 0, 1
KLA_DIAG, KLA_ISO = 0, 1
# KLA_NOALLOC_SCRATCH_BYTES of include/kla.h: the fixed scratch area of kla_forward_noalloc
NOALLOC_SCRATCH_BYTES = 32 << 20

# Every symbol include/kla.h declares.
EXPORTS = ("kla_workspace_bytes", "kla_precision_workspace_bytes", "kla_forward", "kla_forward_profiled",
           "kla_plan", "kla_precision",
           "kla_decode_step", "kla_host_device_bytes", "kla_forward_host", "kla_check",
           "kla_status_string", "kla_version", "kla_forward_noalloc", "kla_kdn_forward",
           "kla_prologue", "kla_backward_workspace_bytes", "kla_backward",
           "kla_conv_forward", "kla_conv_backward_workspace_bytes", "kla_conv_backward", "kla_conv_step",
           "kla_ssm_states_bytes", "kla_ssm_forward", "kla_ssm_backward_workspace_bytes", "kla_ssm_backward",
           "kla_ssm_step", "kla_layernorm_forward", "kla_layernorm_backward_workspace_bytes",
           "kla_layernorm_backward")
# Tokens between two recorded states, and the most states per channel (include/kla.h kla_ssm_forward)
SSM_STATE_EVERY, SSM_MAX_STATES = 16, 128


class KlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, status_string(status), status))


class KlaDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("dtype", ctypes.c_int),
                ("mode", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int)]


class KlaConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("W", ctypes.c_int),
                ("dtype", ctypes.c_int), ("silu", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
                ("num_seqs", ctypes.c_int), ("ld_x", ctypes.c_longlong), ("zero_rest", ctypes.c_int)]


class KlaSsmDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("G", ctypes.c_int),
                ("N", ctypes.c_int), ("dtype", ctypes.c_int), ("softplus", ctypes.c_int),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int), ("ld_x", ctypes.c_longlong),
                ("ld_dt", ctypes.c_longlong), ("ld_z", ctypes.c_longlong), ("ld_b", ctypes.c_longlong),
                ("ld_c", ctypes.c_longlong), ("zero_rest", ctypes.c_int)]


class KlaNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("ld_x", ctypes.c_longlong), ("ld_residual", ctypes.c_longlong)]


_lib = None
_P = ctypes.c_void_p


def lib():
    """Load libkla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkla.so not found at %s; run `python -m bayesian_filter_scan_b200.build`"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        D = ctypes.POINTER(KlaDesc)
        L.kla_workspace_bytes.argtypes = [D]
        L.kla_workspace_bytes.restype = ctypes.c_size_t
        L.kla_precision_workspace_bytes.argtypes = [D]
        L.kla_precision_workspace_bytes.restype = ctypes.c_size_t
        L.kla_forward.argtypes = [D] + [_P] * 11 + [_P, ctypes.c_size_t, _P]
        L.kla_forward.restype = ctypes.c_int
        L.kla_forward_profiled.argtypes = [D] + [_P] * 11 + [_P, ctypes.c_size_t, _P, _P]
        L.kla_forward_profiled.restype = ctypes.c_int
        L.kla_plan.argtypes = [D, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                               ctypes.POINTER(ctypes.c_int)]
        L.kla_plan.restype = ctypes.c_int
        L.kla_precision.argtypes = [D] + [_P] * 6 + [_P, ctypes.c_size_t, _P]
        L.kla_precision.restype = ctypes.c_int
        L.kla_decode_step.argtypes = [D] + [_P] * 9 + [_P]
        L.kla_decode_step.restype = ctypes.c_int
        L.kla_host_device_bytes.argtypes = [D]
        L.kla_host_device_bytes.restype = ctypes.c_size_t
        L.kla_forward_host.argtypes = [D] + [_P] * 11 + [_P, ctypes.c_size_t, _P]
        L.kla_forward_host.restype = ctypes.c_int
        L.kla_forward_noalloc.argtypes = [D] + [_P] * 11 + [_P]
        L.kla_forward_noalloc.restype = ctypes.c_int
        L.kla_kdn_forward.argtypes = [D] + [_P] * 11 + [_P]
        L.kla_kdn_forward.restype = ctypes.c_int
        L.kla_prologue.argtypes = [D, ctypes.c_int] + [_P] * 18 + [_P]
        L.kla_prologue.restype = ctypes.c_int
        L.kla_backward_workspace_bytes.argtypes = [D]
        L.kla_backward_workspace_bytes.restype = ctypes.c_size_t
        L.kla_backward.argtypes = [D] + [_P] * 19 + [_P, ctypes.c_size_t, _P]
        L.kla_backward.restype = ctypes.c_int
        S, CD, SD, ND = ctypes.c_size_t, *(ctypes.POINTER(t) for t in (KlaConvDesc, KlaSsmDesc, KlaNormDesc))
        for name, res, args in (
                ("kla_conv_forward", ctypes.c_int, [CD] + [_P] * 7),
                ("kla_conv_backward_workspace_bytes", S, [CD]),
                ("kla_conv_backward", ctypes.c_int, [CD] + [_P] * 11 + [S, _P]),
                ("kla_conv_step", ctypes.c_int, [CD] + [_P] * 6),
                ("kla_ssm_states_bytes", S, [SD]),
                ("kla_ssm_forward", ctypes.c_int, [SD] + [_P] * 13),
                ("kla_ssm_backward_workspace_bytes", S, [SD, ctypes.c_int]),
                ("kla_ssm_backward", ctypes.c_int, [SD] + [_P] * 22 + [S, _P]),
                ("kla_ssm_step", ctypes.c_int, [SD] + [_P] * 11),
                ("kla_layernorm_forward", ctypes.c_int, [ND] + [_P] * 9),
                ("kla_layernorm_backward_workspace_bytes", S, [ND]),
                ("kla_layernorm_backward", ctypes.c_int, [ND] + [_P] * 10 + [S, _P])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        L.kla_check.argtypes = [_P]
        L.kla_check.restype = ctypes.c_int
        L.kla_status_string.argtypes = [ctypes.c_int]
        L.kla_status_string.restype = ctypes.c_char_p
        L.kla_version.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().kla_status_string(int(s)).decode()


def _check(s: int, what: str):
    if s != KLA_OK:
        raise KlaError(s, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_desc(B, T, H, dk, dv, dtype=KLA_BF16, mode=KLA_DIAG, cu_seqlens=None, num_seqs=0) -> KlaDesc:
    return KlaDesc(int(B), int(T), int(H), int(dk), int(dv), int(dtype), int(mode),
                   None if cu_seqlens is None else ctypes.c_void_p(cu_seqlens.data_ptr()), int(num_seqs))


def _desc_from(q, v, B, T, mode, cu_seqlens):
    Ntok, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype == torch.bfloat16:
        dt = KLA_BF16
    elif q.dtype == torch.float32:
        dt = KLA_FP32
    else:
        raise TypeError("q, k, v must be bfloat16 or float32")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens must be a CUDA int32 tensor")
        return make_desc(1, Ntok, H, dk, dv, dt, mode, cu_seqlens, cu_seqlens.numel() - 1), cu_seqlens.numel() - 1
    B = B if B is not None else 1
    T = T if T is not None else Ntok // max(B, 1)
    if B * T != Ntok:
        raise ValueError("B*T must equal the number of tokens")
    return make_desc(B, T, H, dk, dv, dt, mode), B


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _mode(mode) -> int:
    return KLA_ISO if mode in ("iso", KLA_ISO) else KLA_DIAG


def plan(desc: KlaDesc) -> dict:
    """Segments per row, launches per call and tensor-core use for ``desc``."""
    seg, lau, tc = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().kla_plan(ctypes.byref(desc), ctypes.byref(seg), ctypes.byref(lau), ctypes.byref(tc)), "kla_plan")
    return {"segments": seg.value, "launches": lau.value, "tensor_core": bool(tc.value)}


def workspace_bytes(desc: KlaDesc) -> int:
    return int(lib().kla_workspace_bytes(ctypes.byref(desc)))


def forward(q, k, v, a, qn, beta, lambda0=None, eta0=None, cu_seqlens=None, B=None, T=None,
            mode="diag", final_state=False, out=None, workspace=None):
    """KLA forward on CUDA tensors in the layouts of include/kla.h.
    Returns ``out`` or ``(out, final_lambda, final_eta)`` with ``final_state``."""
    m = _mode(mode)
    desc, N = _desc_from(q, v, B, T, m, cu_seqlens)
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("qn", qn), ("beta", beta)):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    for name, t in (("a", a), ("qn", qn), ("beta", beta), ("lambda0", lambda0), ("eta0", eta0)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("%s must be float32" % name)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    if out is None:
        out = torch.empty(q.shape[0], H, dv, dtype=q.dtype, device=q.device)
    fl = fe = None
    if final_state:
        fl = torch.empty((N, H) if m == KLA_ISO else (N, H, dk), dtype=torch.float32, device=q.device)
        fe = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    nbytes = workspace_bytes(desc)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    s = lib().kla_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                          _ptr(lambda0), _ptr(eta0), _ptr(out), _ptr(fl), _ptr(fe), _ptr(workspace),
                          nbytes, _stream())
    _check(s, "kla_forward")
    return (out, fl, fe) if final_state else out


def kdn_forward(q, k, v, a, qn, beta, lambda0=None, M0=None, cu_seqlens=None, B=None, T=None,
                mode="diag", final_state=False, out=None):
    """Kalman Delta Network forward (the Kalman-gain residual write) on CUDA
    tensors in the layouts of include/kla.h. Returns ``out`` or
    ``(out, final_lambda, final_M)`` with ``final_state`` (final_M: the
    posterior mean [N,H,dk,dv])."""
    m = _mode(mode)
    desc, N = _desc_from(q, v, B, T, m, cu_seqlens)
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("qn", qn), ("beta", beta)):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    for name, t in (("a", a), ("qn", qn), ("beta", beta), ("lambda0", lambda0), ("M0", M0)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("%s must be float32" % name)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    if out is None:
        out = torch.empty(q.shape[0], H, dv, dtype=q.dtype, device=q.device)
    fl = fm = None
    if final_state:
        fl = torch.empty((N, H) if m == KLA_ISO else (N, H, dk), dtype=torch.float32, device=q.device)
        fm = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    s = lib().kla_kdn_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                              _ptr(lambda0), _ptr(M0), _ptr(out), _ptr(fl), _ptr(fm), _stream())
    _check(s, "kla_kdn_forward")
    return (out, fl, fm) if final_state else out


def backward(q, k, v, a, qn, beta, dout, lambda0=None, eta0=None, dfinal_lambda=None, dfinal_eta=None,
             cu_seqlens=None, B=None, T=None, mode="diag", workspace=None):
    """Gradients of ``forward`` (include/kla.h kla_backward) on CUDA tensors:
    returns a dict of fp32 tensors ``dq, dk, dv, da, dqn, dbeta, dlambda0,
    deta0`` in the layouts of the corresponding inputs."""
    m = _mode(mode)
    desc, N = _desc_from(q, v, B, T, m, cu_seqlens)
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("qn", qn), ("beta", beta), ("dout", dout)):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v, dout must share a dtype")
    for name, t in (("a", a), ("qn", qn), ("beta", beta), ("lambda0", lambda0), ("eta0", eta0),
                    ("dfinal_lambda", dfinal_lambda), ("dfinal_eta", dfinal_eta)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("%s must be float32" % name)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32), "dv": torch.empty(v.shape, **f32),
         "da": torch.empty(a.shape, **f32), "dqn": torch.empty(qn.shape, **f32),
         "dbeta": torch.empty(beta.shape, **f32),
         "dlambda0": torch.empty((N, H) if m == KLA_ISO else (N, H, dk), **f32),
         "deta0": torch.empty(N, H, dk, dv, **f32)}
    nbytes = lib().kla_backward_workspace_bytes(ctypes.byref(desc))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    s = lib().kla_backward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                           _ptr(lambda0), _ptr(eta0), _ptr(dout), _ptr(dfinal_lambda), _ptr(dfinal_eta),
                           *(_ptr(g[n]) for n in ("dq", "dk", "dv", "da", "dqn", "dbeta", "dlambda0", "deta0")),
                           _ptr(workspace), workspace.numel(), _stream())
    _check(s, "kla_backward")
    return g


def prologue(xq, xk, xv, xa, xqn, xbeta, wq, wk, wv, bq=None, bk=None, bv=None, cu_seqlens=None,
             B=None, T=None, mode="diag", out=None):
    """The mixer's input prologue on CUDA tensors (include/kla.h kla_prologue):
    returns ``(q, k, v, a, qn, beta)`` in the forward pass's layouts."""
    m = _mode(mode)
    desc, N = _desc_from(xq, xv, B, T, m, cu_seqlens)
    ts = (xq, xk, xv, xa, xqn, xbeta, wq, wk, wv) + tuple(t for t in (bq, bk, bv) if t is not None)
    for t in ts:
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("prologue inputs must be contiguous CUDA tensors")
    W = wq.shape[-1]
    if out is None:
        out = (torch.empty_like(xq), torch.empty_like(xk), torch.empty_like(xv), torch.empty_like(xa),
               torch.empty_like(xqn), torch.empty_like(xbeta))
    s = lib().kla_prologue(ctypes.byref(desc), W, *[_ptr(t) for t in (xq, xk, xv, xa, xqn, xbeta, wq, wk, wv,
                                                                        bq, bk, bv)],
                           *[_ptr(t) for t in out], _stream())
    _check(s, "kla_prologue")
    return out


def precision(k, a, qn, beta, lambda0=None, cu_seqlens=None, B=None, T=None, mode="diag"):
    """Posterior precision after every token ([Ntok,H,dk], iso [Ntok,H])."""
    m = _mode(mode)
    desc, N = _desc_from(k, k, B, T, m, cu_seqlens)
    Ntok, H, dk = k.shape
    lam = torch.empty((Ntok, H) if m == KLA_ISO else (Ntok, H, dk), dtype=torch.float32, device=k.device)
    nbytes = int(lib().kla_precision_workspace_bytes(ctypes.byref(desc)))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=k.device) if nbytes else None
    s = lib().kla_precision(ctypes.byref(desc), _ptr(k), _ptr(a), _ptr(qn), _ptr(beta), _ptr(lambda0),
                            _ptr(lam), _ptr(ws), nbytes, _stream())
    _check(s, "kla_precision")
    return lam


def decode_step(q, k, v, a, qn, beta, lam, eta, mode="diag", out=None):
    """One recurrent step per row: q,k,v [N,H,d], a,qn [N,H,dk] (iso [N,H]),
    beta [N,H]; ``lam``/``eta`` (the belief) are updated in place. Returns out."""
    m = _mode(mode)
    N, H, dk = q.shape
    dv = v.shape[-1]
    desc = make_desc(N, 1, H, dk, dv, KLA_BF16 if q.dtype == torch.bfloat16 else KLA_FP32, m)
    if out is None:
        out = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    s = lib().kla_decode_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                              _ptr(lam), _ptr(eta), _ptr(out), _stream())
    _check(s, "kla_decode_step")
    return out


def host_device_bytes(desc: KlaDesc) -> int:
    return int(lib().kla_host_device_bytes(ctypes.byref(desc)))


def forward_host(desc: KlaDesc, q, k, v, a, qn, beta, out, lambda0=None, eta0=None,
                 final_lambda=None, final_eta=None, device_buffer=None, stream=None):
    """kla_forward_host on CPU tensors (pinned for asynchronous copies). The
    call copies inputs in, runs, copies results out and synchronises."""
    nbytes = host_device_bytes(desc)
    if device_buffer is None:
        device_buffer = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    s = lib().kla_forward_host(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                               _ptr(lambda0), _ptr(eta0), _ptr(out), _ptr(final_lambda), _ptr(final_eta),
                               _ptr(device_buffer), nbytes, st)
    _check(s, "kla_forward_host")
    return out


def forward_noalloc(q, k, v, a, qn, beta, lambda0=None, eta0=None, B=None, T=None, mode="diag",
                    final_state=False, out=None):
    """kla_forward_noalloc: the forward pass with the library's fixed device
    scratch area as workspace, for callers that cannot allocate device memory
    (outputs passed in via ``out`` are used as given)."""
    m = _mode(mode)
    desc, N = _desc_from(q, v, B, T, m, None)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    if out is None:
        out = torch.empty(q.shape[0], H, dv, dtype=q.dtype, device=q.device)
    fl = fe = None
    if final_state:
        fl = torch.empty((N, H) if m == KLA_ISO else (N, H, dk), dtype=torch.float32, device=q.device)
        fe = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    s = lib().kla_forward_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(qn), _ptr(beta),
                                  _ptr(lambda0), _ptr(eta0), _ptr(out), _ptr(fl), _ptr(fe), _stream())
    _check(s, "kla_forward_noalloc")
    return (out, fl, fe) if final_state else out


# ---- the recurrent block around the mixers: short convolution, selective scan, layer norm ----

_F32, _DTYPES = torch.float32, {torch.bfloat16: KLA_BF16, torch.float32: KLA_FP32}


def _p(t):
    return None if t is None else t.data_ptr()


# the current stream's handle on a device, without the object around it where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _enqueue(fn, x, *args):
    """Calls the library for tensors on x's device: that device made current, the work
    on its current stream."""
    index = x.get_device()
    if index == torch.cuda.current_device():
        s = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            s = fn(*args, _raw_stream(index))
    if s != KLA_OK:
        raise KlaError(s, fn.__name__)


def _bytes(fn, x, *args):
    """A size that the library computes for x's device."""
    if x.get_device() == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(x.get_device()):
        return fn(*args)


def _io_dtype(x):
    if not x.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError("token tensors must be bfloat16 or float32")
    return dt


def _tokens(name, t, like, shape):
    """A token tensor: like's dtype and device, the given shape, rows at one
    stride with contiguous values. Returns the token stride, or 0 for a
    contiguous tensor."""
    if (t.dtype is like.dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == like.get_device()):
        return 0
    if t.dtype is not like.dtype:
        raise TypeError("%s must have the dtype of x" % name)
    if t.get_device() != like.get_device():
        raise ValueError("%s must be on the device of x" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    st, width = t.stride(), 1
    for n, k in zip(reversed(shape[1:]), reversed(st[1:])):
        if n > 1 and k != width:
            raise ValueError("the values of a row of %s must be contiguous" % name)
        width *= n
    if shape[0] <= 1:
        return 0
    if st[0] < width:
        raise ValueError("rows of %s must not overlap" % name)
    return st[0]


def _dense(name, t, like, shape, dtype=_F32):
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                     and t.get_device() == like.get_device()):
        return
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (name, str(dtype).replace("torch.", "")))
    if t.get_device() != like.get_device():
        raise ValueError("%s must be on the device of x" % name)
    raise ValueError("%s must be contiguous with shape %s" % (name, tuple(shape)))


def _axis(x, cu_seqlens, B, T):
    """(rows, tokens per row, offsets pointer, packed sequences, sequences) of the token axis of x."""
    n = x.shape[0]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device:
            raise TypeError("cu_seqlens must be an int32 tensor on the device of x")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous with at least two offsets")
        if B is not None or T is not None:
            raise ValueError("B and T do not go with cu_seqlens")
        k = cu_seqlens.numel() - 1
        return 1, n, cu_seqlens.data_ptr(), k, k
    if B is None:
        B = 1 if T is None else (n // T if T else 0)
    if T is None:
        T = n // B if B else 0
    if B < 0 or T < 0 or B * T != n:
        raise ValueError("B*T must equal the number of tokens")
    return B, T, None, 0, B


def _out_like(name, out, x, shape):
    if out is None:
        return torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)
    _dense(name, out, x, shape, x.dtype)
    return out


def _conv(x, weight, bias, cu_seqlens, B, T, silu):
    dt = _io_dtype(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [Ntok, D] and weight [D, W]")
    D, W = x.shape[1], weight.shape[1]
    if not 1 <= W <= 4:
        raise ValueError("a convolution has 1 to 4 taps")
    ld = _tokens("x", x, x, x.shape)
    _dense("weight", weight, x, (D, W))
    _dense("bias", bias, x, (D,))
    b, t, cu, k, N = _axis(x, cu_seqlens, B, T)
    return KlaConvDesc(b, t, D, W, dt, 1 if silu else 0, cu, k, ld), D, W, N


def conv_forward(x, weight, bias=None, state0=None, cu_seqlens=None, B=None, T=None, silu=True, final_state=False,
                 out=None):
    """Short causal convolution with SiLU (include/kla.h kla_conv_forward): x
    [Ntok, D] (rows may be strided), weight [D, W], bias [D]; the history state0
    [N, W-1, D] holds the inputs before each sequence. Returns ``out`` or
    ``(out, state)`` with ``final_state``: the history after each sequence. Rows of
    tokens outside the offsets are 0 in a new ``out``, and stay in a given one."""
    d, D, W, N = _conv(x, weight, bias, cu_seqlens, B, T, silu)
    d.zero_rest = out is None
    _dense("state0", state0, x, (N, W - 1, D), x.dtype)
    out = _out_like("out", out, x, (x.shape[0], D))
    fs = x.new_empty((N, W - 1, D)) if final_state else None
    _enqueue(lib().kla_conv_forward, x, ctypes.byref(d), x.data_ptr(), weight.data_ptr(), _p(bias), _p(state0),
             out.data_ptr(), _p(fs))
    return (out, fs) if final_state else out


def conv_backward(x, weight, dout, bias=None, state0=None, dfinal_state=None, cu_seqlens=None, B=None, T=None,
                  silu=True, workspace=None):
    """Gradients of ``conv_forward`` (include/kla.h kla_conv_backward): a dict of
    ``dx`` and ``dstate0`` (x's dtype; dstate0 only with a state0) and ``dweight``,
    ``dbias`` (fp32). Tokens outside the offsets have gradient 0."""
    d, D, W, N = _conv(x, weight, bias, cu_seqlens, B, T, silu)
    d.zero_rest = 1
    _dense("dout", dout, x, (x.shape[0], D), x.dtype)
    _dense("state0", state0, x, (N, W - 1, D), x.dtype)
    _dense("dfinal_state", dfinal_state, x, (N, W - 1, D), x.dtype)
    f32 = dict(dtype=_F32)
    g = {"dx": x.new_empty((x.shape[0], D)), "dweight": x.new_empty((D, W), **f32),
         "dbias": x.new_empty(D, **f32)}
    if state0 is not None:
        g["dstate0"] = x.new_empty((N, W - 1, D))
    need = _bytes(lib().kla_conv_backward_workspace_bytes, x, ctypes.byref(d))
    workspace = _workspace(workspace, need, x)
    _enqueue(lib().kla_conv_backward, x, ctypes.byref(d), x.data_ptr(), weight.data_ptr(), _p(bias), _p(state0),
             dout.data_ptr(), _p(dfinal_state), g["dx"].data_ptr(), g["dweight"].data_ptr(), g["dbias"].data_ptr(),
             _p(g.get("dstate0")), workspace.data_ptr(), workspace.numel())
    return g


def _workspace(ws, need, x):
    if ws is None:
        return x.new_empty(max(need, 16), dtype=torch.uint8)
    if ws.dtype != torch.uint8 or ws.device != x.device or not ws.is_contiguous() or ws.numel() < need:
        raise ValueError("workspace must be a contiguous uint8 tensor of at least %d bytes on the device of x" % need)
    return ws


def conv_step(x, weight, state, bias=None, silu=True, out=None):
    """One token per row: x [B, D]; ``state`` [B, W-1, D] is shifted in place.
    Returns out [B, D]."""
    d, D, W, N = _conv(x, weight, bias, None, x.shape[0], 1, silu)
    _dense("state", state, x, (N, W - 1, D), x.dtype)
    out = _out_like("out", out, x, (N, D))
    _enqueue(lib().kla_conv_step, x, ctypes.byref(d), x.data_ptr(), weight.data_ptr(), _p(bias), _p(state),
             out.data_ptr())
    return out


def _ssm(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens, B, T, softplus):
    io = _io_dtype(x)
    if x.dim() != 2 or A.dim() != 2 or Bm.dim() != 3:
        raise ValueError("x must be [Ntok, D], A [D, N], Bm and Cm [Ntok, G, N]")
    n, ch = x.shape
    G, N = Bm.shape[1], A.shape[1]
    if G < 1 or ch % G:
        raise ValueError("the groups of Bm must divide the channels")
    shape = x.shape
    ld = (_tokens("x", x, x, shape), _tokens("dt", dt, x, shape),
          _tokens("z", z, x, shape) if z is not None else 0,
          _tokens("Bm", Bm, x, (n, G, N)), _tokens("Cm", Cm, x, (n, G, N)))
    _dense("A", A, x, (ch, N))
    _dense("D", D, x, (ch,))
    _dense("dt_bias", dt_bias, x, (ch,))
    b, t, cu, k, seqs = _axis(x, cu_seqlens, B, T)
    return KlaSsmDesc(b, t, ch, G, N, io, 1 if softplus else 0, cu, k, *ld), ch, N, G, seqs


def ssm_forward(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state0=None, cu_seqlens=None, B=None, T=None,
                softplus=True, final_state=False, save_states=False, out=None):
    """Selective state space scan (include/kla.h kla_ssm_forward): x, dt, z
    [Ntok, D], Bm, Cm [Ntok, G, N] (rows may be strided), A [D, N], D and dt_bias
    [D], state0 [Nseq, D, N]. Returns ``out``, then the final state with
    ``final_state``, then what ``ssm_backward`` takes as ``states`` with
    ``save_states``. Rows of tokens outside the offsets are 0 in a new ``out``, and
    stay in a given one."""
    d, ch, N, G, seqs = _ssm(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens, B, T, softplus)
    d.zero_rest = out is None
    _dense("state0", state0, x, (seqs, ch, N))
    out = _out_like("out", out, x, (x.shape[0], ch))
    fs = x.new_empty((seqs, ch, N), dtype=_F32) if final_state else None
    st = None
    if save_states:
        st = x.new_empty(lib().kla_ssm_states_bytes(ctypes.byref(d)) // 4, dtype=_F32)
    _enqueue(lib().kla_ssm_forward, x, ctypes.byref(d), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
             Cm.data_ptr(), _p(D), _p(z), _p(dt_bias), _p(state0), out.data_ptr(), _p(fs), _p(st))
    res = (out,) + ((fs,) if final_state else ()) + ((st,) if save_states else ())
    return res if len(res) > 1 else out


def ssm_backward(x, dt, A, Bm, Cm, dout, D=None, z=None, dt_bias=None, state0=None, dfinal_state=None, states=None,
                 cu_seqlens=None, B=None, T=None, softplus=True, workspace=None):
    """Gradients of ``ssm_forward`` (include/kla.h kla_ssm_backward): a dict of
    ``dx, ddt, dBm, dCm`` and ``dz`` (with z) in x's dtype, and ``dA, dD,
    ddt_bias, dstate0`` in fp32. ``states``: what the forward call returned with
    ``save_states`` for the same inputs (walked again without). Tokens outside the
    offsets have gradient 0."""
    d, ch, N, G, seqs = _ssm(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens, B, T, softplus)
    d.zero_rest = 1
    n = x.shape[0]
    _dense("dout", dout, x, (n, ch), x.dtype)
    _dense("state0", state0, x, (seqs, ch, N))
    _dense("dfinal_state", dfinal_state, x, (seqs, ch, N))
    L = lib()
    if states is not None:
        _dense("states", states, x, (L.kla_ssm_states_bytes(ctypes.byref(d)) // 4,))
    f32 = dict(dtype=_F32)
    g = {"dx": x.new_empty((n, ch)), "ddt": x.new_empty((n, ch)),
         "dBm": x.new_empty((n, G, N)), "dCm": x.new_empty((n, G, N)),
         "dA": x.new_empty((ch, N), **f32), "dD": x.new_empty(ch, **f32), "ddt_bias": x.new_empty(ch, **f32),
         "dstate0": x.new_empty((seqs, ch, N), **f32)}
    if z is not None:
        g["dz"] = x.new_empty((n, ch))
    need = _bytes(L.kla_ssm_backward_workspace_bytes, x, ctypes.byref(d), states is not None)
    workspace = _workspace(workspace, need, x)
    _enqueue(L.kla_ssm_backward, x, ctypes.byref(d), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
             Cm.data_ptr(), _p(D), _p(z), _p(dt_bias), _p(state0), _p(states), dout.data_ptr(), _p(dfinal_state),
             g["dx"].data_ptr(), g["ddt"].data_ptr(), g["dA"].data_ptr(), g["dBm"].data_ptr(), g["dCm"].data_ptr(),
             g["dD"].data_ptr(), _p(g.get("dz")), g["ddt_bias"].data_ptr(), g["dstate0"].data_ptr(),
             workspace.data_ptr(), workspace.numel())
    return g


def ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, softplus=True, out=None):
    """One token per row through the scan: x, dt, z [B, D], Bm, Cm [B, G, N];
    ``state`` [B, D, N] is updated in place. Returns out [B, D]."""
    d, ch, N, G, seqs = _ssm(x, dt, A, Bm, Cm, D, z, dt_bias, None, x.shape[0], 1, softplus)
    _dense("state", state, x, (seqs, ch, N))
    out = _out_like("out", out, x, (seqs, ch))
    _enqueue(lib().kla_ssm_step, x, ctypes.byref(d), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
             Cm.data_ptr(), _p(D), _p(z), _p(dt_bias), state.data_ptr(), out.data_ptr())
    return out


def _norm(x, weight, bias, residual, eps):
    dt = _io_dtype(x)
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("x must be [rows, D]")
    shape = x.shape
    ld = _tokens("x", x, x, shape)
    ld_r = _tokens("residual", residual, x, shape) if residual is not None else 0
    _dense("weight", weight, x, shape[1:])
    _dense("bias", bias, x, shape[1:])
    return KlaNormDesc(shape[0], shape[1], dt, eps, ld, ld_r), shape


def layernorm_forward(x, weight=None, bias=None, residual=None, eps=1e-5, stats=False, out=None, sum_out=None):
    """Layer norm over the last axis of x [rows, D], or of x + residual
    (include/kla.h kla_layernorm_forward). Returns ``out``, then the sum with a
    residual, then ``mean, rstd`` with ``stats``."""
    d, shape = _norm(x, weight, bias, residual, eps)
    if sum_out is not None and residual is None:
        raise ValueError("sum_out goes with a residual")
    out = _out_like("out", out, x, shape)
    total = _out_like("sum_out", sum_out, x, shape) if residual is not None else None
    mean = rstd = None
    if stats:
        mean = x.new_empty(shape[0], dtype=_F32)
        rstd = x.new_empty(shape[0], dtype=_F32)
    _enqueue(lib().kla_layernorm_forward, x, ctypes.byref(d), x.data_ptr(), _p(residual), _p(weight), _p(bias),
             out.data_ptr(), _p(total), _p(mean), _p(rstd))
    res = (out,) + ((total,) if residual is not None else ()) + ((mean, rstd) if stats else ())
    return res if len(res) > 1 else out


def layernorm_backward(x, dout, mean, rstd, weight=None, dsum=None, workspace=None):
    """Gradients of ``layernorm_forward`` (include/kla.h kla_layernorm_backward): x
    is the tensor that was normalised (the sum, with a residual) and dsum the
    gradient that reaches it past the norm. A dict of ``dx`` (x's dtype; of the
    residual alike) and ``dweight``, ``dbias`` (fp32)."""
    d, shape = _norm(x, weight, None, None, 1.0)
    _dense("mean", mean, x, shape[:1])
    _dense("rstd", rstd, x, shape[:1])
    _dense("dout", dout, x, shape, x.dtype)
    _dense("dsum", dsum, x, shape, x.dtype)
    f32 = dict(dtype=_F32)
    g = {"dx": x.new_empty(shape), "dweight": x.new_empty(shape[1], **f32),
         "dbias": x.new_empty(shape[1], **f32)}
    workspace = _workspace(workspace, _bytes(lib().kla_layernorm_backward_workspace_bytes, x, ctypes.byref(d)), x)
    _enqueue(lib().kla_layernorm_backward, x, ctypes.byref(d), x.data_ptr(), _p(weight), _p(mean), _p(rstd),
             dout.data_ptr(), _p(dsum), g["dx"].data_ptr(), g["dweight"].data_ptr(), g["dbias"].data_ptr(),
             workspace.data_ptr(), workspace.numel())
    return g


def check(stream=None):
    """Synchronise and read the device status word (raises on an error)."""
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    _check(lib().kla_check(st), "kla_check")
