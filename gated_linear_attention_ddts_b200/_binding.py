"""ctypes binding of librdm_ddts.so (include/rdm_ddts.h).

Argument marshalling only: torch tensors become device pointers, the current
torch stream becomes the cudaStream_t, statuses become exceptions.  Every step
of the computation runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librdm_ddts.so")

RDM_OK, RDM_ERR_INVALID_ARG, RDM_ERR_UNSUPPORTED, RDM_ERR_CUDA, RDM_ERR_TIMEOUT, \
    RDM_ERR_WORKSPACE = range(6)
RDM_F32, RDM_BF16 = 0, 1
IMPL = {"auto": 0, "simt": 1, "tc": 2, 0: 0, 1: 1, 2: 2}
# what g, tau, beta hold: the gates, or their pre-activations (softplus, sigmoid,
# sigmoid applied inside; gradients then refer to the pre-activations)
GATES = {"activated": 0, "preact": 1, 0: 0, 1: 1}

_VP = ctypes.c_void_p
_I = ctypes.c_int


class FwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("dk", _I), ("dv", _I), ("chunk", _I),
                ("dtype", _I), ("impl", _I),
                ("q", _VP), ("k", _VP), ("v", _VP), ("g", _VP), ("tau", _VP), ("beta", _VP),
                ("S0", _VP), ("o", _VP), ("ST", _VP), ("saved_states", _VP),
                ("workspace", _VP), ("workspace_bytes", ctypes.c_size_t), ("gate_inputs", _I),
                ("feedthrough", _VP), ("beta_rank", _I), ("beta_u", _VP), ("beta_w", _VP)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("dk", _I), ("dv", _I), ("chunk", _I),
                ("dtype", _I), ("impl", _I),
                ("q", _VP), ("k", _VP), ("v", _VP), ("g", _VP), ("tau", _VP), ("beta", _VP),
                ("S0", _VP), ("grad_o", _VP), ("grad_ST", _VP), ("saved_states", _VP),
                ("grad_q", _VP), ("grad_k", _VP), ("grad_v", _VP), ("grad_g", _VP),
                ("grad_tau", _VP), ("grad_beta", _VP), ("grad_S0", _VP),
                ("workspace", _VP), ("workspace_bytes", ctypes.c_size_t), ("gate_inputs", _I),
                ("feedthrough", _VP), ("grad_feedthrough", _VP), ("beta_rank", _I),
                ("beta_u", _VP), ("beta_w", _VP), ("grad_beta_u", _VP), ("grad_beta_w", _VP)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("dk", _I), ("dv", _I), ("dtype", _I),
                ("q", _VP), ("k", _VP), ("v", _VP), ("g", _VP), ("tau", _VP), ("beta", _VP),
                ("S", _VP), ("o", _VP), ("feedthrough", _VP)]


class ConvArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("D", _I), ("W", _I), ("dtype", _I), ("silu", _I),
                ("x", _VP), ("weight", _VP), ("bias", _VP), ("state_in", _VP), ("y", _VP),
                ("state_out", _VP)]


class ConvBwdArgs(ctypes.Structure):
    _fields_ = [("fwd", ConvArgs), ("grad_y", _VP), ("grad_state_out", _VP), ("grad_x", _VP),
                ("grad_weight", _VP), ("grad_bias", _VP), ("grad_state_in", _VP)]


class SkaFwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("dk", _I), ("dv", _I), ("window", _I),
                ("scale", ctypes.c_float), ("dtype", _I), ("q", _VP), ("k", _VP), ("v", _VP),
                ("o", _VP), ("k_cache", _VP), ("v_cache", _VP), ("pos", _VP)]


class SkaDecodeArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("dk", _I), ("dv", _I), ("window", _I),
                ("scale", ctypes.c_float), ("dtype", _I), ("q", _VP), ("k", _VP), ("v", _VP),
                ("k_cache", _VP), ("v_cache", _VP), ("pos", _VP), ("advance_pos", _I), ("o", _VP)]


class SsmArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("G", _I), ("T", _I), ("D", _I), ("N", _I), ("W", _I), ("dtype", _I),
                ("gate_inputs", _I), ("conv_silu", _I), ("x", _VP), ("dt", _VP), ("Bm", _VP), ("Cm", _VP),
                ("z", _VP), ("A", _VP), ("dt_bias", _VP), ("feedthrough", _VP), ("conv_weight", _VP),
                ("conv_bias", _VP), ("conv_state_in", _VP), ("S0", _VP), ("lengths", _VP), ("y", _VP),
                ("ST", _VP), ("conv_state_out", _VP), ("saved_states", _VP), ("workspace", _VP),
                ("workspace_bytes", ctypes.c_size_t)]


class SsmBwdArgs(ctypes.Structure):
    _fields_ = [("fwd", SsmArgs), ("grad_y", _VP), ("grad_ST", _VP), ("grad_conv_state_out", _VP),
                ("grad_x", _VP), ("grad_dt", _VP), ("grad_z", _VP), ("grad_B", _VP), ("grad_C", _VP),
                ("grad_A", _VP), ("grad_dt_bias", _VP), ("grad_feedthrough", _VP), ("grad_conv_weight", _VP),
                ("grad_conv_bias", _VP), ("grad_S0", _VP), ("grad_conv_state_in", _VP)]


class SsmStepArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("G", _I), ("D", _I), ("N", _I), ("W", _I), ("dtype", _I),
                ("gate_inputs", _I), ("conv_silu", _I), ("x", _VP), ("dt", _VP), ("Bm", _VP), ("Cm", _VP),
                ("z", _VP), ("A", _VP), ("dt_bias", _VP), ("feedthrough", _VP), ("conv_weight", _VP),
                ("conv_bias", _VP), ("S", _VP), ("conv_state", _VP), ("y", _VP)]


class SkaQ8Cache(ctypes.Structure):
    _fields_ = [("B", _I), ("H", _I), ("dk", _I), ("dv", _I), ("window", _I), ("block", _I), ("type", _I),
                ("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("k_tail", _VP), ("v_tail", _VP),
                ("pos", _VP)]


class SkaQ8FillArgs(ctypes.Structure):
    _fields_ = [("cache", SkaQ8Cache), ("T", _I), ("dtype", _I), ("k", _VP), ("v", _VP), ("lengths", _VP)]


class SkaQ8DecodeArgs(ctypes.Structure):
    _fields_ = [("cache", SkaQ8Cache), ("scale", ctypes.c_float), ("dtype", _I), ("q", _VP), ("k", _VP),
                ("v", _VP), ("o", _VP), ("advance_pos", _I), ("workspace", _VP),
                ("workspace_bytes", ctypes.c_size_t)]


class RdmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None

EXPORTS = ["rdm_ddts_fwd", "rdm_ddts_fwd_workspace_size", "rdm_ddts_saved_states_size", "rdm_ddts_bwd",
           "rdm_ddts_bwd_workspace_size", "rdm_ddts_bwd_noalloc", "rdm_ddts_decode_step", "rdm_ddts_decode",
           "rdm_ddts_sync_status",
           "rdm_status_string", "rdm_ddts_set_test_hooks", "rdm_ddts_version", "rdm_shortconv_fwd",
           "rdm_shortconv_bwd", "rdm_shortconv_fwd_many", "rdm_shortconv_bwd_many", "rdm_ska_fwd",
           "rdm_ska_decode", "rdm_ssm_fwd", "rdm_ssm_fwd_workspace_size", "rdm_ssm_saved_states_size",
           "rdm_ssm_bwd", "rdm_ssm_bwd_workspace_size", "rdm_ssm_step", "rdm_ska_q8_fill",
           "rdm_ska_q8_decode", "rdm_ska_q8_decode_workspace_size"]


def load():
    """Open librdm_ddts.so and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "`python -m gated_linear_attention_ddts_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        lib.rdm_ddts_fwd.argtypes = [ctypes.POINTER(FwdArgs), _VP]
        lib.rdm_ddts_fwd.restype = _I
        lib.rdm_ddts_fwd_workspace_size.argtypes = [ctypes.POINTER(FwdArgs)]
        lib.rdm_ddts_fwd_workspace_size.restype = ctypes.c_size_t
        lib.rdm_ddts_saved_states_size.argtypes = [_I] * 6
        lib.rdm_ddts_saved_states_size.restype = ctypes.c_size_t
        lib.rdm_ddts_bwd.argtypes = [ctypes.POINTER(BwdArgs), _VP]
        lib.rdm_ddts_bwd.restype = _I
        lib.rdm_ddts_bwd_workspace_size.argtypes = [ctypes.POINTER(BwdArgs)]
        lib.rdm_ddts_bwd_workspace_size.restype = ctypes.c_size_t
        lib.rdm_ddts_bwd_noalloc.argtypes = [ctypes.POINTER(BwdArgs), _VP]
        lib.rdm_ddts_bwd_noalloc.restype = _I
        lib.rdm_ddts_decode_step.argtypes = [_I] * 5 + [_VP] * 9
        lib.rdm_ddts_decode_step.restype = _I
        lib.rdm_ddts_decode.argtypes = [ctypes.POINTER(DecodeArgs), _VP]
        lib.rdm_ddts_decode.restype = _I
        lib.rdm_ddts_sync_status.argtypes = [_VP]
        lib.rdm_ddts_sync_status.restype = _I
        lib.rdm_status_string.argtypes = [_I]
        lib.rdm_status_string.restype = ctypes.c_char_p
        lib.rdm_shortconv_fwd.argtypes = [ctypes.POINTER(ConvArgs), _VP]
        lib.rdm_shortconv_fwd.restype = _I
        lib.rdm_shortconv_bwd.argtypes = [ctypes.POINTER(ConvBwdArgs), _VP]
        lib.rdm_shortconv_bwd.restype = _I
        lib.rdm_shortconv_fwd_many.argtypes = [ctypes.POINTER(ConvArgs), _I, _VP]
        lib.rdm_shortconv_fwd_many.restype = _I
        lib.rdm_shortconv_bwd_many.argtypes = [ctypes.POINTER(ConvBwdArgs), _I, _VP]
        lib.rdm_shortconv_bwd_many.restype = _I
        lib.rdm_ska_fwd.argtypes = [ctypes.POINTER(SkaFwdArgs), _VP]
        lib.rdm_ska_fwd.restype = _I
        lib.rdm_ska_decode.argtypes = [ctypes.POINTER(SkaDecodeArgs), _VP]
        lib.rdm_ska_decode.restype = _I
        for name, args in (("rdm_ssm_fwd", SsmArgs), ("rdm_ssm_bwd", SsmBwdArgs)):
            fn, size = getattr(lib, name), getattr(lib, name + "_workspace_size")
            fn.argtypes = [ctypes.POINTER(args), _VP]
            fn.restype = _I
            size.argtypes = [ctypes.POINTER(args)]
            size.restype = ctypes.c_size_t
        lib.rdm_ssm_saved_states_size.argtypes = [_I] * 5
        lib.rdm_ssm_saved_states_size.restype = ctypes.c_size_t
        lib.rdm_ssm_step.argtypes = [ctypes.POINTER(SsmStepArgs), _VP]
        lib.rdm_ssm_step.restype = _I
        lib.rdm_ska_q8_fill.argtypes = [ctypes.POINTER(SkaQ8FillArgs), _VP]
        lib.rdm_ska_q8_fill.restype = _I
        lib.rdm_ska_q8_decode.argtypes = [ctypes.POINTER(SkaQ8DecodeArgs), _VP]
        lib.rdm_ska_q8_decode.restype = _I
        lib.rdm_ska_q8_decode_workspace_size.argtypes = [ctypes.POINTER(SkaQ8DecodeArgs)]
        lib.rdm_ska_q8_decode_workspace_size.restype = ctypes.c_size_t
        lib.rdm_ddts_set_test_hooks.argtypes = [ctypes.c_longlong, _I]
        lib.rdm_ddts_set_test_hooks.restype = _I
        lib.rdm_ddts_version.argtypes = []
        lib.rdm_ddts_version.restype = _I
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().rdm_status_string(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RDM_BF16
    if t.dtype == torch.float32:
        return RDM_F32
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _check(status: int, where: str):
    if status != RDM_OK:
        raise RdmError(status, where)


def rdm_ddts_saved_states_size(B, H, T, dk, dv, chunk=0) -> int:
    return int(load().rdm_ddts_saved_states_size(B, H, T, dk, dv, chunk))


def _lowrank(beta_lowrank):
    """(rank, u, w) of a low-rank beta_hat given as (u [B,T,r], w_up [H,r,dv])."""
    if beta_lowrank is None:
        return 0, None, None
    u, w = beta_lowrank
    return int(u.shape[-1]), u, w


def _fwd_args(q, k, v, g, tau, beta, S0, o, ST, saved_states, ws, ws_bytes, chunk, impl,
              gates="activated", feedthrough=None, beta_lowrank=None):
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    r, u, w = _lowrank(beta_lowrank)
    return FwdArgs(B, H, T, dk, dv, chunk, _dtype_code(q), IMPL[impl],
                   _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(tau), _ptr(beta), _ptr(S0), _ptr(o),
                   _ptr(ST), _ptr(saved_states), _ptr(ws), ws_bytes, GATES[gates],
                   _ptr(feedthrough), r, _ptr(u), _ptr(w))


def rdm_ddts_fwd_workspace_size(q, k, v, g, tau, beta, *, chunk=0, impl="auto",
                                gates="activated", beta_lowrank=None) -> int:
    a = _fwd_args(q, k, v, g, tau, beta, None, None, None, None, None, 0, chunk, impl, gates,
                  None, beta_lowrank)
    n = load().rdm_ddts_fwd_workspace_size(ctypes.byref(a))
    if n == ctypes.c_size_t(-1).value:
        raise RdmError(RDM_ERR_INVALID_ARG, "rdm_ddts_fwd_workspace_size")
    return int(n)


def rdm_ddts_fwd(q, k, v, g, tau, beta, S0=None, o=None, ST=None, saved_states=None, *,
                 workspace=None, chunk=0, impl="auto", return_state=False, stream=None,
                 gates="activated", feedthrough=None, beta_lowrank=None):
    """Forward over [B,H,T,D] sequences.  Allocates o (and S_T when
    return_state) with torch if not given, and the sequence-segment workspace
    when none is passed (workspace=False runs without one).  feedthrough: [H,dv]
    float32 weights d, o_t += d * v_t.  beta_lowrank: (u [B,T,r], w_up [H,r,dv]
    float32) for beta_hat = sigmoid(u . w_up) (gates="preact"; beta unused, may
    be None).  Returns (o, S_T or None)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if ST is None and return_state:
        ST = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if workspace is None:
        need = rdm_ddts_fwd_workspace_size(q, k, v, g, tau, beta, chunk=chunk, impl=impl,
                                           gates=gates, beta_lowrank=beta_lowrank)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    elif workspace is False:
        workspace = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a = _fwd_args(q, k, v, g, tau, beta, S0, o, ST, saved_states, workspace, ws_bytes, chunk,
                  impl, gates, feedthrough, beta_lowrank)
    _check(load().rdm_ddts_fwd(ctypes.byref(a), _stream(stream)), "rdm_ddts_fwd")
    return o, ST


def _bwd_args(q, k, v, g, tau, beta, S0, grad_o, grad_ST, saved_states, grads, ws, ws_bytes,
              chunk, impl, gates="activated", feedthrough=None, beta_lowrank=None):
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    r, u, w = _lowrank(beta_lowrank)
    return BwdArgs(B, H, T, dk, dv, chunk, _dtype_code(q), IMPL[impl],
                   _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(tau), _ptr(beta), _ptr(S0),
                   _ptr(grad_o), _ptr(grad_ST), _ptr(saved_states),
                   *(_ptr(grads.get(n)) for n in ("dq", "dk", "dv", "dg", "dtau", "dbeta",
                                                    "dS0")),
                   _ptr(ws), ws_bytes, GATES[gates], _ptr(feedthrough), _ptr(grads.get("dfeed")),
                   r, _ptr(u), _ptr(w), _ptr(grads.get("du")), _ptr(grads.get("dw_up")))


def _alloc_grads(grads, q, k, v, g, tau, beta, beta_lowrank):
    refs = [("dq", q), ("dk", k), ("dg", g), ("dtau", tau), ("dv", v)]
    if beta_lowrank is None:
        refs.append(("dbeta", beta))
    else:
        refs += [("du", beta_lowrank[0]), ("dw_up", beta_lowrank[1])]
    for n, ref in refs:
        if grads.get(n) is None:
            grads[n] = torch.empty_like(ref)


def rdm_ddts_bwd_workspace_size(q, k, v, g, tau, beta, S0=None, grad_o=None, grad_ST=None,
                                saved_states=None, *, chunk=0, impl="auto",
                                gates="activated", beta_lowrank=None) -> int:
    a = _bwd_args(q, k, v, g, tau, beta, S0, grad_o, grad_ST, saved_states, {}, None, 0,
                  chunk, impl, gates, None, beta_lowrank)
    n = load().rdm_ddts_bwd_workspace_size(ctypes.byref(a))
    if n == ctypes.c_size_t(-1).value:
        raise RdmError(RDM_ERR_INVALID_ARG, "rdm_ddts_bwd_workspace_size")
    return int(n)


def rdm_ddts_bwd(q, k, v, g, tau, beta, S0, grad_o, grad_ST=None, saved_states=None, *,
                 grads=None, workspace=None, chunk=0, impl="auto", want_dS0=True, stream=None,
                 gates="activated", feedthrough=None, beta_lowrank=None):
    """Backward.  `grads` may hold preallocated dq, dk, dv, dg, dtau, dbeta, dS0
    (and dfeed when feedthrough is given; du and dw_up in place of dbeta with
    beta_lowrank); missing ones are allocated with torch, as is the workspace.
    Returns the dict."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    grads = dict(grads or {})
    _alloc_grads(grads, q, k, v, g, tau, beta, beta_lowrank)
    if want_dS0 and grads.get("dS0") is None:
        grads["dS0"] = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if feedthrough is not None and grads.get("dfeed") is None:
        grads["dfeed"] = torch.empty(H, dv, dtype=torch.float32, device=q.device)
    if workspace is None:
        need = rdm_ddts_bwd_workspace_size(q, k, v, g, tau, beta, S0, grad_o, grad_ST,
                                           saved_states, chunk=chunk, impl=impl, gates=gates,
                                           beta_lowrank=beta_lowrank)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    a = _bwd_args(q, k, v, g, tau, beta, S0, grad_o, grad_ST, saved_states, grads, workspace,
                  workspace.numel() * workspace.element_size(), chunk, impl, gates, feedthrough,
                  beta_lowrank)
    _check(load().rdm_ddts_bwd(ctypes.byref(a), _stream(stream)), "rdm_ddts_bwd")
    return grads


def rdm_ddts_bwd_noalloc(q, k, v, g, tau, beta, S0, grad_o, grad_ST=None, *, grads=None,
                         chunk=0, want_dS0=True, stream=None, gates="activated", beta_lowrank=None):
    """Backward through the library's own fixed scratch (no workspace
    argument).  Gradient tensors are allocated with torch if not given;
    returns the dict of gradients."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    grads = dict(grads or {})
    _alloc_grads(grads, q, k, v, g, tau, beta, beta_lowrank)
    if want_dS0 and grads.get("dS0") is None:
        grads["dS0"] = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    a = _bwd_args(q, k, v, g, tau, beta, S0, grad_o, grad_ST, None, grads, None, 0, chunk, "simt",
                  gates, None, beta_lowrank)
    _check(load().rdm_ddts_bwd_noalloc(ctypes.byref(a), _stream(stream)), "rdm_ddts_bwd_noalloc")
    return grads


def rdm_ddts_decode_step(q, k, v, g, tau, beta, S, o=None, *, stream=None):
    """One token per (b,h): q,k,g,tau [B,H,dk], v,beta [B,H,dv]; S [B,H,dk,dv]
    float32 updated in place.  Returns o [B,H,dv]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    st = load().rdm_ddts_decode_step(B, H, dk, dv, _dtype_code(q), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(g), _ptr(tau), _ptr(beta), _ptr(S), _ptr(o),
                                     _stream(stream))
    _check(st, "rdm_ddts_decode_step")
    return o


def rdm_ddts_decode(q, k, v, g, tau, beta, S, o=None, *, feedthrough=None, stream=None):
    """rdm_ddts_decode_step with the feedthrough: o = S^T q + d * v when
    feedthrough ([H,dv] float32) is given."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    a = DecodeArgs(B, H, dk, dv, _dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(tau),
                   _ptr(beta), _ptr(S), _ptr(o), _ptr(feedthrough))
    _check(load().rdm_ddts_decode(ctypes.byref(a), _stream(stream)), "rdm_ddts_decode")
    return o


def _conv_args(x, weight, bias, state_in, y, state_out, silu):
    B, H, T, D = x.shape
    return ConvArgs(B, H, T, D, weight.shape[-1], _dtype_code(x), int(bool(silu)), _ptr(x),
                    _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(y), _ptr(state_out))


def rdm_shortconv_fwd(x, weight, bias=None, state_in=None, *, silu=False, y=None,
                      return_state=False, stream=None):
    """Causal depthwise short convolution along the tokens: x [B,H,T,D], weight
    [H,D,W] float32, bias [H,D] float32, state_in [B,H,W-1,D] (the previous
    W-1 inputs).  Returns (y, state_out or None)."""
    B, H, T, D = x.shape
    W = weight.shape[-1]
    if y is None:
        y = torch.empty_like(x)
    state_out = torch.empty(B, H, W - 1, D, dtype=x.dtype, device=x.device) if return_state else None
    a = _conv_args(x, weight, bias, state_in, y, state_out, silu)
    _check(load().rdm_shortconv_fwd(ctypes.byref(a), _stream(stream)), "rdm_shortconv_fwd")
    return y, state_out


def rdm_shortconv_bwd(x, weight, bias, state_in, grad_y, grad_state_out=None, *, silu=False,
                      out=None, stream=None):
    """Reverse mode of rdm_shortconv_fwd.  Returns dict dx, dw, dbias (None
    without bias) and dxs (None without state_in); `out` may hold them
    preallocated."""
    out = dict(out or {})
    if out.get("dx") is None:
        out["dx"] = torch.empty_like(x)
    if out.get("dw") is None:
        out["dw"] = torch.empty_like(weight)
    if out.get("dbias") is None:
        out["dbias"] = torch.empty_like(bias) if bias is not None else None
    if out.get("dxs") is None:
        out["dxs"] = torch.empty_like(state_in) if state_in is not None else None
    a = ConvBwdArgs(_conv_args(x, weight, bias, state_in, None, None, silu), _ptr(grad_y),
                    _ptr(grad_state_out), _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out["dbias"]),
                    _ptr(out["dxs"]))
    _check(load().rdm_shortconv_bwd(ctypes.byref(a), _stream(stream)), "rdm_shortconv_bwd")
    return out


def rdm_shortconv_fwd_many(problems, *, silu=False, stream=None):
    """Several independent ShortConv forwards in one launch.  `problems` is a
    list (at most 4) of dicts with x, weight and optionally bias, state_in, y
    and return_state, as for rdm_shortconv_fwd (same dtype and W in all).
    Returns a list of (y, state_out or None)."""
    outs, args = [], []
    for pr in problems:
        x, weight = pr["x"], pr["weight"]
        B, H, T, D = x.shape
        W = weight.shape[-1]
        y = pr.get("y")
        if y is None:
            y = torch.empty_like(x)
        state_out = (torch.empty(B, H, W - 1, D, dtype=x.dtype, device=x.device)
                     if pr.get("return_state") else None)
        args.append(_conv_args(x, weight, pr.get("bias"), pr.get("state_in"), y, state_out, silu))
        outs.append((y, state_out))
    arr = (ConvArgs * len(args))(*args)
    _check(load().rdm_shortconv_fwd_many(arr, len(args), _stream(stream)), "rdm_shortconv_fwd_many")
    return outs


def rdm_shortconv_bwd_many(problems, *, silu=False, stream=None):
    """Several independent ShortConv backwards in one launch.  `problems` is a
    list (at most 4) of dicts with x, weight, grad_y and optionally bias,
    state_in, grad_state_out and out, as for rdm_shortconv_bwd.  Returns a list
    of dicts dx, dw, dbias, dxs."""
    outs, args = [], []
    for pr in problems:
        x, weight, bias, state_in = pr["x"], pr["weight"], pr.get("bias"), pr.get("state_in")
        out = dict(pr.get("out") or {})
        if out.get("dx") is None:
            out["dx"] = torch.empty_like(x)
        if out.get("dw") is None:
            out["dw"] = torch.empty_like(weight)
        if out.get("dbias") is None:
            out["dbias"] = torch.empty_like(bias) if bias is not None else None
        if out.get("dxs") is None:
            out["dxs"] = torch.empty_like(state_in) if state_in is not None else None
        args.append(ConvBwdArgs(_conv_args(x, weight, bias, state_in, None, None, silu),
                                _ptr(pr["grad_y"]), _ptr(pr.get("grad_state_out")), _ptr(out["dx"]),
                                _ptr(out["dw"]), _ptr(out["dbias"]), _ptr(out["dxs"])))
        outs.append(out)
    arr = (ConvBwdArgs * len(args))(*args)
    _check(load().rdm_shortconv_bwd_many(arr, len(args), _stream(stream)), "rdm_shortconv_bwd_many")
    return outs


def rdm_ska_fwd(q, k, v, window, *, scale=0.0, o=None, k_cache=None, v_cache=None, pos=None,
                stream=None):
    """Sliding-window shared-key attention: q [B,H,T,dk], k [B,T,dk] (one key
    row per token, shared by the heads), v [B,H,T,dv], all bf16; token t
    attends to tokens t-window+1..t.  scale 0 means 1/sqrt(dk).  With k_cache
    [B,window,dk] / v_cache [B,H,window,dv] / pos [B] int32 given, the last
    min(T, window) keys and values are written to slot (position mod window)
    and pos is set to T.  Returns o [B,H,T,dv]."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    a = SkaFwdArgs(B, H, T, dk, dv, int(window), float(scale), _dtype_code(q), _ptr(q), _ptr(k),
                   _ptr(v), _ptr(o), _ptr(k_cache), _ptr(v_cache), _ptr(pos))
    _check(load().rdm_ska_fwd(ctypes.byref(a), _stream(stream)), "rdm_ska_fwd")
    return o


def rdm_ska_decode(q, k, v, k_cache, v_cache, pos, *, scale=0.0, advance_pos=True, o=None,
                   stream=None):
    """One SW-SKA decode step against ring caches: q [B,H,dk], k [B,dk], v
    [B,H,dv] bf16; k_cache [B,window,dk], v_cache [B,H,window,dv] updated in
    place; pos [B] int32 tokens seen before this one (incremented when
    advance_pos).  Returns o [B,H,dv]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    window = k_cache.shape[1]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    a = SkaDecodeArgs(B, H, dk, dv, int(window), float(scale), _dtype_code(q), _ptr(q), _ptr(k),
                      _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos), int(bool(advance_pos)),
                      _ptr(o))
    _check(load().rdm_ska_decode(ctypes.byref(a), _stream(stream)), "rdm_ska_decode")
    return o


# ---------------------------------------------------------------- selective scan
# A call's arguments go into the C struct by one struct.pack (the layouts are
# checked against the ctypes structures when the library is loaded): a single
# token takes a few microseconds on the GPU, less than ctypes spends on thirty
# fields.
_SSM = struct.Struct("@10i18PN")
_SSM_BWD = struct.Struct("@10i18PN15P")
_SSM_STEP = struct.Struct("@9i13P")
_Q8_FILL = struct.Struct("@7i7P2i3P")
_Q8_DECODE = struct.Struct("@7i7Pfi4PiPN")
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_CODES = {_F32: RDM_F32, _BF16: RDM_BF16}
_packed = {}


def _load_packed(name):
    """The library's function `name`, taking its arguments as packed bytes."""
    if not _packed:  # all of them are published at once: another thread may come in meanwhile
        declared = {}
        lib = load()
        for layout, ty in ((_SSM, SsmArgs), (_SSM_BWD, SsmBwdArgs), (_SSM_STEP, SsmStepArgs), (_Q8_FILL, SkaQ8FillArgs),
                           (_Q8_DECODE, SkaQ8DecodeArgs)):
            if layout.size > ctypes.sizeof(ty) or ctypes.sizeof(ty) - layout.size >= 8:
                raise RuntimeError(f"{ty.__name__}: {ctypes.sizeof(ty)} bytes, packed {layout.size}")
        for n in ("rdm_ssm_fwd", "rdm_ssm_bwd", "rdm_ssm_step", "rdm_ska_q8_fill", "rdm_ska_q8_decode",
                  "rdm_ssm_fwd_workspace_size", "rdm_ssm_bwd_workspace_size", "rdm_ska_q8_decode_workspace_size"):
            fn = lib[n]
            size = n.endswith("_size")
            fn.argtypes = [ctypes.c_char_p] if size else [ctypes.c_char_p, _VP]
            fn.restype = ctypes.c_size_t if size else _I
            declared[n] = fn
        _packed.update(declared)
    return _packed[name]


def _size(name, packed) -> int:
    n = _load_packed(name + "_workspace_size")(packed)
    if n == _NO_SIZE:
        raise RdmError(RDM_ERR_INVALID_ARG, name)
    return n


_NO_SIZE = ctypes.c_size_t(-1).value


def _launch(name, packed, dev):
    status = _load_packed(name)(packed, torch._C._cuda_getCurrentRawStream(dev))
    if status != RDM_OK:
        raise RdmError(status, name)


def _on(stream):
    """Context in which `stream` (torch stream or handle) is the current one, so
    that what a call allocates belongs to the stream it runs on."""
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(_stream(stream)))


def _current(t, name) -> int:
    """The device of `t`, which has to be the current one: the library launches there."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors passed to the library must be contiguous CUDA tensors")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _arg(t, name, shape, dtype, dev):
    """The pointer of argument `name` after its checks; None is a null pointer
    (which the library refuses where it needs one)."""
    if t is None:
        return 0
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor") from None
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: tensors passed to the library must be contiguous and on cuda:{dev}")


def _buffer(t, dev):
    """Pointer and bytes of a workspace."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: tensors passed to the library must be contiguous and on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _width(conv_weight, a=None, b=None, c=None):
    """Taps of the convolution, 0 without one (and then none of its bias and states)."""
    if conv_weight is None:
        if a is None and b is None and c is None:
            return 0
    elif conv_weight.dim() != 3:
        raise ValueError("conv_weight: expected [H,D,W]")
    elif conv_weight.shape[2]:
        return conv_weight.shape[2]
    raise ValueError("a convolution's bias or state needs conv_weight [H,D,W] with W >= 1")


def _ssm_args(x, dt, A, Bm, Cm, S0, z, dt_bias, feedthrough, conv_weight, conv_bias, conv_state_in,
              conv_silu, lengths, gates, y, ST, conv_state_out, saved_states):
    """The fields of rdm_ssm_args up to the workspace, and the device."""
    dev = _current(x, "x")
    if x.dim() != 4 or A.dim() != 3 or Bm.dim() != 4:
        raise ValueError("x: expected [B,H,T,D], A: [H,D,N], Bm: [B,G,T,N]")
    B, H, T, D = x.shape
    N, G, ty = A.shape[-1], Bm.shape[1], x.dtype
    W = _width(conv_weight, conv_bias, conv_state_in, conv_state_out)
    seq, group, state, chan, cstate = (B, H, T, D), (B, G, T, N), (B, H, D, N), (H, D), (B, H, W - 1, D)
    return (B, H, G, T, D, N, W, _code(x, "x"), GATES[gates], 1 if conv_silu else 0, _arg(x, "x", seq, ty, dev),
            _arg(dt, "dt", seq, ty, dev), _arg(Bm, "Bm", group, ty, dev), _arg(Cm, "Cm", group, ty, dev),
            _arg(z, "z", seq, ty, dev), _arg(A, "A", (H, D, N), _F32, dev), _arg(dt_bias, "dt_bias", chan, _F32, dev),
            _arg(feedthrough, "feedthrough", chan, _F32, dev), _arg(conv_weight, "conv_weight", (H, D, W), _F32, dev),
            _arg(conv_bias, "conv_bias", chan, _F32, dev), _arg(conv_state_in, "conv_state_in", cstate, ty, dev),
            _arg(S0, "S0", state, _F32, dev), _arg(lengths, "lengths", (B,), _I32, dev), _arg(y, "y", seq, ty, dev),
            _arg(ST, "ST", state, _F32, dev), _arg(conv_state_out, "conv_state_out", cstate, ty, dev),
            _arg(saved_states, "saved_states", (B, H, (T + 15) // 16, D, N), _F32, dev)), dev


def rdm_ssm_saved_states_size(B, H, T, D, N) -> int:
    return int(load().rdm_ssm_saved_states_size(B, H, T, D, N))


def rdm_ssm_saved_states(x, A):
    """A buffer [B,H,ceil(T/16),D,N] for the states that rdm_ssm_fwd saves for
    rdm_ssm_bwd."""
    B, H, T, D = x.shape
    return torch.empty(B, H, (T + 15) // 16, D, A.shape[-1], dtype=_F32, device=x.device)


def rdm_ssm_fwd_workspace_size(x, dt, A, Bm, Cm, *, conv_weight=None, gates="preact") -> int:
    a, _ = _ssm_args(x, dt, A, Bm, Cm, None, None, None, None, conv_weight, None, None, True, None, gates,
                     None, None, None, None)
    return _size("rdm_ssm_fwd", _SSM.pack(*a, 0, 0))


def rdm_ssm_fwd(x, dt, A, Bm, Cm, *, S0=None, z=None, dt_bias=None, feedthrough=None, conv_weight=None,
                conv_bias=None, conv_state_in=None, conv_silu=True, lengths=None, gates="preact", y=None,
                ST=None, conv_state_out=None, saved_states=None, return_state=False, workspace=None,
                stream=None):
    """Selective state space scan over [B,H,T,D] sequences (include/rdm_ddts.h):
    x, dt, z [B,H,T,D] and Bm, Cm [B,G,T,N] in one dtype, A [H,D,N], dt_bias,
    feedthrough [H,D] float32; with conv_weight [H,D,W] (conv_bias [H,D],
    conv_state_in [B,H,W-1,D]) x first goes through the causal convolution and,
    unless conv_silu is False, its SiLU.  lengths [B] int32: tokens of each
    sequence, rows of y behind them are left as they were (a y that is
    allocated here starts with zeros then).  return_state allocates ST and
    conv_state_out; workspace=False runs without one.  Returns (y, ST or None,
    conv_state_out or None)."""
    if stream is not None:
        with _on(stream):
            return rdm_ssm_fwd(x, dt, A, Bm, Cm, S0=S0, z=z, dt_bias=dt_bias, feedthrough=feedthrough,
                               conv_weight=conv_weight, conv_bias=conv_bias, conv_state_in=conv_state_in,
                               conv_silu=conv_silu, lengths=lengths, gates=gates, y=y, ST=ST,
                               conv_state_out=conv_state_out, saved_states=saved_states,
                               return_state=return_state, workspace=workspace)
    if y is None:
        y = torch.empty_like(x) if lengths is None else torch.zeros_like(x)
    if return_state:
        B, H, _, D = x.shape
        if ST is None:
            ST = A.new_empty((B, H, D, A.shape[-1]))
        if conv_state_out is None and conv_weight is not None:
            conv_state_out = x.new_empty((B, H, conv_weight.shape[-1] - 1, D))
    a, dev = _ssm_args(x, dt, A, Bm, Cm, S0, z, dt_bias, feedthrough, conv_weight, conv_bias, conv_state_in,
                       conv_silu, lengths, gates, y, ST, conv_state_out, saved_states)
    packed = _SSM.pack(*a, 0, 0)
    if workspace is None:
        need = _size("rdm_ssm_fwd", packed)
        if need:
            workspace = x.new_empty(need, dtype=torch.uint8)
    if workspace is not None and workspace is not False:
        packed = _SSM.pack(*a, *_buffer(workspace, dev))
    _launch("rdm_ssm_fwd", packed, dev)
    return y, ST, conv_state_out


def _ssm_bwd_args(a, grad_y, grad_ST, grad_conv_state_out, g, ty, dev):
    """The fields of rdm_ssm_bwd_args behind the forward's."""
    B, H, G, T, D, N, W = a[:7]
    seq, state, group, chan, cstate = (B, H, T, D), (B, H, D, N), (B, G, T, N), (H, D), (B, H, W - 1, D)
    return (_arg(grad_y, "grad_y", seq, ty, dev), _arg(grad_ST, "grad_ST", state, _F32, dev),
            _arg(grad_conv_state_out, "grad_conv_state_out", cstate, ty, dev), _arg(g["dx"], "dx", seq, ty, dev),
            _arg(g["ddt"], "ddt", seq, ty, dev), _arg(g["dz"], "dz", seq, ty, dev), _arg(g["dB"], "dB", group, ty, dev),
            _arg(g["dC"], "dC", group, ty, dev), _arg(g["dA"], "dA", (H, D, N), _F32, dev),
            _arg(g["ddt_bias"], "ddt_bias", chan, _F32, dev), _arg(g["dfeed"], "dfeed", chan, _F32, dev),
            _arg(g["dconv_weight"], "dconv_weight", (H, D, W), _F32, dev),
            _arg(g["dconv_bias"], "dconv_bias", chan, _F32, dev), _arg(g["dS0"], "dS0", state, _F32, dev),
            _arg(g["dconv_state_in"], "dconv_state_in", cstate, ty, dev))


def rdm_ssm_bwd_workspace_size(x, dt, A, Bm, Cm, saved_states=None, *, conv_weight=None, gates="preact") -> int:
    a, _ = _ssm_args(x, dt, A, Bm, Cm, None, None, None, None, conv_weight, None, None, True, None, gates,
                     None, None, None, saved_states)
    return _size("rdm_ssm_bwd", _SSM_BWD.pack(*a, 0, 0, *([0] * 15)))


def rdm_ssm_bwd(x, dt, A, Bm, Cm, grad_y, grad_ST=None, grad_conv_state_out=None, *, S0=None, z=None,
                dt_bias=None, feedthrough=None, conv_weight=None, conv_bias=None, conv_state_in=None,
                conv_silu=True, lengths=None, gates="preact", saved_states=None, grads=None, workspace=None,
                stream=None):
    """Reverse mode of rdm_ssm_fwd with the same arguments.  `grads` may hold
    preallocated dx, ddt, dz, dB, dC, dA, ddt_bias, dfeed, dconv_weight,
    dconv_bias, dconv_state_in, dS0; those whose input is given are allocated
    with torch if missing, the others are None.  saved_states: the forward's
    (None runs its recurrence again).  Returns the dict."""
    if stream is not None:
        with _on(stream):
            return rdm_ssm_bwd(x, dt, A, Bm, Cm, grad_y, grad_ST, grad_conv_state_out, S0=S0, z=z, dt_bias=dt_bias,
                               feedthrough=feedthrough, conv_weight=conv_weight, conv_bias=conv_bias,
                               conv_state_in=conv_state_in, conv_silu=conv_silu, lengths=lengths, gates=gates,
                               saved_states=saved_states, grads=grads, workspace=workspace)
    g = dict(grads) if grads else {}
    for n, ref in (("dx", x), ("ddt", dt), ("dz", z), ("dB", Bm), ("dC", Cm), ("dA", A), ("ddt_bias", dt_bias),
                   ("dfeed", feedthrough), ("dconv_weight", conv_weight), ("dconv_bias", conv_bias),
                   ("dconv_state_in", conv_state_in), ("dS0", S0)):
        if g.get(n) is None:
            g[n] = None if ref is None else torch.empty_like(ref)
    a, dev = _ssm_args(x, dt, A, Bm, Cm, S0, z, dt_bias, feedthrough, conv_weight, conv_bias, conv_state_in,
                       conv_silu, lengths, gates, None, None, None, saved_states)
    _width(conv_weight, grad_conv_state_out, g["dconv_weight"], g["dconv_state_in"])
    b = _ssm_bwd_args(a, grad_y, grad_ST, grad_conv_state_out, g, x.dtype, dev)
    if workspace is None:
        need = _size("rdm_ssm_bwd", _SSM_BWD.pack(*a, 0, 0, *b))
        ws = (0, 0)
        if need:
            workspace = x.new_empty(need, dtype=torch.uint8)
    if workspace is not None:
        ws = _buffer(workspace, dev)
    _launch("rdm_ssm_bwd", _SSM_BWD.pack(*a, *ws, *b), dev)
    return g


def rdm_ssm_step(x, dt, A, Bm, Cm, S, *, z=None, dt_bias=None, feedthrough=None, conv_weight=None,
                 conv_bias=None, conv_state=None, conv_silu=True, gates="preact", y=None, stream=None):
    """One token of the selective scan: x, dt, z [B,H,D], Bm, Cm [B,G,N]; S
    [B,H,D,N] float32 and conv_state [B,H,W-1,D] are updated in place.  Returns
    y [B,H,D]."""
    if stream is not None:
        with _on(stream):
            return rdm_ssm_step(x, dt, A, Bm, Cm, S, z=z, dt_bias=dt_bias, feedthrough=feedthrough,
                                conv_weight=conv_weight, conv_bias=conv_bias, conv_state=conv_state,
                                conv_silu=conv_silu, gates=gates, y=y)
    dev = _current(x, "x")
    if x.dim() != 3 or A.dim() != 3 or Bm.dim() != 3:
        raise ValueError("x: expected [B,H,D], A: [H,D,N], Bm: [B,G,N]")
    seq = x.shape
    B, H, D = seq
    N, G, ty, chan = A.shape[-1], Bm.shape[1], x.dtype, (H, D)
    W = _width(conv_weight, conv_bias, conv_state)
    if y is None:
        y = torch.empty_like(x)
    _launch("rdm_ssm_step", _SSM_STEP.pack(
        B, H, G, D, N, W, _code(x, "x"), GATES[gates], 1 if conv_silu else 0, _arg(x, "x", seq, ty, dev),
        _arg(dt, "dt", seq, ty, dev), _arg(Bm, "Bm", (B, G, N), ty, dev), _arg(Cm, "Cm", (B, G, N), ty, dev),
        _arg(z, "z", seq, ty, dev), _arg(A, "A", (H, D, N), _F32, dev), _arg(dt_bias, "dt_bias", chan, _F32, dev),
        _arg(feedthrough, "feedthrough", chan, _F32, dev), _arg(conv_weight, "conv_weight", (H, D, W), _F32, dev),
        _arg(conv_bias, "conv_bias", chan, _F32, dev), _arg(S, "S", (B, H, D, N), _F32, dev),
        _arg(conv_state, "conv_state", (B, H, W - 1, D), ty, dev) if W > 1 else 0, _arg(y, "y", seq, ty, dev)), dev)
    return y


# ---------------------------------------------------------------- SW-SKA, 8-bit cache
_CACHE_TYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}


def rdm_ska_q8_cache(B, H, dk, dv, window, *, block=64, dtype=torch.float8_e4m3fn, device="cuda"):
    """Tensors of an empty 8-bit ring cache, in the order in which
    rdm_ska_q8_fill and rdm_ska_q8_decode take them: k_cache, v_cache (codes,
    torch.float8_e4m3fn or torch.int8), k_scale, v_scale, k_tail, v_tail, pos."""
    if dtype not in _CACHE_TYPES:
        raise TypeError(f"unsupported cache dtype {dtype} (float8_e4m3fn or int8)")
    nb = (window + block - 1) // block
    at = dict(device=device)
    return (torch.zeros(B, window, dk, dtype=torch.uint8, **at).view(dtype),
            torch.zeros(B, H, window, dv, dtype=torch.uint8, **at).view(dtype),
            torch.ones(B, nb, **at), torch.ones(B, H, nb, **at),
            torch.zeros(B, block, dk, dtype=_BF16, **at), torch.zeros(B, H, block, dv, dtype=_BF16, **at),
            torch.zeros(B, dtype=_I32, **at))


def _q8_cache(B, H, dk, dv, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, dev):
    """The fields of rdm_ska_q8_cache."""
    ty = k_cache.dtype
    kind = _CACHE_TYPES.get(ty)
    if kind is None:
        raise TypeError(f"unsupported cache dtype {ty} (float8_e4m3fn or int8)")
    if k_cache.dim() != 3 or k_tail.dim() != 3 or k_tail.shape[1] < 1:
        raise ValueError("k_cache: expected [B,window,dk], k_tail: [B,block,dk]")
    w, R = k_cache.shape[1], k_tail.shape[1]
    nb = (w + R - 1) // R
    return (B, H, dk, dv, w, R, kind, _arg(k_cache, "k_cache", (B, w, dk), ty, dev),
            _arg(v_cache, "v_cache", (B, H, w, dv), ty, dev), _arg(k_scale, "k_scale", (B, nb), _F32, dev),
            _arg(v_scale, "v_scale", (B, H, nb), _F32, dev), _arg(k_tail, "k_tail", (B, R, dk), _BF16, dev),
            _arg(v_tail, "v_tail", (B, H, R, dv), _BF16, dev), _arg(pos, "pos", (B,), _I32, dev))


def rdm_ska_q8_fill(k, v, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, *, lengths=None, stream=None):
    """Fills an 8-bit ring cache (rdm_ska_q8_cache) from a prompt's keys
    [B,T,dk] and values [B,H,T,dv] in bf16, as so many decode steps would, and
    sets pos; lengths [B] int32: tokens of each sequence."""
    if stream is not None:
        with _on(stream):
            return rdm_ska_q8_fill(k, v, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, lengths=lengths)
    dev = _current(k, "k")
    if k.dim() != 3 or v.dim() != 4:
        raise ValueError("k: expected [B,T,dk], v: [B,H,T,dv]")
    B, T, dk = k.shape
    _, H, _, dv = v.shape
    ty = k.dtype
    _launch("rdm_ska_q8_fill", _Q8_FILL.pack(
        *_q8_cache(B, H, dk, dv, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, dev), T, _code(k, "k"),
        _arg(k, "k", (B, T, dk), ty, dev), _arg(v, "v", (B, H, T, dv), ty, dev),
        _arg(lengths, "lengths", (B,), _I32, dev)), dev)


def _q8_decode_args(q, k, v, cache, scale, o, advance_pos):
    """The fields of rdm_ska_q8_decode_args up to the workspace, and the device."""
    dev = _current(q, "q")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q: expected [B,H,dk], v: [B,H,dv]")
    B, H, dk = q.shape
    dv, ty = v.shape[2], q.dtype
    return (*_q8_cache(B, H, dk, dv, *cache, dev), float(scale), _code(q, "q"), _arg(q, "q", (B, H, dk), ty, dev),
            _arg(k, "k", (B, dk), ty, dev), _arg(v, "v", (B, H, dv), ty, dev), _arg(o, "o", (B, H, dv), ty, dev),
            1 if advance_pos else 0), dev


def rdm_ska_q8_decode_workspace_size(q, k, v, *cache) -> int:
    a, _ = _q8_decode_args(q, k, v, cache, 0.0, None, True)
    return _size("rdm_ska_q8_decode", _Q8_DECODE.pack(*a, 0, 0))


def rdm_ska_q8_decode(q, k, v, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, *, scale=0.0,
                      advance_pos=True, o=None, workspace=None, stream=None):
    """One SW-SKA decode step over an 8-bit ring cache (rdm_ska_q8_cache),
    updated in place: q [B,H,dk], k [B,dk], v [B,H,dv] bf16.  scale 0 means
    1/sqrt(dk); workspace=False runs without one.  Returns o [B,H,dv]."""
    if stream is not None:
        with _on(stream):
            return rdm_ska_q8_decode(q, k, v, k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos, scale=scale,
                                     advance_pos=advance_pos, o=o, workspace=workspace)
    if o is None:
        o = torch.empty_like(v)
    a, dev = _q8_decode_args(q, k, v, (k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos), scale, o, advance_pos)
    packed = _Q8_DECODE.pack(*a, 0, 0)
    if workspace is None:
        need = _size("rdm_ska_q8_decode", packed)
        if need:
            workspace = q.new_empty(need, dtype=torch.uint8)
    if workspace is not None and workspace is not False:
        packed = _Q8_DECODE.pack(*a, *_buffer(workspace, dev))
    _launch("rdm_ska_q8_decode", packed, dev)
    return o


def rdm_ddts_sync_status(stream=None) -> int:
    return int(load().rdm_ddts_sync_status(_stream(stream)))


def rdm_status_string(status: int) -> str:
    return status_string(status)


def rdm_ddts_set_test_hooks(wait_limit_cycles: int = 0, withhold_segment_flags: int = 0) -> None:
    """Test hooks of the bounded on-device waits (see include/rdm_ddts.h);
    (0, 0) restores the defaults."""
    _check(load().rdm_ddts_set_test_hooks(int(wait_limit_cycles), int(withhold_segment_flags)),
           "rdm_ddts_set_test_hooks")


def rdm_ddts_version() -> int:
    return int(load().rdm_ddts_version())
