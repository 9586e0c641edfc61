"""Thin Python binding of libssmscan.so: torch tensors in, raw device pointers to the C ABI out.

Argument marshalling only: every step of the scan runs in the library's HIP kernels. torch
provides device memory and the current stream. There is no fallback: if the library is missing
or the tensors are not on a ROCm GPU, the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libssmscan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_OK = 0
STATUS_NAMES = {0: "SSM_OK", 1: "SSM_ERR_NULL", 2: "SSM_ERR_SHAPE", 3: "SSM_ERR_UNSUPPORTED",
                4: "SSM_ERR_HIP", 5: "SSM_ERR_ALIAS", 6: "SSM_ERR_SCRATCH"}
SSM_ERR_SCRATCH = 6
NOALLOC_SCRATCH_BYTES = 32 << 20


class SsmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class FwdOpts(ctypes.Structure):
    """ssm_fwd_opts_t."""
    _fields_ = [("seg_len", ctypes.c_int32), ("lanes_per_channel", ctypes.c_int32),
                ("initial_state", ctypes.c_void_p), ("ev_begin", ctypes.c_void_p),
                ("ev_end", ctypes.c_void_p), ("reserved", ctypes.c_int64 * 4)]


class FwdPlan(ctypes.Structure):
    """ssm_fwd_plan_t."""
    _fields_ = [("seg_len", ctypes.c_int32), ("lanes_per_channel", ctypes.c_int32),
                ("states_per_lane", ctypes.c_int32), ("n_segments", ctypes.c_int32),
                ("waves_per_segment", ctypes.c_int64),
                ("groups_output_pass", ctypes.c_int64), ("groups_aggregate_pass", ctypes.c_int64),
                ("scratch_bytes", ctypes.c_int64)]


class LinAttnStrides(ctypes.Structure):
    """ssm_linattn_strides_t: elements between batch rows, steps and heads of each input."""
    _fields_ = [(f"{t}_{a}", ctypes.c_int64) for t in ("q", "k", "v", "do") for a in ("b", "t", "h")]


class AttnRows(ctypes.Structure):
    """ssm_attn_rows_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu_q", "cu_k", "len_q", "len_k")] + \
               [(n, ctypes.c_int64) for n in ("b", "Lq", "Lk", "tokens_q", "tokens_k")]


class Pages(ctypes.Structure):
    """ssm_pages_t."""
    _fields_ = [("page_table", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("pages", "page_size", "max_pages", "k_page", "v_page")]


class Tokens(ctypes.Structure):
    """ssm_tokens_t."""
    _fields_ = [("cu", ctypes.c_void_p), ("new_lengths", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("b", "L", "T")]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded C library with argument types declared (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                           "(hipcc --offload-arch=gfx950) first")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    fwd = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, vp]
    L.ssm_scan_fwd.argtypes = fwd
    L.ssm_scan_fwd.restype = i32
    L.ssm_scan_fwd_ex.argtypes = fwd + [ctypes.POINTER(FwdOpts)]
    L.ssm_scan_fwd_ex.restype = i32
    L.ssm_scan_fwd_noalloc.argtypes = fwd + [ctypes.POINTER(FwdOpts)]
    L.ssm_scan_fwd_noalloc.restype = i32
    L.ssm_scan_fwd_plan.argtypes = [i64, i64, i64, i64, i32, ctypes.POINTER(FwdOpts), ctypes.POINTER(FwdPlan)]
    L.ssm_scan_fwd_plan.restype = i32
    L.ssm_scan_step.argtypes = [vp] * 9 + [i64, i64, i64, i32, vp]
    L.ssm_scan_step.restype = i32
    L.ssm_scan_bwd.argtypes = [vp] * 18 + [i64, i64, i64, i64, i32, vp]
    L.ssm_scan_bwd.restype = i32
    L.ssm_conv1d_fwd.argtypes = [vp] * 6 + [i64, i64, i64, i64, i32, i32, vp]
    L.ssm_conv1d_fwd.restype = i32
    L.ssm_conv1d_step.argtypes = [vp] * 5 + [i64, i64, i64, i32, i32, vp]
    L.ssm_conv1d_step.restype = i32
    L.ssm_scan_fwd_conv.argtypes = [vp, vp, vp, vp, i64, vp, vp, i32] + [vp] * 10 + [i64, i64, i64, i64, i32, vp]
    L.ssm_scan_fwd_conv.restype = i32
    L.ssm_scan_step_conv.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, i32] + [vp] * 7 + [i64, i64, i64, i32, vp]
    L.ssm_scan_step_conv.restype = i32
    L.ssm_lti_kernel.argtypes = [vp] * 5 + [i64, i64, i64, vp]
    L.ssm_lti_kernel.restype = i32
    L.ssm_lti_conv.argtypes = [vp] * 5 + [i64, i64, i64, i32, vp]
    L.ssm_lti_conv.restype = i32
    L.ssm_lti_fwd.argtypes = [vp] * 8 + [i64, i64, i64, i64, i32, vp]
    L.ssm_lti_fwd.restype = i32
    L.ssm_ssd_fwd.argtypes = [vp] * 10 + [i64, i64, i64, i64, i64, i32, vp]
    L.ssm_ssd_fwd.restype = i32
    f32 = ctypes.c_float
    strides = ctypes.POINTER(LinAttnStrides)
    L.ssm_linattn_workspace.argtypes = [i32] + [i64] * 6 + [i32, i32, ctypes.POINTER(i64)]
    L.ssm_linattn_workspace.restype = i32
    L.ssm_linattn_fwd.argtypes = [vp] * 4 + [i32, f32] + [vp] * 4 + [i64] * 6 + [i32, strides, vp, i64, vp]
    L.ssm_linattn_fwd.restype = i32
    L.ssm_linattn_step.argtypes = [vp] * 5 + [i32, f32, vp] + [i64] * 5 + [i32, strides, vp]
    L.ssm_linattn_step.restype = i32
    L.ssm_linattn_bwd.argtypes = [vp] * 4 + [i32, f32] + [vp] * 9 + [i64] * 6 + [i32, strides, vp, i64, vp]
    L.ssm_linattn_bwd.restype = i32
    L.ssm_layernorm_fwd.argtypes = [vp] * 6 + [i64] * 4 + [f32, i32, vp]
    L.ssm_layernorm_fwd.restype = i32
    L.ssm_layernorm_bwd_workspace.argtypes = [i64] * 3 + [ctypes.POINTER(i64)]
    L.ssm_layernorm_bwd_workspace.restype = i32
    L.ssm_layernorm_bwd.argtypes = [vp] * 8 + [i64] * 5 + [i32, vp, i64, vp]
    L.ssm_layernorm_bwd.restype = i32
    rows, pages, tokens = ctypes.POINTER(AttnRows), ctypes.POINTER(Pages), ctypes.POINTER(Tokens)
    L.ssm_attn_fwd_workspace.argtypes = [rows, i64, i64, i64, i32, ctypes.POINTER(i64)]
    L.ssm_attn_fwd_workspace.restype = i32
    L.ssm_attn_fwd.argtypes = [vp] * 3 + [f32, i32, rows, vp, vp] + [i64] * 3 + [i32, strides, vp, i64, vp]
    L.ssm_attn_fwd.restype = i32
    L.ssm_attn_bwd_workspace.argtypes = [rows, i64, i64, i64, ctypes.POINTER(i64)]
    L.ssm_attn_bwd_workspace.restype = i32
    L.ssm_attn_bwd.argtypes = [vp] * 6 + [f32, i32, rows] + [vp] * 3 + [i64] * 3 + [i32, strides, vp, i64, vp]
    L.ssm_attn_bwd.restype = i32
    L.ssm_attn_step_workspace.argtypes = [i64] * 4 + [pages, i64, ctypes.POINTER(i64)]
    L.ssm_attn_step_workspace.restype = i32
    L.ssm_attn_step.argtypes = [vp] * 3 + [pages, vp, f32, vp, vp] + [i64] * 7 + [i32, vp, i64, vp]
    L.ssm_attn_step.restype = i32
    L.ssm_kv_append.argtypes = [vp] * 7 + [pages, vp, tokens, vp, i64, i32] + [i64] * 3 + [i32, strides, vp]
    L.ssm_kv_append.restype = i32
    L.ssm_rope.argtypes = [vp] * 3 + [tokens, vp, i64, i32, i32] + [i64] * 5 + [i32, vp]
    L.ssm_rope.restype = i32
    L.ssm_status_string.argtypes = [i32]
    L.ssm_status_string.restype = ctypes.c_char_p
    L.ssm_abi_version.argtypes = []
    L.ssm_abi_version.restype = i32
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().ssm_status_string(int(status)).decode()


def _raise(status: int, what: str):
    if status != SSM_OK:
        raise SsmError(status, f"{what}: {status_string(status)}")


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return SSM_F32
    if t == torch.bfloat16:
        return SSM_BF16
    raise TypeError(f"unsupported storage dtype {t}; use float32 or bfloat16")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(name, t, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def ssm_scan_fwd(x, delta, A, B, C, D=None, z=None, *, y=None, final_state=None, return_final_state=True,
                 seg_len=0, lanes_per_channel=0, initial_state=None, events=None, noalloc=False):
    """Prefill scan. x, delta, z: [b, d, L]; A: [d, N] fp32; B, C: [b, L, N]; D: [d] fp32.
    x, delta, z, B, C share one storage dtype (float32 or bfloat16); y gets it too.
    Returns (y, final_state) (final_state is None when return_final_state is False and none is given).
    events: optional (begin, end) torch.cuda.Event pair recorded around the output-pass kernel.
    noalloc: call ssm_scan_fwd_noalloc (scratch in the library's fixed device array; y and final_state
    should then be given, since allocating them here would defeat the purpose)."""
    if x.dim() != 3:
        raise ValueError("x must be [b, d, L]")
    b, d, L = x.shape
    if A.dim() != 2:
        raise ValueError("A must be [d, N]")
    N = A.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    st = x.dtype
    code = _dtype_code(st)
    _check("delta", delta, (b, d, L), st, dev)
    _check("A", A, (d, N), torch.float32, dev)
    _check("B", B, (b, L, N), st, dev)
    _check("C", C, (b, L, N), st, dev)
    _check("D", D, (d,), torch.float32, dev)
    _check("z", z, (b, d, L), st, dev)
    _check("x", x, (b, d, L), st, dev)
    _check("initial_state", initial_state, (b, d, N), torch.float32, dev)
    if y is None:
        y = torch.empty((b, d, L), dtype=st, device=dev)
    _check("y", y, (b, d, L), st, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((b, d, N), dtype=torch.float32, device=dev)
    _check("final_state", final_state, (b, d, N), torch.float32, dev)
    args = [_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(final_state),
            b, d, L, N, code, _stream(dev)]
    if noalloc or seg_len or lanes_per_channel or initial_state is not None or events is not None:
        o = FwdOpts()
        o.seg_len = int(seg_len)
        o.lanes_per_channel = int(lanes_per_channel)
        o.initial_state = None if initial_state is None else initial_state.data_ptr()
        if events is not None:
            o.ev_begin = events[0].cuda_event
            o.ev_end = events[1].cuda_event
        fn = lib().ssm_scan_fwd_noalloc if noalloc else lib().ssm_scan_fwd_ex
        status = fn(*args, ctypes.byref(o))
    else:
        status = lib().ssm_scan_fwd(*args)
    _raise(status, "ssm_scan_fwd_noalloc" if noalloc else "ssm_scan_fwd")
    return y, final_state


def ssm_scan_fwd_conv(xin, conv_w, delta, A, B, C, D=None, z=None, *, conv_bias=None, conv_state_in=None,
                      delta_bias=None, delta_softplus=False, initial_state=None, y=None, final_state=None,
                      conv_state_out=None, x_out=None, return_states=True, want_x=False):
    """The Mamba block's main branch in one prefill pass: Conv1D (conv_w [d, W], W <= 4) + SiLU on xin
    [b, d, L], Δ = delta + delta_bias (softplus when delta_softplus), then the scan. Returns
    (y, final_state, conv_state_out, x_out); the states are allocated when return_states is set and none is
    given, x_out (the convolved input) when want_x is set."""
    if xin.dim() != 3 or conv_w.dim() != 2:
        raise ValueError("xin must be [b, d, L] and conv_w [d, W]")
    b, d, L = xin.shape
    N = A.shape[1]
    W = conv_w.shape[1]
    dev = xin.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    st = xin.dtype
    code = _dtype_code(st)
    f32 = torch.float32
    for name, t, shape, dt in (("delta", delta, (b, d, L), st), ("A", A, (d, N), f32), ("B", B, (b, L, N), st),
                               ("C", C, (b, L, N), st), ("D", D, (d,), f32), ("z", z, (b, d, L), st),
                               ("conv_w", conv_w, (d, W), f32), ("conv_bias", conv_bias, (d,), f32),
                               ("conv_state_in", conv_state_in, (b, d, W - 1), f32),
                               ("delta_bias", delta_bias, (d,), f32), ("initial_state", initial_state, (b, d, N), f32),
                               ("xin", xin, (b, d, L), st)):
        _check(name, t, shape, dt, dev)
    if y is None:
        y = torch.empty((b, d, L), dtype=st, device=dev)
    if return_states and final_state is None:
        final_state = torch.empty((b, d, N), dtype=f32, device=dev)
    if return_states and conv_state_out is None and W > 1:
        conv_state_out = torch.empty((b, d, W - 1), dtype=f32, device=dev)
    if want_x and x_out is None:
        x_out = torch.empty((b, d, L), dtype=st, device=dev)
    _check("y", y, (b, d, L), st, dev)
    _check("final_state", final_state, (b, d, N), f32, dev)
    _check("conv_state_out", conv_state_out, (b, d, W - 1), f32, dev)
    _check("x_out", x_out, (b, d, L), st, dev)
    status = lib().ssm_scan_fwd_conv(_ptr(xin), _ptr(conv_w), _ptr(conv_bias), _ptr(conv_state_in), W, _ptr(delta),
                                     _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                     _ptr(z), _ptr(initial_state), _ptr(y), _ptr(final_state), _ptr(conv_state_out),
                                     _ptr(x_out), b, d, L, N, code, _stream(dev))
    _raise(status, "ssm_scan_fwd_conv")
    return y, final_state, conv_state_out, x_out


def ssm_scan_step_conv(state, conv_state, xin, conv_w, delta, A, B, C, D=None, z=None, *, conv_bias=None,
                       delta_bias=None, delta_softplus=False, y=None, x_out=None):
    """One decode step of the Mamba block's main branch: state [b, d, N] and conv_state [b, d, W-1] (fp32,
    both updated in place); xin, delta, z [b, d]; conv_w [d, W]. Returns (y, x_out) (x_out None unless
    given)."""
    b, d, N = state.shape
    W = conv_w.shape[1]
    dev = state.device
    st = xin.dtype
    code = _dtype_code(st)
    f32 = torch.float32
    for name, t, shape, dt in (("state", state, (b, d, N), f32), ("conv_state", conv_state, (b, d, W - 1), f32),
                               ("xin", xin, (b, d), st), ("delta", delta, (b, d), st), ("A", A, (d, N), f32),
                               ("B", B, (b, N), st), ("C", C, (b, N), st), ("D", D, (d,), f32), ("z", z, (b, d), st),
                               ("conv_w", conv_w, (d, W), f32), ("conv_bias", conv_bias, (d,), f32),
                               ("delta_bias", delta_bias, (d,), f32)):
        _check(name, t, shape, dt, dev)
    if y is None:
        y = torch.empty((b, d), dtype=st, device=dev)
    _check("y", y, (b, d), st, dev)
    _check("x_out", x_out, (b, d), st, dev)
    status = lib().ssm_scan_step_conv(_ptr(state), _ptr(conv_state) if W > 1 else None, _ptr(xin), _ptr(conv_w),
                                      _ptr(conv_bias), W, _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                                      _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(x_out), b, d, N, code,
                                      _stream(dev))
    _raise(status, "ssm_scan_step_conv")
    return y, x_out


def ssm_scan_step(state, x, delta, A, B, C, D=None, z=None, *, y=None):
    """Decode step: state [b, d, N] fp32 (updated in place); x, delta, z [b, d]; B, C [b, N];
    A [d, N] fp32; D [d] fp32. Returns y [b, d]."""
    if state.dim() != 3:
        raise ValueError("state must be [b, d, N]")
    b, d, N = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    st = x.dtype
    code = _dtype_code(st)
    _check("state", state, (b, d, N), torch.float32, dev)
    _check("x", x, (b, d), st, dev)
    _check("delta", delta, (b, d), st, dev)
    _check("A", A, (d, N), torch.float32, dev)
    _check("B", B, (b, N), st, dev)
    _check("C", C, (b, N), st, dev)
    _check("D", D, (d,), torch.float32, dev)
    _check("z", z, (b, d), st, dev)
    if y is None:
        y = torch.empty((b, d), dtype=st, device=dev)
    _check("y", y, (b, d), st, dev)
    status = lib().ssm_scan_step(_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                 _ptr(y), b, d, N, code, _stream(dev))
    _raise(status, "ssm_scan_step")
    return y


def ssm_scan_bwd(x, delta, A, B, C, D=None, z=None, *, dy, initial_state=None, d_final_state=None,
                 want_dD=True, want_d_initial_state=True) -> dict:
    """Gradients of ssm_scan_fwd for an upstream gradient dy [b, d, L] (and optionally d_final_state
    [b, d, N]). Returns a dict: dx, ddelta, dz ([b, d, L], storage dtype; dz None without z),
    dA [d, N], dB, dC [b, L, N], dD [d] (None unless want_dD), d_initial_state [b, d, N] (None unless
    want_d_initial_state), all fp32 except the first three."""
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [b, d, L] and A [d, N]")
    b, d, L = x.shape
    N = A.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    st = x.dtype
    code = _dtype_code(st)
    for name, t, shape, dt in (("delta", delta, (b, d, L), st), ("A", A, (d, N), torch.float32),
                               ("B", B, (b, L, N), st), ("C", C, (b, L, N), st), ("D", D, (d,), torch.float32),
                               ("z", z, (b, d, L), st), ("dy", dy, (b, d, L), st),
                               ("initial_state", initial_state, (b, d, N), torch.float32),
                               ("d_final_state", d_final_state, (b, d, N), torch.float32)):
        _check(name, t, shape, dt, dev)
    f32 = torch.float32
    out = {"dx": torch.empty((b, d, L), dtype=st, device=dev), "ddelta": torch.empty((b, d, L), dtype=st, device=dev),
           "dz": None if z is None else torch.empty((b, d, L), dtype=st, device=dev),
           "dA": torch.empty((d, N), dtype=f32, device=dev), "dB": torch.empty((b, L, N), dtype=f32, device=dev),
           "dC": torch.empty((b, L, N), dtype=f32, device=dev),
           "dD": torch.empty((d,), dtype=f32, device=dev) if want_dD else None,
           "d_initial_state": torch.empty((b, d, N), dtype=f32, device=dev) if want_d_initial_state else None}
    status = lib().ssm_scan_bwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                _ptr(initial_state), _ptr(dy), _ptr(d_final_state), _ptr(out["dx"]),
                                _ptr(out["ddelta"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                                _ptr(out["dD"]), _ptr(out["dz"]), _ptr(out["d_initial_state"]), b, d, L, N, code,
                                _stream(dev))
    _raise(status, "ssm_scan_bwd")
    return out


def ssm_conv1d_fwd(xin, w, bias=None, *, state_in=None, x_out=None, state_out=None, return_state=True,
                   silu=True):
    """Causal depthwise Conv1D (+ SiLU): xin [b, d, L] (float32 or bfloat16), w [d, W] fp32, bias [d] fp32.
    Returns (x [b, d, L] in xin's dtype, state [b, d, W-1] fp32 or None)."""
    if xin.dim() != 3 or w.dim() != 2:
        raise ValueError("xin must be [b, d, L] and w [d, W]")
    b, d, L = xin.shape
    W = w.shape[1]
    dev = xin.device
    st = xin.dtype
    code = _dtype_code(st)
    _check("xin", xin, (b, d, L), st, dev)
    _check("w", w, (d, W), torch.float32, dev)
    _check("bias", bias, (d,), torch.float32, dev)
    _check("state_in", state_in, (b, d, W - 1), torch.float32, dev)
    if x_out is None:
        x_out = torch.empty((b, d, L), dtype=st, device=dev)
    _check("x_out", x_out, (b, d, L), st, dev)
    if state_out is None and return_state and W > 1:
        state_out = torch.empty((b, d, W - 1), dtype=torch.float32, device=dev)
    _check("state_out", state_out, (b, d, W - 1), torch.float32, dev)
    status = lib().ssm_conv1d_fwd(_ptr(xin), _ptr(w), _ptr(bias), _ptr(state_in), _ptr(x_out), _ptr(state_out),
                                  b, d, L, W, int(bool(silu)), code, _stream(dev))
    _raise(status, "ssm_conv1d_fwd")
    return x_out, state_out


def ssm_lti_kernel(delta, A, B, C, L, *, K=None):
    """K̄ [d, L] fp32 of the time-invariant system per channel: delta [d], A, B, C [d, N], all fp32."""
    if A.dim() != 2:
        raise ValueError("A must be [d, N]")
    d, N = A.shape
    dev = A.device
    for name, t, shape in (("delta", delta, (d,)), ("A", A, (d, N)), ("B", B, (d, N)), ("C", C, (d, N))):
        _check(name, t, shape, torch.float32, dev)
    if K is None:
        K = torch.empty((d, int(L)), dtype=torch.float32, device=dev)
    _check("K", K, (d, int(L)), torch.float32, dev)
    status = lib().ssm_lti_kernel(_ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(K), d, int(L), N, _stream(dev))
    _raise(status, "ssm_lti_kernel")
    return K


def ssm_lti_conv(x, K, D=None, z=None, *, y=None):
    """y = x ∗ K̄ + D·x (· silu(z)) by FFT: x, z [b, d, L] (float32 or bfloat16), K [d, L] fp32, D [d] fp32."""
    if x.dim() != 3:
        raise ValueError("x must be [b, d, L]")
    b, d, L = x.shape
    dev, st = x.device, x.dtype
    code = _dtype_code(st)
    _check("K", K, (d, L), torch.float32, dev)
    _check("D", D, (d,), torch.float32, dev)
    _check("z", z, (b, d, L), st, dev)
    if y is None:
        y = torch.empty((b, d, L), dtype=st, device=dev)
    _check("y", y, (b, d, L), st, dev)
    status = lib().ssm_lti_conv(_ptr(x), _ptr(K), _ptr(D), _ptr(z), _ptr(y), b, d, L, code, _stream(dev))
    _raise(status, "ssm_lti_conv")
    return y


def ssm_lti_fwd(x, delta, A, B, C, D=None, z=None, *, y=None):
    """The LTI scan as a convolution in one call: K̄ from (delta [d], A, B, C [d, N]), then ssm_lti_conv."""
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [b, d, L] and A [d, N]")
    b, d, L = x.shape
    N = A.shape[1]
    dev, st = x.device, x.dtype
    code = _dtype_code(st)
    for name, t, shape in (("delta", delta, (d,)), ("A", A, (d, N)), ("B", B, (d, N)), ("C", C, (d, N)),
                           ("D", D, (d,))):
        _check(name, t, shape, torch.float32, dev)
    _check("z", z, (b, d, L), st, dev)
    if y is None:
        y = torch.empty((b, d, L), dtype=st, device=dev)
    _check("y", y, (b, d, L), st, dev)
    status = lib().ssm_lti_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y),
                               b, d, L, N, code, _stream(dev))
    _raise(status, "ssm_lti_fwd")
    return y


def ssm_ssd_fwd(x, delta, A, B, C, D=None, z=None, *, y=None, initial_state=None, final_state=None,
                return_final_state=True):
    """Scalar-decay (state space duality) form, chunked on the MFMA units. x, z: [b, H*P, L] with P = 64;
    delta: [b, H, L]; A: [H] fp32 (one decay per head); B, C: [b, L, N] with N in {32, 64, 128};
    D: [H*P] fp32. Returns (y, final_state [b, H*P, N] fp32 or None)."""
    if x.dim() != 3 or delta.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [b, H*P, L], delta [b, H, L], B and C [b, L, N]")
    b, d, L = x.shape
    H = delta.shape[1]
    if d % H:
        raise ValueError("the channels must split evenly into heads")
    P, N = d // H, B.shape[2]
    dev, st = x.device, x.dtype
    code = _dtype_code(st)
    _check("delta", delta, (b, H, L), st, dev)
    _check("A", A, (H,), torch.float32, dev)
    _check("B", B, (b, L, N), st, dev)
    _check("C", C, (b, L, N), st, dev)
    _check("D", D, (d,), torch.float32, dev)
    _check("z", z, (b, d, L), st, dev)
    _check("initial_state", initial_state, (b, d, N), torch.float32, dev)
    if y is None:
        y = torch.empty((b, d, L), dtype=st, device=dev)
    _check("y", y, (b, d, L), st, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((b, d, N), dtype=torch.float32, device=dev)
    _check("final_state", final_state, (b, d, N), torch.float32, dev)
    status = lib().ssm_ssd_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                               _ptr(initial_state), _ptr(y), _ptr(final_state), b, H, P, L, N, code, _stream(dev))
    _raise(status, "ssm_ssd_fwd")
    return y, final_state


def ssm_conv1d_step(state, xin, w, bias=None, *, x_out=None, silu=True):
    """Decode step of the Conv1D: state [b, d, W-1] fp32 (shifted in place), xin [b, d]. Returns x [b, d]."""
    b, d = xin.shape
    W = w.shape[1]
    dev = xin.device
    st = xin.dtype
    code = _dtype_code(st)
    _check("state", state, (b, d, W - 1), torch.float32, dev)
    _check("w", w, (d, W), torch.float32, dev)
    _check("bias", bias, (d,), torch.float32, dev)
    if x_out is None:
        x_out = torch.empty((b, d), dtype=st, device=dev)
    _check("x_out", x_out, (b, d), st, dev)
    status = lib().ssm_conv1d_step(_ptr(state), _ptr(xin), _ptr(w), _ptr(bias), _ptr(x_out), b, d, W,
                                   int(bool(silu)), code, _stream(dev))
    _raise(status, "ssm_conv1d_step")
    return x_out


def ssm_scan_fwd_plan(b, d, L, N, dtype=torch.float32, seg_len=0, lanes_per_channel=0) -> dict:
    """The launch plan ssm_scan_fwd would use (host only)."""
    o = FwdOpts()
    o.seg_len = int(seg_len)
    o.lanes_per_channel = int(lanes_per_channel)
    p = FwdPlan()
    status = lib().ssm_scan_fwd_plan(b, d, L, N, _dtype_code(dtype), ctypes.byref(o), ctypes.byref(p))
    _raise(status, "ssm_scan_fwd_plan")
    return {k: getattr(p, k) for k, _ in FwdPlan._fields_}


def _check_rows(name, t, shape, dtype, device):
    """As _check, but only the last axis has to be dense (a slice of a packed projection, a broadcast view)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")


def _linattn_inputs(q, k, v, g, lead):
    """Checks the inputs that the prompt, step and gradient calls share; lead: (b, L) or (b,).
    Returns (H, G, N, P, storage dtype code, whether g is per step)."""
    G, N = q.shape[-2:]
    H, P = v.shape[-2:]
    dev, st = v.device, v.dtype
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    code = _dtype_code(st)
    _check_rows("q", q, (*lead, G, N), st, dev)
    _check_rows("k", k, (*lead, G, N), st, dev)
    _check_rows("v", v, (*lead, H, P), st, dev)
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch.Tensor")
    per_step = g.dim() != 1
    _check("g", g, (*lead, H) if per_step else (H,), torch.float32, dev)
    return H, G, N, P, code, per_step


def _linattn_strides(q, k, v, do=None):
    """The strides of [b, L, heads, width] (or [b, heads, width]) inputs, or None when all are dense."""
    if all(t is None or t.is_contiguous() for t in (q, k, v, do)):
        return None
    s = LinAttnStrides()
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        if t is not None:
            st = t.stride()
            setattr(s, f"{name}_b", st[0])
            setattr(s, f"{name}_t", st[1] if len(st) == 4 else 0)
            setattr(s, f"{name}_h", st[-2])
    return ctypes.byref(s)


def _workspace(bytes_, device):
    """Scratch of a call from torch's allocator on the current stream, so that a call captured into a graph keeps it
    for the graph's life."""
    return torch.empty(bytes_, dtype=torch.uint8, device=device) if bytes_ else None


def _on_device(device):
    """Makes `device` current for the launches of a call (nothing to do where it is)."""
    return _HERE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


_HERE = contextlib.nullcontext()


def _raw_stream(device) -> int:
    """The current stream's handle, without a Stream object."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _linattn_bytes(gradient, b, L, H, G, N, P, code, per_step) -> int:
    n = ctypes.c_int64()
    status = lib().ssm_linattn_workspace(gradient, b, L, H, G, N, P, code, per_step, ctypes.byref(n))
    _raise(status, "ssm_linattn_workspace")
    return n.value


def _layernorm_bytes(rows, d, w_rows) -> int:
    n = ctypes.c_int64()
    status = lib().ssm_layernorm_bwd_workspace(rows, d, w_rows, ctypes.byref(n))
    _raise(status, "ssm_layernorm_bwd_workspace")
    return n.value


def ssm_linattn_workspace(b, L, H, G, N, P, dtype=torch.float32, *, gradient=False, g_per_step=True) -> int:
    """Workspace bytes of ssm_linattn_fwd (or ssm_linattn_bwd) for this shape (host only)."""
    return _linattn_bytes(int(bool(gradient)), b, L, H, G, N, P, _dtype_code(dtype), int(bool(g_per_step)))


def ssm_linattn_fwd(q, k, v, g, *, scale=1.0, initial_state=None, lengths=None, o=None, final_state=None,
                    return_final_state=True):
    """Linear attention with a per-head decay over a prompt: S_t = e^{g_t} S_{t-1} + v_t k_tᵀ, o_t = scale·S_t q_t.
    q, k: [b, L, G, N] and v: [b, L, H, P] (float32 or bfloat16, G divides H, N <= 128; views whose last axis is
    contiguous, such as slices of a packed projection, are read in place); g: log-decay, float32, [b, L, H], or
    [H] for the same decay at every step; initial_state: [b, H, P, N] float32; lengths: [b] int32 on the GPU, the
    steps of each row of a padded batch (o is 0 past them). Returns (o [b, L, H, P], final_state [b, H, P, N] or
    None)."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k must be [b, L, G, N] and v [b, L, H, P]")
    b, L = v.shape[:2]
    H, G, N, P, code, per_step = _linattn_inputs(q, k, v, g, (b, L))
    dev = v.device
    _check("initial_state", initial_state, (b, H, P, N), torch.float32, dev)
    _check("lengths", lengths, (b,), torch.int32, dev)
    with _on_device(dev):
        if o is None:
            o = torch.empty((b, L, H, P), dtype=v.dtype, device=dev)
        else:
            _check("o", o, (b, L, H, P), v.dtype, dev)
        if final_state is not None:
            _check("final_state", final_state, (b, H, P, N), torch.float32, dev)
        elif return_final_state:
            final_state = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
        need = _linattn_bytes(0, b, L, H, G, N, P, code, per_step)
        ws = _workspace(need, dev)
        status = lib().ssm_linattn_fwd(_at(q), _at(k), _at(v), _at(g), per_step, float(scale), _at(initial_state),
                                       _at(lengths), _at(o), _at(final_state), b, L, H, G, N, P, code,
                                       _linattn_strides(q, k, v), _at(ws), need, _raw_stream(dev))
    _raise(status, "ssm_linattn_fwd")
    return o, final_state


def ssm_linattn_step(state, q, k, v, g, *, scale=1.0, o=None):
    """One token of ssm_linattn_fwd's recurrence: state [b, H, P, N] float32 (updated in place); q, k: [b, G, N];
    v: [b, H, P]; g: [b, H] or [H] float32. Returns o [b, H, P]."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k must be [b, G, N] and v [b, H, P]")
    b = v.shape[0]
    H, G, N, P, code, per_step = _linattn_inputs(q, k, v, g, (b,))
    dev = v.device
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    _check("state", state, (b, H, P, N), torch.float32, dev)
    with _on_device(dev):
        if o is None:
            o = torch.empty((b, H, P), dtype=v.dtype, device=dev)
        else:
            _check("o", o, (b, H, P), v.dtype, dev)
        status = lib().ssm_linattn_step(_at(state), _at(q), _at(k), _at(v), _at(g), per_step, float(scale), _at(o),
                                        b, H, G, N, P, code, _linattn_strides(q, k, v), _raw_stream(dev))
    _raise(status, "ssm_linattn_step")
    return o


def ssm_linattn_bwd(q, k, v, g, *, do, scale=1.0, initial_state=None, d_final_state=None, lengths=None,
                    want_d_initial_state=True) -> dict:
    """Gradients of ssm_linattn_fwd for an upstream gradient do [b, L, H, P] (and optionally d_final_state
    [b, H, P, N]). Returns a dict: dq, dk [b, L, G, N], dv [b, L, H, P] (storage dtype), dg (g's shape, float32),
    d_initial_state [b, H, P, N] float32 (None unless want_d_initial_state)."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k must be [b, L, G, N] and v [b, L, H, P]")
    b, L = v.shape[:2]
    H, G, N, P, code, per_step = _linattn_inputs(q, k, v, g, (b, L))
    dev, st, f32 = v.device, v.dtype, torch.float32
    _check_rows("do", do, (b, L, H, P), st, dev)
    _check("initial_state", initial_state, (b, H, P, N), f32, dev)
    _check("d_final_state", d_final_state, (b, H, P, N), f32, dev)
    _check("lengths", lengths, (b,), torch.int32, dev)
    with _on_device(dev):
        out = {"dq": torch.empty((b, L, G, N), dtype=st, device=dev), "dk": torch.empty((b, L, G, N), dtype=st, device=dev),
               "dv": torch.empty((b, L, H, P), dtype=st, device=dev), "dg": torch.empty(g.shape, dtype=f32, device=dev),
               "d_initial_state": torch.empty((b, H, P, N), dtype=f32, device=dev) if want_d_initial_state else None}
        need = _linattn_bytes(1, b, L, H, G, N, P, code, per_step)
        ws = _workspace(need, dev)
        status = lib().ssm_linattn_bwd(_at(q), _at(k), _at(v), _at(g), per_step, float(scale), _at(initial_state),
                                       _at(lengths), _at(do), _at(d_final_state), _at(out["dq"]), _at(out["dk"]),
                                       _at(out["dv"]), _at(out["dg"]), _at(out["d_initial_state"]), b, L, H, G, N, P,
                                       code, _linattn_strides(q, k, v, do), _at(ws), need, _raw_stream(dev))
    _raise(status, "ssm_linattn_bwd")
    return out


def _norm_rows(name, x):
    """(rows, elements between them) of a tensor [..., d] whose rows are evenly spaced."""
    if x.is_contiguous():
        return x.numel() // x.shape[-1], x.shape[-1]
    if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= x.shape[1]:
        return x.shape[0], x.stride(0)
    raise ValueError(f"{name} must be contiguous, or [rows, d] with contiguous rows")


def _norm_weight_rows(x, *weights):
    """Weight rows of a norm over x [..., K, d]: K for weights [K, d], 1 for weights [d]; all weights alike."""
    d = x.shape[-1]
    given = [w for w in weights if w is not None]
    k = x.shape[-2] if given and given[0].dim() == 2 and x.dim() > 1 else 1
    for w in given:
        _check("weight or bias", w, (k, d) if given[0].dim() == 2 else (d,), torch.float32, x.device)
    return k


def ssm_layernorm_fwd(x, w=None, bias=None, *, eps=1e-5, y=None, return_stats=False):
    """Layer norm over the last axis: x [..., d] (float32 or bfloat16, d <= 16384), contiguous, or [rows, d] with
    contiguous rows (columns of a wider buffer; flatten the leading axes of one first); w, bias: [d] float32, or
    [K, d] with a row per head for x [..., K, d]. Returns y, or (y, mean, rstd) with mean and rstd float32 of x's
    shape without its last axis when return_stats is set. y may be x itself."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., d] with d >= 1")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    code = _dtype_code(x.dtype)
    rows, stride = _norm_rows("x", x)
    k = _norm_weight_rows(x, w, bias)
    with _on_device(dev):
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        else:
            _check("y", y, x.shape, x.dtype, dev)
        mean = rstd = None
        if return_stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
        status = lib().ssm_layernorm_fwd(_at(x), _at(w), _at(bias), _at(y), _at(mean), _at(rstd), rows,
                                         x.shape[-1], k, stride, float(eps), code, _raw_stream(dev))
    _raise(status, "ssm_layernorm_fwd")
    return (y, mean, rstd) if return_stats else y


def ssm_layernorm_bwd(x, w=None, *, dy, mean, rstd, want_dw=True, want_dbias=True, w_rows=None) -> dict:
    """Gradients of ssm_layernorm_fwd for an upstream gradient dy, from the forward call's mean and rstd. Returns a
    dict: dx (x's shape and dtype), dw, dbias (float32; w's shape, or without w [d], or [w_rows, d] for w_rows;
    None unless wanted)."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., d] with d >= 1")
    dev, d = x.device, x.shape[-1]
    if dev.type != "cuda":
        raise ValueError("tensors must live on a ROCm GPU")
    code = _dtype_code(x.dtype)
    rows, stride = _norm_rows("x", x)
    _check_rows("dy", dy, x.shape, x.dtype, dev)
    dy_stride = _norm_rows("dy", dy)[1]
    k = _norm_weight_rows(x, w)
    shape = tuple(w.shape) if w is not None else (d,)
    if w is None and w_rows is not None:
        if x.dim() < 2 or x.shape[-2] != w_rows:
            raise ValueError("w_rows must be the length of x's axis before the last")
        k, shape = w_rows, (w_rows, d)
    _check("mean", mean, x.shape[:-1], torch.float32, dev)
    _check("rstd", rstd, x.shape[:-1], torch.float32, dev)
    with _on_device(dev):
        out = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev),
               "dw": torch.empty(shape, dtype=torch.float32, device=dev) if want_dw else None,
               "dbias": torch.empty(shape, dtype=torch.float32, device=dev) if want_dbias else None}
        need = _layernorm_bytes(rows, d, k) if want_dw or want_dbias else 0
        ws = _workspace(need, dev)
        status = lib().ssm_layernorm_bwd(_at(x), _at(w), _at(dy), _at(mean), _at(rstd), _at(out["dx"]),
                                         _at(out["dw"]), _at(out["dbias"]), rows, d, k, stride, dy_stride, code,
                                         _at(ws), need, _raw_stream(dev))
    _raise(status, "ssm_layernorm_bwd")
    return out


def _on_gpu(t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on a ROCm GPU")


def _alike(*tensors):
    """Whether all are contiguous tensors of one type on one device: nothing else is left to check but shapes."""
    a = tensors[0]
    dtype, device = a.dtype, a.device
    return all(isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_contiguous() and t.device == device
               for t in tensors)


@functools.lru_cache(maxsize=1024)
def _attn_bytes(gradient, packed, b, Lq, Lk, tokens_q, tokens_k, H, G, D, code) -> int:
    """Workspace bytes of ssm_attn_fwd or ssm_attn_bwd, which go by sizes alone."""
    one = 16 if packed else None  # any address: only whether there is one matters here
    r, n = AttnRows(one, one, None, None, b, Lq, Lk, tokens_q, tokens_k), ctypes.c_int64()
    if gradient:
        _raise(lib().ssm_attn_bwd_workspace(ctypes.byref(r), H, G, D, ctypes.byref(n)), "ssm_attn_bwd_workspace")
    else:
        _raise(lib().ssm_attn_fwd_workspace(ctypes.byref(r), H, G, D, code, ctypes.byref(n)), "ssm_attn_fwd_workspace")
    return n.value


@functools.lru_cache(maxsize=1024)
def _step_bytes(b, H, G, D, pages, page_size, max_pages, k_page, v_page, max_len) -> int:
    """Workspace bytes of ssm_attn_step, which go by sizes alone."""
    g, n = Pages(None, pages, page_size, max_pages, k_page, v_page), ctypes.c_int64()
    _raise(lib().ssm_attn_step_workspace(b, H, G, D, ctypes.byref(g), max_len, ctypes.byref(n)), "ssm_attn_step_workspace")
    return n.value


def _attn_rows(q, k, cu_seqlens, max_len, cu_seqlens_k, max_len_k, lengths, lengths_k):
    """Where the sequences of q and k lie: the descriptor of a packed batch [T, heads, D] or of rows [b, L, heads, D]."""
    dev = q.device
    if q.dim() == 4 and k.dim() == 4:
        if cu_seqlens is not None or cu_seqlens_k is not None or max_len is not None or max_len_k is not None:
            raise ValueError("cu_seqlens and max_len are for packed sequences [T, heads, D]")
        b, Lq = q.shape[:2]
        Lk = k.shape[1]
        if lengths is not None and lengths_k is None:
            if Lk != Lq:
                raise ValueError("lengths of queries and keys: give lengths_k as well where there are more keys than queries")
            lengths_k = lengths
        _check("lengths", lengths, (b,), torch.int32, dev)
        _check("lengths_k", lengths_k, (b,), torch.int32, dev)
        return AttnRows(None, None, _at(lengths), _at(lengths_k), b, Lq, Lk, 0, 0)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [b, L, heads, D], or [T, heads, D] with cu_seqlens")
    if cu_seqlens is None or max_len is None:
        raise ValueError("packed sequences [T, heads, D] need cu_seqlens and max_len")
    if lengths is not None or lengths_k is not None:
        raise ValueError("lengths are for rows [b, L, heads, D]")
    if (cu_seqlens_k is None) != (max_len_k is None):
        raise ValueError("cu_seqlens_k and max_len_k go together")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be a torch.Tensor [b + 1]")
    b = cu_seqlens.shape[0] - 1
    _check("cu_seqlens", cu_seqlens, (b + 1,), torch.int32, dev)
    _check("cu_seqlens_k", cu_seqlens_k, (b + 1,), torch.int32, dev)
    cu_q = cu_seqlens.data_ptr()
    cu_k = cu_q if cu_seqlens_k is None else cu_seqlens_k.data_ptr()
    return AttnRows(cu_q, cu_k, None, None, b, max_len, max_len if max_len_k is None else max_len_k, q.shape[0], k.shape[0])


def _attn_inputs(q, k, v):
    """Checks q [..., H, D], k and v [..., G, D]. Returns (H, G, D, storage dtype code, whether all are dense)."""
    _on_gpu(q)
    if q.dim() < 2 or not isinstance(k, torch.Tensor) or k.dim() != q.dim():
        raise ValueError("q and k must have the same number of axes")
    H, D = q.shape[-2:]
    G = k.shape[-2]
    code = _dtype_code(q.dtype)
    dense = _alike(q, k, v)
    if dense and v.shape == k.shape and k.shape[-1] == D and (q.dim() == 3 or k.shape[0] == q.shape[0]):
        return H, G, D, code, True
    dev, st = q.device, q.dtype
    _check_rows("q", q, q.shape, st, dev)
    _check_rows("k", k, (q.shape[0], *k.shape[1:-1], D) if q.dim() == 4 else (k.shape[0], G, D), st, dev)
    _check_rows("v", v, k.shape, st, dev)
    return H, G, D, code, dense


def _attn_strides(q, k, v, do=None):
    """As _linattn_strides, for [b, L, heads, D] or [T, heads, D] of which not all are dense."""
    s = LinAttnStrides()
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        if t is not None:
            st = t.stride()
            setattr(s, f"{name}_b", st[0] if len(st) == 4 else 0)
            setattr(s, f"{name}_t", st[-3])
            setattr(s, f"{name}_h", st[-2])
    return ctypes.byref(s)


def _scale(scale, D):
    return D ** -0.5 if scale is None else float(scale)


def ssm_attn_fwd(q, k, v, *, scale=None, causal=True, cu_seqlens=None, max_len=None, cu_seqlens_k=None, max_len_k=None,
                 lengths=None, lengths_k=None, o=None, return_lse=False):
    """Softmax attention over prompts: o_i = Σ_j p_ij v_j, p = softmax_j(scale·q_i·k_j) over the keys j <= i + nk − nq of
    its sequence (causal; nq queries, nk keys) or over all of them. Head h of q reads head h·G/H of k and v; scale is
    D^-1/2 unless given. float32 or bfloat16, G divides H, D <= 128; views whose last axis is contiguous (slices of a packed
    projection) are read in place.

    Rows: q [b, L, H, D], k and v [b, Lk, G, D]; lengths and lengths_k ([b] int32 on the GPU) say how many steps of each row
    count (lengths alone: of both); outputs past them are 0. Packed: q [T, H, D], k and v [Tk, G, D] with cu_seqlens
    ([b + 1] int32 on the GPU, rising offsets) and max_len, the longest sequence's length or more (a longer one is cut);
    cu_seqlens_k and max_len_k where the keys' differ. Tokens of no sequence: 0, or as they were in an `o` that is given.

    Returns o (q's shape), or (o, lse) with lse = log Σ_j e^(scale·q_i·k_j) float32 [..., H] when return_lse is set. A query
    that sees no key has o = 0 and lse = −inf."""
    H, G, D, code, dense = _attn_inputs(q, k, v)
    r = _attn_rows(q, k, cu_seqlens, max_len, cu_seqlens_k, max_len_k, lengths, lengths_k)
    dev, packed = q.device, q.dim() == 3
    with _on_device(dev):
        lse = None
        if return_lse:
            lse = torch.full(q.shape[:-1], float("-inf"), dtype=torch.float32, device=dev) if packed else \
                torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
        if o is None:
            o = torch.zeros(q.shape, dtype=q.dtype, device=dev) if packed else torch.empty(q.shape, dtype=q.dtype, device=dev)
        else:
            _check("o", o, q.shape, q.dtype, dev)
        need = _attn_bytes(False, packed, r.b, r.Lq, r.Lk, r.tokens_q, r.tokens_k, H, G, D, code)
        ws = _workspace(need, dev)
        status = lib().ssm_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _scale(scale, D), bool(causal), ctypes.byref(r),
                                    o.data_ptr(), _at(lse), H, G, D, code, None if dense else _attn_strides(q, k, v), _at(ws),
                                    need, _raw_stream(dev))
    _raise(status, "ssm_attn_fwd")
    return (o, lse) if return_lse else o


def ssm_attn_bwd(q, k, v, *, o, lse, do, scale=None, causal=True, cu_seqlens=None, max_len=None, cu_seqlens_k=None,
                 max_len_k=None, lengths=None, lengths_k=None) -> dict:
    """Gradients of ssm_attn_fwd for an upstream gradient do on o, from the forward call's o and lse (contiguous; the other
    arguments as in that call). Returns a dict: dq, dk, dv (the shapes and dtype of q, k, v; dk and dv summed over the heads
    that share a key head). o and lse may be those of more keys than are given here (keys in shards): dk and dv are then those
    of the given keys, and dq is the sum over the calls."""
    H, G, D, code, dense = _attn_inputs(q, k, v)
    r = _attn_rows(q, k, cu_seqlens, max_len, cu_seqlens_k, max_len_k, lengths, lengths_k)
    dev, st, packed = q.device, q.dtype, q.dim() == 3
    for name, t, shape, dtype in (("o", o, q.shape, st), ("lse", lse, q.shape[:-1], torch.float32)):
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")
        _check(name, t, shape, dtype, dev)
    _check_rows("do", do, q.shape, st, dev)
    dense = dense and do.is_contiguous()
    with _on_device(dev):
        new = torch.zeros if packed else torch.empty
        out = {"dq": new(q.shape, dtype=st, device=dev), "dk": new(k.shape, dtype=st, device=dev),
               "dv": new(k.shape, dtype=st, device=dev)}
        need = _attn_bytes(True, packed, r.b, r.Lq, r.Lk, r.tokens_q, r.tokens_k, H, G, D, code)
        ws = _workspace(need, dev)
        status = lib().ssm_attn_bwd(_at(q), _at(k), _at(v), _at(o), _at(lse), _at(do), _scale(scale, D), bool(causal),
                                    ctypes.byref(r), _at(out["dq"]), _at(out["dk"]), _at(out["dv"]), H, G, D, code,
                                    None if dense else _attn_strides(q, k, v, do), _at(ws), need, _raw_stream(dev))
    _raise(status, "ssm_attn_bwd")
    return out


def _pages(k_cache, v_cache, page_table, b, G, D, dtype, dev):
    """The descriptor of a paged cache [pages, page_size, G, D] whose pages are dense."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a torch.Tensor [b, max_pages]")
    most = page_table.shape[1]
    _check("page_table", page_table, (b, most), torch.int32, dev)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a torch.Tensor [pages, page_size, G, D]")
    shape = k_cache.shape
    n, size = shape[:2]
    if _alike(k_cache, v_cache) and v_cache.shape == shape and shape[2] == G and shape[3] == D and \
            k_cache.dtype == dtype and k_cache.device == dev:
        return Pages(page_table.data_ptr(), n, size, most, 0, 0)
    apart = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check_rows(name, t, (n, size, G, D), dtype, dev)
        st = t.stride()
        dense = all(m == 1 or s == want for m, s, want in zip(shape[1:], st[1:], (G * D, D, 1)))
        if not dense or (n > 1 and st[0] < size * G * D):
            raise ValueError(f"the pages of {name} must be contiguous")
        apart.append(st[0] if n > 1 else 0)
    return Pages(page_table.data_ptr(), n, size, most, *apart)


def ssm_attn_step(q, k_cache, v_cache, page_table, lengths, *, scale=None, max_len=0, o=None, return_lse=False):
    """Softmax attention of one new token a row over a paged cache (ssm_kv_append fills it): q [b, H, D]; k_cache and
    v_cache [pages, page_size, G, D], contiguous or with pages further apart (halves of one pool); page_table [b,
    max_pages] int32: token t of row i is in slot t mod page_size of page page_table[i, t // page_size]; lengths [b] int32:
    tokens of each row in the cache, the new one among them (all on the GPU). Table entries that are no page count as
    pages that are not there. max_len: the longest length that the call is planned for (0: what the table holds); rows may be
    longer. Returns o [b, H, D], or (o, lse [b, H] float32) when return_lse is set; a row without tokens has o = 0."""
    _on_gpu(q)
    if q.dim() != 3 or not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("q must be [b, H, D] and k_cache [pages, page_size, G, D]")
    b, H, D = q.shape
    G, dev, st = k_cache.shape[2], q.device, q.dtype
    code = _dtype_code(st)
    _check_rows("q", q, (b, H, D), st, dev)
    g = _pages(k_cache, v_cache, page_table, b, G, D, st, dev)
    if lengths is None:
        raise TypeError("lengths must be a torch.Tensor")
    _check("lengths", lengths, (b,), torch.int32, dev)
    with _on_device(dev):
        if o is None:
            o = torch.empty((b, H, D), dtype=st, device=dev)
        else:
            _check("o", o, (b, H, D), st, dev)
        lse = torch.empty((b, H), dtype=torch.float32, device=dev) if return_lse else None
        need = _step_bytes(b, H, G, D, g.pages, g.page_size, g.max_pages, g.k_page, g.v_page, max_len)
        ws = _workspace(need, dev)
        q_b, q_h = (0, 0) if q.is_contiguous() else q.stride()[:2]
        if (q_b, q_h) == (0, 0) and not q.is_contiguous():  # one row and head for all: as a tensor of its own
            q = q.contiguous()
        status = lib().ssm_attn_step(_at(q), _at(k_cache), _at(v_cache), ctypes.byref(g), _at(lengths), _scale(scale, D),
                                     _at(o), _at(lse), b, H, G, D, q_b, q_h, max_len, code, _at(ws), need,
                                     _raw_stream(dev))
    _raise(status, "ssm_attn_step")
    return (o, lse) if return_lse else o


def _new_tokens(x, cu_seqlens, new_lengths):
    """The descriptor of new tokens x: [b, heads, D] one a row, [b, L, heads, D], or [T, heads, D] with cu_seqlens."""
    dev = x.device
    if x.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens is for packed tokens [T, heads, D]")
        b, L = x.shape[:2]
        _check("new_lengths", new_lengths, (b,), torch.int32, dev)
        return Tokens(None, _at(new_lengths), b, L, b * L)
    if x.dim() != 3:
        raise ValueError("new tokens must be [b, heads, D], [b, L, heads, D], or [T, heads, D] with cu_seqlens")
    if new_lengths is not None:
        raise ValueError("new_lengths is for rows [b, L, heads, D]")
    T = x.shape[0]
    if cu_seqlens is None:
        return Tokens(None, None, T, 1, T)
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be a torch.Tensor [b + 1]")
    b = cu_seqlens.shape[0] - 1
    _check("cu_seqlens", cu_seqlens, (b + 1,), torch.int32, dev)
    return Tokens(cu_seqlens.data_ptr(), None, b, 0, T)


def _rotary(freq, D, dev) -> int:
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise ValueError("freq must be a torch.Tensor [rotary / 2]")
    _check("freq", freq, freq.shape, torch.float64, dev)
    if not 1 <= freq.shape[0] <= D // 2:
        raise ValueError("freq must have 1 to D / 2 entries")
    return 2 * freq.shape[0]


def ssm_kv_append(k, v, k_cache, v_cache, page_table, lengths, *, q=None, freq=None, cu_seqlens=None, new_lengths=None,
                  interleaved=False, q_out=None, k_out=None, return_k=False):
    """Appends the keys and values of new tokens to a paged cache (ssm_attn_step's), turning keys, and queries q if given,
    by their positions on the way. k, v: [b, G, D] (one token a row), [b, L, G, D] (new_lengths [b] int32: how many of each
    row count), or packed [T, G, D] with cu_seqlens [b + 1] int32; q likewise with H heads; views whose last axis is
    contiguous are read in place. lengths [b] int32: tokens of each row in the cache with the new ones, which are its last.
    freq [rotary/2] float64: radians a position of each coordinate pair (coordinates m and m + rotary/2, or 2m and 2m + 1 where
    interleaved); None: no rotation. Tokens that the row's pages do not reach are not stored.

    Returns (q_out, k_out): the turned queries (None without q) and, if return_k or k_out is given, the turned keys (else
    None). q_out may be q, and k_out k, where they are contiguous. Tokens of no row are 0 there (in place: as they were)."""
    _on_gpu(k)
    t = _new_tokens(k, cu_seqlens, new_lengths)
    G, D = k.shape[-2:]
    dev, st = k.device, k.dtype
    code = _dtype_code(st)
    _check_rows("k", k, k.shape, st, dev)
    _check_rows("v", v, k.shape, st, dev)
    H = G
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != k.dim():
            raise ValueError("q must be a torch.Tensor with as many axes as k")
        H = q.shape[-2]
        _check_rows("q", q, (*k.shape[:-2], H, D), st, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    g = _pages(k_cache, v_cache, page_table, t.b, G, D, st, dev)
    if lengths is None:
        raise TypeError("lengths must be a torch.Tensor")
    _check("lengths", lengths, (t.b,), torch.int32, dev)
    rotary = 0 if freq is None else _rotary(freq, D, dev)
    with _on_device(dev):
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=st, device=dev)
        if q is not None:
            _check("q_out", q_out, q.shape, st, dev)
        if return_k and k_out is None:
            k_out = torch.empty(k.shape, dtype=st, device=dev)
        _check("k_out", k_out, k.shape, st, dev)
        status = lib().ssm_kv_append(_at(q), _at(k), _at(v), _at(q_out), _at(k_out), _at(k_cache), _at(v_cache),
                                     ctypes.byref(g), _at(lengths), ctypes.byref(t), _at(freq), rotary, bool(interleaved), H, G,
                                     D, code, _token_strides(q, k, v), _raw_stream(dev))
    _raise(status, "ssm_kv_append")
    return q_out, k_out


def _token_strides(q, k, v):
    """Strides of new tokens; a single token of a row has those of its row."""
    if k.is_contiguous() and v.is_contiguous() and (q is None or q.is_contiguous()):
        return None
    ks, vs, qs = k.stride(), v.stride(), (0, 0, 0) if q is None else q.stride()
    return ctypes.byref(LinAttnStrides(qs[0], qs[-3], qs[-2], ks[0], ks[-3], ks[-2], vs[0], vs[-3], vs[-2]))


def ssm_rope(x, freq, *, lengths=None, cu_seqlens=None, new_lengths=None, interleaved=False, inverse=False, out=None):
    """Turns the heads of tokens x by their positions, as ssm_kv_append does on the way to the cache. x: [b, heads, D],
    [b, L, heads, D], or packed [T, heads, D] with cu_seqlens. The tokens of a row stand at its positions 0, 1, ..., or at the
    last ones of lengths [b] int32. inverse: by the opposite angles (the gradient: the rotation of a gradient back). Returns out
    (x's shape), which may be x itself where that is contiguous."""
    _on_gpu(x)
    t = _new_tokens(x, cu_seqlens, new_lengths)
    H, D = x.shape[-2:]
    dev, st = x.device, x.dtype
    code = _dtype_code(st)
    _check_rows("x", x, x.shape, st, dev)
    _check("lengths", lengths, (t.b,), torch.int32, dev)
    rotary = _rotary(freq, D, dev)
    with _on_device(dev):
        if out is None:
            out = torch.empty(x.shape, dtype=st, device=dev)
        _check("out", out, x.shape, st, dev)
        s = (0, 0, 0) if x.is_contiguous() else (x.stride(0), x.stride(-3), x.stride(-2))
        if s == (0, 0, 0) and not x.is_contiguous():
            x = x.contiguous()
        status = lib().ssm_rope(_at(x), _at(out), _at(lengths), ctypes.byref(t), _at(freq), rotary, bool(interleaved),
                                bool(inverse), H, D, *s, code, _raw_stream(dev))
    _raise(status, "ssm_rope")
    return out
