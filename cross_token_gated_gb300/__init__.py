"""GB300-native cross-token gate aggregation (TANGO / WANGO).

Python binding of the C-ABI library declared in ``include/tango.h``.  The binding
only marshals arguments: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  There is no fallback: if
the library cannot be loaded, every call raises.

Functions (same names as the C ABI):
  tango_aggregate, tango_aggregate_noalloc, wango_aggregate, tango_aggregate_save,
  wango_aggregate_save, tango_aggregate_backward, wango_aggregate_backward, wango_decode_step,
  tango_block_forward, tango_model_forward,
  tango_qk_norm_rope, tango_qk_norm_rope_backward, tg_rope_freqs, tango_cache_append, tango_paged_aggregate,
  tango_embed, tango_embed_backward, tango_norm, tango_norm_backward, tango_distill, tango_distill_backward,
  tango_sample,
  tg_workspace_size, tg_status_string, tg_check_device_error, tg_version
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

import torch

from . import build as _build

TG_OK, TG_ERR_INVALID_ARG, TG_ERR_UNSUPPORTED, TG_ERR_WORKSPACE, TG_ERR_CUDA, TG_ERR_TIMEOUT, \
    TG_ERR_DEVICE = range(7)
TG_F32, TG_BF16 = 0, 1
TG_FLAG_QK_NORMALIZED = 0x1
TG_FLAG_DEBUG_TIMEOUT = 0x100
TG_FLAG_FUSED_V = 0x200
TG_FLAG_BWD_FAR_SCAN = 0x400
TG_FLAG_BWD_FAR_PAIRS = 0x800
TG_MODE_TANGO, TG_MODE_WANGO = 0, 1
TG_WS_TANGO, TG_WS_WANGO, TG_WS_BLOCK, TG_WS_MODEL, TG_WS_DECODE, TG_WS_TANGO_BWD, TG_WS_WANGO_BWD = range(7)
TG_WS_QK_BWD, TG_WS_PAGED, TG_WS_EMBED_BWD, TG_WS_NORM_BWD = range(16, 20)
TG_ROPE_HALF, TG_ROPE_INTERLEAVED = 0, 1
TG_NORM_NONE, TG_NORM_UNIT, TG_NORM_RMS, TG_NORM_LAYER = range(4)
TG_MAX_TEACHER = 1024

HEADER = os.path.join(_build.INCLUDE, "tango.h")


class TgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class tg_agg_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("d_qk", ctypes.c_int),
                ("m", ctypes.c_int), ("s", ctypes.c_float), ("tau", ctypes.c_void_p),
                ("null_bias", ctypes.c_void_p), ("window", ctypes.c_int), ("phi_mode", ctypes.c_int),
                ("flags", ctypes.c_uint), ("dtype", ctypes.c_int), ("m_pitch", ctypes.c_int)]


class tg_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("rms_gamma", "Wq", "Wk", "Wg", "Wv", "Wo")]


class tg_block_params(ctypes.Structure):
    _fields_ = [("agg", tg_agg_params), ("d", ctypes.c_int), ("mode", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("rope_base", ctypes.c_float)]


class tg_model_weights(ctypes.Structure):
    _fields_ = [("embedding", ctypes.c_void_p), ("final_gamma", ctypes.c_void_p),
                ("sets", ctypes.POINTER(tg_block_weights))]


class tg_model_params(ctypes.Structure):
    _fields_ = [("block", tg_block_params), ("vocab", ctypes.c_int), ("n_apps", ctypes.c_int),
                ("n_sets", ctypes.c_int), ("set_of_app", ctypes.POINTER(ctypes.c_int)),
                ("final_rms_eps", ctypes.c_float)]


class tg_qk_params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("H", ctypes.c_int), ("H_k", ctypes.c_int), ("d_h", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int), ("norm", ctypes.c_int),
                ("eps", ctypes.c_float), ("T", ctypes.c_int), ("positions", ctypes.c_void_p),
                ("freqs", ctypes.c_void_p), ("q_gain", ctypes.c_void_p), ("k_gain", ctypes.c_void_p),
                ("q_pitch", ctypes.c_longlong), ("k_pitch", ctypes.c_longlong), ("dtype", ctypes.c_int)]


class tg_paged_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "d_h", "m", "m_pitch", "N", "max_new", "max_len", "page_size",
                                            "n_pages", "table_pitch")] + \
               [(n, ctypes.c_void_p) for n in ("cu_new", "lens", "page_table")] + \
               [("s", ctypes.c_float), ("tau", ctypes.c_void_p), ("null_bias", ctypes.c_void_p),
                ("v_pitch", ctypes.c_longlong), ("dtype", ctypes.c_int), ("flags", ctypes.c_uint)]


class tg_append_params(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int), ("norm", ctypes.c_int),
                ("eps", ctypes.c_float), ("freqs", ctypes.c_void_p), ("silu", ctypes.c_int),
                ("q_pitch", ctypes.c_longlong), ("k_pitch", ctypes.c_longlong), ("g_pitch", ctypes.c_longlong)]


class tg_embed_params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("d", ctypes.c_int), ("vocab", ctypes.c_int), ("scale", ctypes.c_float),
                ("pad_id", ctypes.c_int), ("pitch", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int)]


class tg_norm_params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("d", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_pitch", ctypes.c_longlong), ("dtype", ctypes.c_int)]


class tg_distill_params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("vocab", ctypes.c_int), ("k", ctypes.c_int),
                ("temperature", ctypes.c_float), ("pitch", ctypes.c_longlong), ("grad_pitch", ctypes.c_longlong),
                ("dtype", ctypes.c_int)]


class tg_sample_params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("vocab", ctypes.c_int), ("pitch", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("temperature", ctypes.c_float), ("top_k", ctypes.c_int), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()


def declared_functions() -> list[str]:
    """Names of the functions include/tango.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads (building in-tree first if needed) the C-ABI library."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_missing:
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"CUDA library {_build.LIB} is missing; build it with "
                               "`python -m cross_token_gated_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(_build.LIB)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        P = ctypes.POINTER
        for name in ("tango_aggregate", "wango_aggregate"):
            f = getattr(lib, name)
            f.argtypes = [P(tg_agg_params), vp, vp, vp, vp, vp, vp, sz, vp]
            f.restype = ctypes.c_int
        for name in ("tango_aggregate_backward", "wango_aggregate_backward"):
            f = getattr(lib, name)
            f.argtypes = [P(tg_agg_params), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            f.restype = ctypes.c_int
        for name in ("tango_aggregate_save", "wango_aggregate_save"):
            f = getattr(lib, name)
            f.argtypes = [P(tg_agg_params), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            f.restype = ctypes.c_int
        lib.tango_aggregate_noalloc.argtypes = [P(tg_agg_params), vp, vp, vp, vp, vp, vp]
        lib.tango_aggregate_noalloc.restype = ctypes.c_int
        lib.tango_block_forward.argtypes = [P(tg_block_params), P(tg_block_weights), vp, vp, vp, sz, vp]
        lib.tango_block_forward.restype = ctypes.c_int
        lib.wango_decode_step.argtypes = [P(tg_agg_params), ctypes.c_longlong, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.wango_decode_step.restype = ctypes.c_int
        lib.tango_model_forward.argtypes = [P(tg_model_params), P(tg_model_weights), vp, vp, vp, sz, vp]
        lib.tango_model_forward.restype = ctypes.c_int
        lib.tango_qk_norm_rope.argtypes = [P(tg_qk_params), vp, vp, vp, vp, vp]
        lib.tango_qk_norm_rope.restype = ctypes.c_int
        lib.tango_qk_norm_rope_backward.argtypes = [P(tg_qk_params)] + [vp] * 9 + [sz, vp]
        lib.tango_qk_norm_rope_backward.restype = ctypes.c_int
        db = ctypes.c_double
        lib.tg_rope_freqs.argtypes = [ctypes.c_int, db, db, ctypes.c_longlong, db, db, P(db)]
        lib.tg_rope_freqs.restype = ctypes.c_int
        lib.tango_cache_append.argtypes = [P(tg_paged_params), P(tg_append_params), vp, vp, vp, vp, vp, vp, vp]
        lib.tango_cache_append.restype = ctypes.c_int
        lib.tango_paged_aggregate.argtypes = [P(tg_paged_params), vp, vp, vp, vp, vp, vp, sz, vp]
        lib.tango_paged_aggregate.restype = ctypes.c_int
        for name, params, n_ptrs, has_ws in (
                ("tango_embed", tg_embed_params, 3, False), ("tango_embed_backward", tg_embed_params, 4, True),
                ("tango_norm", tg_norm_params, 4, False), ("tango_norm_backward", tg_norm_params, 7, True),
                ("tango_distill", tg_distill_params, 5, False), ("tango_distill_backward", tg_distill_params, 7, False),
                ("tango_sample", tg_sample_params, 4, False)):
            f = getattr(lib, name)
            f.argtypes = [P(params)] + [vp] * n_ptrs + ([vp, sz] if has_ws else []) + [vp]
            f.restype = ctypes.c_int
        lib.tg_workspace_size.argtypes = [ctypes.c_int, vp]
        lib.tg_workspace_size.restype = sz
        lib.tg_status_string.argtypes = [ctypes.c_int]
        lib.tg_status_string.restype = ctypes.c_char_p
        lib.tg_check_device_error.argtypes = [vp, P(ctypes.c_uint)]
        lib.tg_check_device_error.restype = ctypes.c_int
        lib.tg_version.argtypes = []
        lib.tg_version.restype = ctypes.c_int
        _lib = lib
        return lib


# ------------------------------------------------------------------ marshalling

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TG_F32
    if t.dtype == torch.bfloat16:
        return TG_BF16
    raise TypeError(f"unsupported storage dtype {t.dtype} (float32 or bfloat16)")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def agg_params(B, T, H, d_qk, m, *, dtype, s=10.0, tau=None, null_bias=None, window=1, phi_mode=0,
               flags=0, m_pitch=0) -> tg_agg_params:
    return tg_agg_params(B, T, H, d_qk, m, float(s), _ptr(tau), _ptr(null_bias), int(window),
                         int(phi_mode), int(flags), int(dtype), int(m_pitch))


def _gate_width(g, H, m_h):
    """(m, m_pitch) for a gate tensor of last dimension H * pitch: the logical total width
    H * m_h and the per-head pitch (0 when dense)."""
    width = g.shape[-1]
    if m_h is None:
        return width, 0
    if width % H != 0:
        raise ValueError("gate tensor width must be H * m_pitch")
    return H * int(m_h), width // H


def status_string(status: int) -> str:
    return load().tg_status_string(int(status)).decode()


tg_status_string = status_string


def tg_workspace_size(which: int, params) -> int:
    return int(load().tg_workspace_size(int(which), ctypes.byref(params)))


def tg_check_device_error(stream=None):
    """(status, raw word) after synchronising the stream."""
    word = ctypes.c_uint(0)
    st = load().tg_check_device_error(_stream(stream), ctypes.byref(word))
    return st, word.value


def tg_version() -> int:
    return int(load().tg_version())


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return None
    if ws is not None:
        return ws
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _scratch(nbytes: int, device, ws, stream):
    """_workspace for a call on `stream`.  Scratch made here is allocated on that stream, so
    that memory is neither taken while another stream's work on it is pending nor given
    away before the call has run."""
    if ws is not None or stream is None:
        return _workspace(nbytes, device, ws)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return _workspace(nbytes, device, None)


def _ws_ptr(ws):
    if ws is None:
        return None, 0
    p = ws.data_ptr()
    aligned = (p + 255) & ~255
    return aligned, ws.numel() - (aligned - p)


def _aggregate(fn_name, q, k, g, v, out, *, H, s, tau, null_bias, window, phi_mode, flags, ws, stream, m_h=None,
               saved=None):
    B, T, d_qk = q.shape
    m, pitch = _gate_width(g, H, m_h)
    p = agg_params(B, T, H, d_qk, m, dtype=_dtype_code(g), s=s, tau=tau, null_bias=null_bias,
                   window=window, phi_mode=phi_mode, flags=flags, m_pitch=pitch)
    which = TG_WS_TANGO if fn_name.startswith("tango") else TG_WS_WANGO
    need = load().tg_workspace_size(which, ctypes.byref(p))
    wbuf = _workspace(need, g.device, ws)
    wp, wn = _ws_ptr(wbuf)
    extra = () if saved is None else (_ptr(saved[0]), _ptr(saved[1]))
    st = getattr(load(), fn_name)(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(g), _ptr(v), _ptr(out), *extra, wp, wn,
                                  _stream(stream))
    if st != TG_OK:
        raise TgError(st, fn_name)
    return out


def tango_aggregate(q, k, g, v, out, *, H, s=10.0, tau=None, null_bias=None, flags=0, ws=None,
                    stream=None, m_h=None):
    """Full-prefix aggregation (eqs. 5-6).  q, k [B, T, d_qk]; g, v, out [B, T, m] on the
    device, one storage dtype.  v may be None (then out = gbar).  With m_h given, the gate
    tensors are [B, T, H * pitch] and each head's m_h gates sit at a pitch of
    g.shape[-1] / H columns (m_pitch in tango.h)."""
    return _aggregate("tango_aggregate", q, k, g, v, out, H=H, s=s, tau=tau, null_bias=null_bias,
                      window=1, phi_mode=0, flags=flags, ws=ws, stream=stream, m_h=m_h)


def wango_aggregate(q, k, g, v, out, *, H, window, s=10.0, tau=None, null_bias=None, phi_mode=0,
                    flags=0, ws=None, stream=None, m_h=None):
    """Windowed aggregation (eqs. 7-10); arguments as for tango_aggregate."""
    return _aggregate("wango_aggregate", q, k, g, v, out, H=H, s=s, tau=tau, null_bias=null_bias,
                      window=window, phi_mode=phi_mode, flags=flags, ws=ws, stream=stream, m_h=m_h)


def tango_aggregate_save(q, k, g, v, out, gbar, den, *, H, s=10.0, tau=None, null_bias=None, flags=0, ws=None,
                         stream=None, m_h=None):
    """tango_aggregate that also writes gbar (laid out as out) and den (float32 [B, H, T])
    for the backward (bf16)."""
    return _aggregate("tango_aggregate_save", q, k, g, v, out, H=H, s=s, tau=tau, null_bias=null_bias, window=1,
                      phi_mode=0, flags=flags, ws=ws, stream=stream, m_h=m_h, saved=(gbar, den))


def wango_aggregate_save(q, k, g, v, out, gbar, den, *, H, window, s=10.0, tau=None, null_bias=None, phi_mode=0,
                         flags=0, ws=None, stream=None, m_h=None):
    """wango_aggregate that also writes gbar and den for the backward (bf16)."""
    return _aggregate("wango_aggregate_save", q, k, g, v, out, H=H, s=s, tau=tau, null_bias=null_bias,
                      window=window, phi_mode=phi_mode, flags=flags, ws=ws, stream=stream, m_h=m_h,
                      saved=(gbar, den))


def _aggregate_backward(fn_name, q, k, g, v, dout, dq, dk, dg, dv, *, H, s, tau, null_bias, window, phi_mode,
                        flags, ws, stream, m_h=None, gbar=None, den=None):
    B, T, d_qk = q.shape
    m, pitch = _gate_width(g, H, m_h)
    p = agg_params(B, T, H, d_qk, m, dtype=_dtype_code(g), s=s, tau=tau, null_bias=null_bias,
                   window=window, phi_mode=phi_mode, flags=flags, m_pitch=pitch)
    which = TG_WS_TANGO_BWD if fn_name == "tango_aggregate_backward" else TG_WS_WANGO_BWD
    need = load().tg_workspace_size(which, ctypes.byref(p))
    wbuf = _workspace(need, g.device, ws)
    wp, wn = _ws_ptr(wbuf)
    st = getattr(load(), fn_name)(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(g), _ptr(v), _ptr(dout), _ptr(gbar),
                                  _ptr(den), _ptr(dq), _ptr(dk), _ptr(dg), _ptr(dv), wp, wn, _stream(stream))
    if st != TG_OK:
        raise TgError(st, fn_name)
    return dq, dk, dg, dv


def tango_aggregate_backward(q, k, g, v, dout, dq, dk, dg, dv, *, H, s=10.0, tau=None, null_bias=None, flags=0,
                             ws=None, stream=None, m_h=None, gbar=None, den=None):
    """Gradients of sum(dout * tango_aggregate(q, k, g, v)) with respect to q, k, g, v
    (bf16).  dq, dk [B, T, d_qk] and dg, dv [B, T, m] are written; v and dv may be None."""
    return _aggregate_backward("tango_aggregate_backward", q, k, g, v, dout, dq, dk, dg, dv, H=H, s=s, tau=tau,
                               null_bias=null_bias, window=1, phi_mode=0, flags=flags, ws=ws, stream=stream,
                               m_h=m_h, gbar=gbar, den=den)


def wango_aggregate_backward(q, k, g, v, dout, dq, dk, dg, dv, *, H, window, s=10.0, tau=None, null_bias=None,
                             phi_mode=0, flags=0, ws=None, stream=None, m_h=None, gbar=None, den=None):
    """Gradients of sum(dout * wango_aggregate(q, k, g, v)); arguments as for
    tango_aggregate_backward."""
    return _aggregate_backward("wango_aggregate_backward", q, k, g, v, dout, dq, dk, dg, dv, H=H, s=s, tau=tau,
                               null_bias=null_bias, window=window, phi_mode=phi_mode, flags=flags, ws=ws,
                               stream=stream, m_h=m_h, gbar=gbar, den=den)


def tango_aggregate_noalloc(q, k, g, v, out, *, H, s=10.0, tau=None, null_bias=None, flags=0,
                            stream=None):
    """tango_aggregate without a workspace: the library's fixed device scratch array is
    used instead (for callers that cannot allocate device memory).  Raises TgError with
    TG_ERR_WORKSPACE when the problem needs more scratch than TG_NOALLOC_SCRATCH_BYTES."""
    B, T, d_qk = q.shape
    m = g.shape[-1]
    p = agg_params(B, T, H, d_qk, m, dtype=_dtype_code(g), s=s, tau=tau, null_bias=null_bias, flags=flags)
    st = load().tango_aggregate_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(g), _ptr(v), _ptr(out),
                                        _stream(stream))
    if st != TG_OK:
        raise TgError(st, "tango_aggregate_noalloc")
    return out


TG_NOALLOC_SCRATCH_BYTES = 16 << 20


def block_params(B, T, d, H, d_qk, m, *, dtype, mode=TG_MODE_TANGO, s=10.0, tau=None, null_bias=None,
                 window=1, phi_mode=0, rms_eps=1e-6, rope_base=10000.0, flags=0) -> tg_block_params:
    return tg_block_params(agg_params(B, T, H, d_qk, m, dtype=dtype, s=s, tau=tau, null_bias=null_bias,
                                      window=window, phi_mode=phi_mode, flags=flags), int(d), int(mode),
                           float(rms_eps), float(rope_base))


def tango_block_forward(h, weights, h_out, *, H, mode=TG_MODE_TANGO, s=10.0, tau=None, null_bias=None,
                        window=1, phi_mode=0, rms_eps=1e-6, rope_base=10000.0, flags=0, ws=None, stream=None):
    """One block application (eqs. 2-10).  h, h_out [B, T, d]; weights: dict with gamma,
    Wq, Wk, Wg, Wv, Wo device tensors of h's dtype.  h_out may be h.  flags: 0,
    TG_FLAG_DEBUG_TIMEOUT (the projection GEMM's test hook) and/or TG_FLAG_FUSED_V
    (WANGO: v formed inside the aggregation instead of by the projection GEMM)."""
    B, T, d = h.shape
    d_qk, m = weights["Wq"].shape[0], weights["Wg"].shape[0]
    p = block_params(B, T, d, H, d_qk, m, dtype=_dtype_code(h), mode=mode, s=s, tau=tau,
                     null_bias=null_bias, window=window, phi_mode=phi_mode, rms_eps=rms_eps,
                     rope_base=rope_base, flags=flags)
    w = tg_block_weights(*[_ptr(weights[n]) for n in ("gamma", "Wq", "Wk", "Wg", "Wv", "Wo")])
    need = load().tg_workspace_size(TG_WS_BLOCK, ctypes.byref(p))
    wbuf = _workspace(need, h.device, ws)
    wp, wn = _ws_ptr(wbuf)
    st = load().tango_block_forward(ctypes.byref(p), ctypes.byref(w), _ptr(h), _ptr(h_out), wp, wn,
                                    _stream(stream))
    if st != TG_OK:
        raise TgError(st, "tango_block_forward")
    return h_out


def block_workspace(B, T, d, H, d_qk, m, *, dtype, mode=TG_MODE_TANGO, window=1, device="cuda"):
    """Allocates a workspace tensor large enough for tango_block_forward."""
    p = block_params(B, T, d, H, d_qk, m, dtype=dtype, mode=mode, window=window)
    return _workspace(tg_workspace_size(TG_WS_BLOCK, p), device, None)


def model_params(B, T, d, H, d_qk, m, vocab, *, dtype, n_apps=4, n_sets=1, set_of_app=None,
                 mode=TG_MODE_TANGO, s=10.0, tau=None, null_bias=None, window=1, phi_mode=0, rms_eps=1e-6,
                 rope_base=10000.0, final_rms_eps=1e-6):
    """tg_model_params; the returned structure keeps its set_of_app array alive."""
    table = None
    if set_of_app is not None:
        table = (ctypes.c_int * len(set_of_app))(*[int(x) for x in set_of_app])
    p = tg_model_params(block_params(B, T, d, H, d_qk, m, dtype=dtype, mode=mode, s=s, tau=tau,
                                     null_bias=null_bias, window=window, phi_mode=phi_mode, rms_eps=rms_eps,
                                     rope_base=rope_base),
                        int(vocab), int(n_apps), int(n_sets),
                        ctypes.cast(table, ctypes.POINTER(ctypes.c_int)) if table is not None else None,
                        float(final_rms_eps))
    p._table = table
    return p


def tango_model_forward(ids, embedding, final_gamma, sets, logits, *, H, n_apps=4, set_of_app=None,
                        mode=TG_MODE_TANGO, s=10.0, tau=None, null_bias=None, window=1, phi_mode=0,
                        rms_eps=1e-6, rope_base=10000.0, final_rms_eps=1e-6, ws=None, stream=None):
    """The shared-block language model (sec. 2.3): embedding, n_apps block applications,
    final RMSNorm, tied logits.  ids: device int32 [B, T]; embedding [vocab, d];
    final_gamma [d]; sets: list of weight dicts (gamma, Wq, Wk, Wg, Wv, Wo) of one gate
    width; logits [B, T, vocab], written."""
    if ids.dtype != torch.int32:
        raise TypeError("ids must be an int32 tensor")
    B, T = ids.shape
    vocab, d = embedding.shape
    d_qk, m = sets[0]["Wq"].shape[0], sets[0]["Wg"].shape[0]
    p = model_params(B, T, d, H, d_qk, m, vocab, dtype=_dtype_code(embedding), n_apps=n_apps,
                     n_sets=len(sets), set_of_app=set_of_app, mode=mode, s=s, tau=tau, null_bias=null_bias,
                     window=window, phi_mode=phi_mode, rms_eps=rms_eps, rope_base=rope_base,
                     final_rms_eps=final_rms_eps)
    arr = (tg_block_weights * len(sets))(
        *[tg_block_weights(*[_ptr(w[n]) for n in ("gamma", "Wq", "Wk", "Wg", "Wv", "Wo")]) for w in sets])
    w = tg_model_weights(_ptr(embedding), _ptr(final_gamma), ctypes.cast(arr, ctypes.POINTER(tg_block_weights)))
    need = load().tg_workspace_size(TG_WS_MODEL, ctypes.byref(p))
    wbuf = _workspace(need, ids.device, ws)
    wp, wn = _ws_ptr(wbuf)
    st = load().tango_model_forward(ctypes.byref(p), ctypes.byref(w), _ptr(ids), _ptr(logits), wp, wn,
                                    _stream(stream))
    if st != TG_OK:
        raise TgError(st, "tango_model_forward")
    return logits


def decode_state(B, H, d_qk, m, *, window, dtype, device="cuda"):
    """Allocates a state buffer for wango_decode_step (cleared by the step at pos 0)."""
    p = agg_params(B, 1, H, d_qk, m, dtype=dtype, window=window)
    return _workspace(tg_workspace_size(TG_WS_DECODE, p), device, None)


def wango_decode_step(q, k, g, v, out, state, pos, *, H, window, s=10.0, tau=None, null_bias=None,
                      phi_mode=0, flags=0, stream=None):
    """One autoregressive WANGO step for B sequences at position pos.  q, k [B, d_qk];
    g, v, out [B, m]; state from decode_state(), kept between steps (pos = 0, 1, ...)."""
    B, d_qk = q.shape
    m = g.shape[-1]
    p = agg_params(B, 1, H, d_qk, m, dtype=_dtype_code(g), s=s, tau=tau, null_bias=null_bias, window=window,
                   phi_mode=phi_mode, flags=flags)
    wp, wn = _ws_ptr(state)
    st = load().wango_decode_step(ctypes.byref(p), int(pos), _ptr(q), _ptr(k), _ptr(g), _ptr(v), _ptr(out),
                                  wp, wn, _stream(stream))
    if st != TG_OK:
        raise TgError(st, "wango_decode_step")
    return out


# ----------------------------------------------- norm and rotary position of q and k

# These calls serve single tokens, whose kernels take a few microseconds: the checks are
# written to cost little beside them.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_HERE = contextlib.nullcontext()


def _on_device(dev):
    """The context that a call on tensors of device dev runs in.  The library launches on the
    current device and sizes its grids and scratch by it, so another one is made current for the
    call; host tensors (dev < 0) are refused, as their addresses mean nothing to a kernel."""
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    return _HERE if dev == _current_device() else torch.cuda.device(dev)


def _given_ws(ws, dev):
    """A caller's scratch, checked as far as the library's own size check does not see."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous memory of the call's device")
    return ws


def _stream_on(stream, dev):
    """The stream to launch on: the caller's, or device dev's current one."""
    if stream is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return _stream(stream)


def _bad(t, name, dtype, dev, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not with the call's other tensors")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, dtype, dev, shape=None):
    """Address of a contiguous tensor of this type, device and shape; raises otherwise."""
    if t.dtype is not dtype or t.get_device() != dev or (shape is not None and t.shape != shape) \
            or not t.is_contiguous():
        _bad(t, name, dtype, dev, shape)
    return t.data_ptr()


_MOST_INT = 2 ** 31 - 1  # of the parameters' int fields, which ctypes would cut to their low bits


def _too_large(name):
    raise ValueError(f"{name}'s sizes and numbers must be below 2^31")


def _rows_pitch(t, name, dtype, dev):
    """(rows, width, pitch in elements) of a [..., width] tensor whose rows lie at one pitch
    (a dense tensor, or a column slice of one)."""
    if t.dtype is not dtype or t.get_device() != dev:
        _bad(t, name, dtype, dev, None)
    shape, stride = t.shape, t.stride()
    if len(shape) < 2 or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be [..., width] with unit stride along its last dimension")
    if shape[-1] > _MOST_INT:
        _too_large(name)
    if len(shape) == 2:
        rows, width = shape
        pitch = stride[0] if rows > 1 else width
        if pitch < width and rows > 1:
            raise ValueError(f"{name}'s rows overlap")
        return rows, width, pitch
    width, rows, pitch = shape[-1], 1, 0
    for n, st in zip(shape[-2::-1], stride[-2::-1]):
        if n != 1:
            if rows == 1:
                pitch = st
            elif rows and st != pitch * rows:
                raise ValueError(f"{name}'s rows must lie at one pitch")
            rows *= n
    if rows > 1 and pitch < width:
        raise ValueError(f"{name}'s rows overlap")
    return rows, width, pitch if pitch > width else width


def _optional(t, name, dtype, dev, shape=None):
    return None if t is None else _dense(t, name, dtype, dev, shape)


def _qk_params(q, k, outs, freqs, H, H_k, positions, layout, norm, q_gain, k_gain, eps):
    """tg_qk_params, and the addresses of the dense tensors `outs`: (name, tensor, input)."""
    dt, dev = q.dtype, q.get_device()
    rows, width, q_pitch = _rows_pitch(q, "q", dt, dev)
    d_h = width // H
    if d_h * H != width:
        raise ValueError("q's width must be H heads")
    k_pitch = 0
    if k is None:
        H_k = 0
    else:
        H_k = H if H_k is None else H_k
        k_rows, k_width, k_pitch = _rows_pitch(k, "k", dt, dev)
        if k_rows != rows or k_width != H_k * d_h:
            raise ValueError("k must have q's rows and H_k heads of q's head width")
    ptrs = []
    for name, t, src in outs:
        if (t is None) != (src is None):
            raise ValueError(f"{name} goes with its input")
        ptrs.append(None if t is None else _dense(t, name, dt, dev, src.shape))
    rotary, fp = 0, None
    if freqs is not None:
        fp = _dense(freqs, "freqs", torch.float64, dev)
        rotary = 2 * freqs.numel()
    pp = None
    if positions is not None:
        pp = _dense(positions, "positions", torch.int32, dev)
        if positions.numel() != rows:
            raise ValueError("positions must hold one entry per row")
    p = tg_qk_params(rows, H, H_k, d_h, rotary, layout, norm, eps, q.shape[-2] or 1, pp, fp,
                     _optional(q_gain, "q_gain", torch.float32, dev, (d_h,)),
                     _optional(k_gain, "k_gain", torch.float32, dev, (d_h,)), q_pitch, k_pitch, _dtype_code(q))
    return p, ptrs, dev


def tg_rope_freqs(rotary_dim, *, base=10000.0, factor=1.0, orig_len=0, turns_lo=1.0, turns_hi=32.0, device="cuda"):
    """float64 [rotary_dim / 2]: radians per position, scaled for contexts `factor` times
    longer than orig_len positions (0: all of them interpolated; see tango.h)."""
    buf = (ctypes.c_double * max(1, rotary_dim // 2))()
    st = load().tg_rope_freqs(int(rotary_dim), float(base), float(factor), int(orig_len), float(turns_lo),
                              float(turns_hi), buf)
    if st != TG_OK:
        raise TgError(st, "tg_rope_freqs")
    return torch.tensor(list(buf)[:rotary_dim // 2], dtype=torch.float64, device=device)


def tango_qk_norm_rope(q, k, q_out, k_out, freqs, *, H, H_k=None, positions=None, layout=TG_ROPE_HALF,
                       norm=TG_NORM_UNIT, q_gain=None, k_gain=None, eps=1e-6, stream=None):
    """Norm and rotary position of every head of q [..., T, H * d_h] and k [..., T, H_k *
    d_h] (k may be None) into q_out, k_out (dense).  q and k may be column slices.  freqs:
    float64 [rotary / 2] from tg_rope_freqs, or None (no rotation).  positions: int32, one
    per row, or None (the index along T).  q_gain, k_gain: float32 [d_h] or None."""
    p, (qo, ko), dev = _qk_params(q, k, (("q_out", q_out, q), ("k_out", k_out, k)), freqs, H, H_k, positions, layout,
                                  norm, q_gain, k_gain, eps)
    with _on_device(dev):
        st = (_lib or load()).tango_qk_norm_rope(ctypes.byref(p), _ptr(q), _ptr(k), qo, ko, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_qk_norm_rope")
    return q_out, k_out


def tango_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, freqs, *, H, H_k=None, positions=None,
                                layout=TG_ROPE_HALF, norm=TG_NORM_UNIT, q_gain=None, k_gain=None, dq_gain=None,
                                dk_gain=None, eps=1e-6, ws=None, stream=None):
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) with respect to q and k (into
    dq, dk, dense) and, where dq_gain / dk_gain (float32 [d_h]) are given, to the gains."""
    p, (dqo, dko, dqp, dkp), dev = _qk_params(
        q, k, (("dq_out", dq_out, q), ("dk_out", dk_out, k), ("dq", dq, q), ("dk", dk, k)), freqs, H, H_k, positions,
        layout, norm, q_gain, k_gain, eps)
    dqg = _optional(dq_gain, "dq_gain", torch.float32, dev, (p.d_h,))
    dkg = _optional(dk_gain, "dk_gain", torch.float32, dev, (p.d_h,))
    wp, wn, wbuf = None, 0, None
    with _on_device(dev):
        if dqg is not None or dkg is not None:
            wbuf = _given_ws(ws, dev) if ws is not None else _scratch(
                load().tg_workspace_size(TG_WS_QK_BWD, ctypes.byref(p)), q.device, None, stream)
            wp, wn = _ws_ptr(wbuf)
        st = load().tango_qk_norm_rope_backward(ctypes.byref(p), _ptr(q), _ptr(k), dqo, dko, dqp, dkp, dqg, dkg, wp,
                                                wn, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_qk_norm_rope_backward")
    return dq, dk


# --------------------------------------------------------------------- paged cache

def cache_pools(n_pages, page_size, H, d_h, m_h, *, dtype=torch.bfloat16, m_pitch=None, device="cuda"):
    """(k_pages, g_pages) of a paged cache: [n_pages, page_size, H * d_h] and [n_pages,
    page_size, H * m_pitch].  In bf16 the default pitch is m_h rounded up to 8."""
    if m_pitch is None:
        m_pitch = -(-m_h // 8) * 8 if dtype == torch.bfloat16 else m_h
    return (torch.zeros(n_pages, page_size, H * d_h, dtype=dtype, device=device),
            torch.zeros(n_pages, page_size, H * m_pitch, dtype=dtype, device=device))


def paged_params(N, k_pages, g_pages, page_table, cu_new, lens, *, H, max_new, max_len, m_h=None, s=10.0, tau=None,
                 null_bias=None, v_pitch=0, flags=0) -> tg_paged_params:
    """tg_paged_params of a batch: page_table int32 [B, pages], cu_new int32 [B + 1], lens
    int32 [B]."""
    n_pages, page_size, dqk = k_pages.shape
    gp, gs, width = g_pages.shape
    pitch = width // H
    if dqk % H != 0 or gp != n_pages or gs != page_size or pitch * H != width:
        raise ValueError("k_pages and g_pages must be [n_pages, page_size, H * width]")
    dt, dev = k_pages.dtype, k_pages.get_device()
    _dense(k_pages, "k_pages", dt, dev)
    _dense(g_pages, "g_pages", dt, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, pages]")
    B, cols = page_table.shape
    i32 = torch.int32
    tp = _dense(page_table, "page_table", i32, dev)
    cp = _dense(cu_new, "cu_new", i32, dev, (B + 1,))
    lp = _dense(lens, "lens", i32, dev, (B,))
    return tg_paged_params(B, H, dqk // H, H * (pitch if m_h is None else int(m_h)), pitch, N, max_new, max_len,
                           page_size, n_pages, cols, cp, lp, tp, s, _optional(tau, "tau", torch.float32, dev, (H,)),
                           _optional(null_bias, "null_bias", torch.float32, dev, (H,)), v_pitch, _dtype_code(k_pages),
                           flags)


def tango_cache_append(q, k, g, q_out, k_pages, g_pages, page_table, cu_new, lens, freqs, *, H, m_h=None,
                       layout=TG_ROPE_HALF, norm=TG_NORM_UNIT, eps=1e-6, silu=True, stream=None):
    """Appends the new tokens of a ragged batch to the paged cache: k [N, H * d_h] normed
    and rotated at its position, g [N, H * pitch] (the gate projection; through SiLU unless
    silu=False).  q (or None) is normed and rotated into q_out for the aggregation.  lens
    [B] counts the new tokens in; cu_new [B + 1] are the sequences' row offsets."""
    dt, dev = k_pages.dtype, k_pages.get_device()
    N, k_width, k_pitch = _rows_pitch(k, "k", dt, dev)
    g_rows, g_width, g_pitch = _rows_pitch(g, "g", dt, dev)
    p = paged_params(N, k_pages, g_pages, page_table, cu_new, lens, H=H, max_new=N or 1,
                     max_len=page_table.shape[-1] * k_pages.shape[1], m_h=m_h)
    if k_width != k_pages.shape[2] or g_width != g_pages.shape[2] or g_rows != N:
        raise ValueError("k and g must have one row per new token, as wide as the cache's")
    if (q is None) != (q_out is None):
        raise ValueError("q_out goes with q")
    q_pitch, qo = 0, None
    if q is not None:
        q_rows, q_width, q_pitch = _rows_pitch(q, "q", dt, dev)
        if q_rows != N or q_width != k_width:
            raise ValueError("q must have k's rows and width")
        qo = _dense(q_out, "q_out", dt, dev, q.shape)
    rotary, fp = 0, None
    if freqs is not None:
        fp = _dense(freqs, "freqs", torch.float64, dev)
        rotary = 2 * freqs.numel()
    a = tg_append_params(rotary, layout, norm, eps, fp, 1 if silu else 0, q_pitch, k_pitch, g_pitch)
    with _on_device(dev):
        st = (_lib or load()).tango_cache_append(ctypes.byref(p), ctypes.byref(a), _ptr(q), k.data_ptr(),
                                                 g.data_ptr(), qo, k_pages.data_ptr(), g_pages.data_ptr(),
                                                 _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_cache_append")
    return q_out


def tango_paged_aggregate(q, v, out, k_pages, g_pages, page_table, cu_new, lens, *, H, max_new, max_len, s=10.0,
                          tau=None, null_bias=None, m_h=None, flags=0, ws=None, stream=None):
    """TANGO aggregation of the new tokens (already appended) over the paged cache.  q [N,
    H * d_h] unit vectors per head; v [N, H * pitch] or None (out = gbar); out [N, H *
    pitch].  max_new, max_len: host bounds of the sequences' new tokens and lengths."""
    dt, dev = k_pages.dtype, k_pages.get_device()
    N, width = q.shape[0], g_pages.shape[2]
    qp = _dense(q, "q", dt, dev)
    op = _dense(out, "out", dt, dev)
    if q.numel() != N * k_pages.shape[2] or out.numel() != N * width:
        raise ValueError("q and out must have one row per new token, as wide as the cache's")
    v_pitch = 0
    if v is not None:
        v_rows, v_width, v_pitch = _rows_pitch(v, "v", dt, dev)
        if v_rows != N or v_width != width:
            raise ValueError("v must have one row per new token, as wide as the cache's gates")
    p = paged_params(N, k_pages, g_pages, page_table, cu_new, lens, H=H, max_new=max_new, max_len=max_len, m_h=m_h,
                     s=s, tau=tau, null_bias=null_bias, v_pitch=v_pitch, flags=flags)
    lib, ref = _lib or load(), ctypes.byref(p)
    with _on_device(dev):
        wbuf = _given_ws(ws, dev) if ws is not None else _scratch(lib.tg_workspace_size(TG_WS_PAGED, ref), q.device,
                                                                  None, stream)
        wp, wn = _ws_ptr(wbuf)
        st = lib.tango_paged_aggregate(ref, qp, _ptr(v), op, k_pages.data_ptr(), g_pages.data_ptr(), wp, wn,
                                       _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_paged_aggregate")
    return out


# ------------------------------------------------------- the model's ends: lookup and norm

def _embed_params(ids, width, rows, pitch, vocab, dtype, grad_dtype, scale, pad_id, dev):
    if ids.numel() != rows:
        raise ValueError("ids must hold one token per row")
    if not -_MOST_INT - 1 <= pad_id <= _MOST_INT:
        raise ValueError("pad_id must be an int32 as ids are")
    ip = _dense(ids, "ids", torch.int32, dev)
    return tg_embed_params(rows, width, vocab, scale, pad_id, pitch, dtype, grad_dtype), ip


def _matrix(t, name, dtype, dev, width=None):
    """Address of a dense [rows, width] tensor."""
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name} must be a matrix" + ("" if width is None else f" of {width} columns"))
    if t.shape[0] > _MOST_INT:  # (its width is looked at with its rows')
        _too_large(name)
    return _dense(t, name, dtype, dev)


def tango_embed(ids, embedding, out, *, scale=1.0, pad_id=-1, stream=None):
    """out[n] = scale * embedding[ids[n]]: ids int32 [...], embedding [vocab, d], out [..., d] (its
    rows at one pitch).  Ids equal to pad_id give zero rows."""
    dt, dev = embedding.dtype, embedding.get_device()
    ep = _matrix(embedding, "embedding", dt, dev)
    vocab, d = embedding.shape
    rows, width, pitch = _rows_pitch(out, "out", dt, dev)
    if width != d:
        raise ValueError("out must be as wide as the embedding")
    code = _dtype_code(embedding)
    p, ip = _embed_params(ids, d, rows, pitch, vocab, code, code, scale, pad_id, dev)
    with _on_device(dev):
        st = (_lib or load()).tango_embed(ctypes.byref(p), ip, ep, out.data_ptr(), _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_embed")
    return out


def tango_embed_backward(ids, dout, dembedding, *, base=None, scale=1.0, pad_id=-1, ws=None, stream=None):
    """dembedding[v] = base[v] + scale * sum of dout's rows whose id is v: ids int32 [...], dout
    [..., d] (its rows at one pitch), dembedding and base [vocab, d] float32 or bfloat16.  base may
    be None (zeros) or dembedding itself (accumulation)."""
    dt, gt, dev = dout.dtype, dembedding.dtype, dout.get_device()
    gp = _matrix(dembedding, "dembedding", gt, dev)
    vocab, d = dembedding.shape
    bp = _optional(base, "base", gt, dev, dembedding.shape)
    rows, width, pitch = _rows_pitch(dout, "dout", dt, dev)
    if width != d:
        raise ValueError("dout must be as wide as dembedding")
    p, ip = _embed_params(ids, d, rows, pitch, vocab, _dtype_code(dout), _dtype_code(dembedding), scale, pad_id, dev)
    lib, ref = _lib or load(), ctypes.byref(p)
    with _on_device(dev):
        wbuf = _given_ws(ws, dev) if ws is not None else _scratch(lib.tg_workspace_size(TG_WS_EMBED_BWD, ref),
                                                                  dout.device, None, stream)
        wp, wn = _ws_ptr(wbuf)
        st = lib.tango_embed_backward(ref, ip, dout.data_ptr(), bp, gp, wp, wn, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_embed_backward")
    return dembedding


def tango_norm(x, gamma, beta, y, *, norm=TG_NORM_RMS, eps=1e-6, stream=None):
    """y = gamma * n + beta with n the RMS (or TG_NORM_LAYER) norm of x's rows: x [..., d], its rows
    at one pitch; gamma and beta [d] or None; y dense, like x."""
    dt, dev = x.dtype, x.get_device()
    rows, d, pitch = _rows_pitch(x, "x", dt, dev)
    yp = _dense(y, "y", dt, dev, x.shape)
    gp = None if gamma is None else _dense(gamma, "gamma", dt, dev, (d,))
    bp = None if beta is None else _dense(beta, "beta", dt, dev, (d,))
    p = tg_norm_params(rows, d, norm, eps, pitch, _dtype_code(x))
    with _on_device(dev):
        st = (_lib or load()).tango_norm(ctypes.byref(p), x.data_ptr(), gp, bp, yp, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_norm")
    return y


def tango_norm_backward(x, gamma, dy, dx, *, norm=TG_NORM_RMS, eps=1e-6, dres=None, dgamma=None, dbeta=None, ws=None,
                        stream=None):
    """Gradients of tango_norm: dx (dense, like x) from dy, plus dres where given; dgamma and dbeta
    (float32 [d]) where given."""
    dt, dev = x.dtype, x.get_device()
    rows, d, pitch = _rows_pitch(x, "x", dt, dev)
    shape, f32 = x.shape, torch.float32
    dyp, dxp = _dense(dy, "dy", dt, dev, shape), _dense(dx, "dx", dt, dev, shape)
    rp = None if dres is None else _dense(dres, "dres", dt, dev, shape)
    gp = None if gamma is None else _dense(gamma, "gamma", dt, dev, (d,))
    dgp = None if dgamma is None else _dense(dgamma, "dgamma", f32, dev, (d,))
    dbp = None if dbeta is None else _dense(dbeta, "dbeta", f32, dev, (d,))
    p = tg_norm_params(rows, d, norm, eps, pitch, _dtype_code(x))
    lib, ref = _lib or load(), ctypes.byref(p)
    wp, wn, wbuf = None, 0, None
    with _on_device(dev):
        if dgp is not None or dbp is not None:
            wbuf = _given_ws(ws, dev) if ws is not None else _scratch(lib.tg_workspace_size(TG_WS_NORM_BWD, ref),
                                                                      x.device, None, stream)
            wp, wn = _ws_ptr(wbuf)
        st = lib.tango_norm_backward(ref, x.data_ptr(), gp, dyp, rp, dxp, dgp, dbp, wp, wn, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_norm_backward")
    return dx


# ------------------------------------------------- the model's ends: distillation, sampling

def _distill_params(logits, t_logits, t_ids, loss, temperature, grad, f32s):
    dt, dev = logits.dtype, logits.get_device()
    rows, vocab, pitch = _rows_pitch(logits, "logits", dt, dev)
    k = t_logits.shape[-1]
    if k > _MOST_INT:
        _too_large("t_logits")
    if t_logits.numel() != rows * k or t_ids.shape != t_logits.shape:
        raise ValueError("t_logits and t_ids must hold k entries per row of logits")
    tp = _dense(t_logits, "t_logits", torch.float32, dev)
    ip = _dense(t_ids, "t_ids", torch.int32, dev)
    grad_pitch = 0
    if grad is not None:
        g_rows, g_width, grad_pitch = _rows_pitch(grad, "dlogits", dt, dev)
        if g_rows != rows or g_width != vocab:
            raise ValueError("dlogits must have logits' rows and width")
    ptrs = []
    for name, t, per_row in f32s:
        if t is not None and t.numel() != rows * per_row:
            raise ValueError(f"{name} must hold {per_row} value(s) per row")
        ptrs.append(_optional(t, name, torch.float32, dev))
    return tg_distill_params(rows, vocab, k, temperature, pitch, grad_pitch, _dtype_code(logits)), tp, ip, ptrs, dev


def tango_distill(logits, t_logits, t_ids, loss, *, temperature=1.0, stats=None, stream=None):
    """Per row, T^2 times the divergence of softmax(logits / T) over the vocabulary from a teacher's
    softmax over its top k entries: logits [..., vocab] (rows at one pitch), t_logits float32 and
    t_ids int32 [..., k] (negative ids: absent), loss float32 [...].  stats: float32 [..., 2] or
    None, kept for the backward."""
    p, tp, ip, (lp, sp), dev = _distill_params(logits, t_logits, t_ids, loss, temperature, None,
                                               (("loss", loss, 1), ("stats", stats, 2)))
    with _on_device(dev):
        st = (_lib or load()).tango_distill(ctypes.byref(p), logits.data_ptr(), tp, ip, lp, sp, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_distill")
    return loss


def tango_distill_backward(logits, t_logits, t_ids, dloss, dlogits, *, temperature=1.0, stats=None, loss=None,
                           stream=None):
    """Gradient of sum(dloss * loss) with respect to the logits, into dlogits (which may be logits).
    stats from tango_distill, or None: formed here, and the loss too where it is given."""
    p, tp, ip, (dp, sp, lp), dev = _distill_params(logits, t_logits, t_ids, loss, temperature, dlogits,
                                                   (("dloss", dloss, 1), ("stats", stats, 2), ("loss", loss, 1)))
    with _on_device(dev):
        st = (_lib or load()).tango_distill_backward(ctypes.byref(p), logits.data_ptr(), tp, ip, dp, sp,
                                                     dlogits.data_ptr(), lp, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_distill_backward")
    return dlogits


def tango_sample(logits, uniform, token, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, logprob=None, stream=None):
    """Draws one token per row of logits [..., vocab] (rows at one pitch) with the uniform numbers
    uniform float32 [...] into token int32 [...], and the ln of its probability into logprob float32
    [...].  Each setting is a number, or a tensor of one per row (float32; top_k int32)."""
    dt, dev = logits.dtype, logits.get_device()
    rows, vocab, pitch = _rows_pitch(logits, "logits", dt, dev)
    if rows > _MOST_INT:
        _too_large("logits")
    if not isinstance(top_k, torch.Tensor):
        top_k = min(max(top_k, 0), _MOST_INT)  # (0 and less, and the vocabulary and more: off)
    f32, i32 = torch.float32, torch.int32
    ptrs = []
    for name, t, kind in (("uniform", uniform, f32), ("token", token, i32), ("logprob", logprob, f32)):
        if t is not None and t.numel() != rows:
            raise ValueError(f"{name} must hold one value per row")
        ptrs.append(_optional(t, name, kind, dev))
    scalars, arrays = [], []
    for name, x, kind in (("temperature", temperature, f32), ("top_k", top_k, i32), ("top_p", top_p, f32),
                          ("min_p", min_p, f32)):
        if isinstance(x, torch.Tensor):
            if x.numel() != rows:
                raise ValueError(f"{name} must hold one value per row")
            scalars.append(0)
            arrays.append(_dense(x, name, kind, dev))
        else:
            scalars.append(x)
            arrays.append(None)
    p = tg_sample_params(rows, vocab, pitch, _dtype_code(logits), *scalars, *arrays)
    with _on_device(dev):
        st = (_lib or load()).tango_sample(ctypes.byref(p), logits.data_ptr(), *ptrs, _stream_on(stream, dev))
    if st != TG_OK:
        raise TgError(st, "tango_sample")
    return token
