"""Thin Python binding of libhils.so (the C ABI in include/hils.h).

Argument marshalling only: tensors are checked for device, dtype and contiguity, outputs and the
workspace are allocated with PyTorch, and every step of the computation runs in the library's
CUDA kernels.  There is no CPU path: if the library is missing, importing this module's functions
raises.
"""
import ctypes
import os
import struct
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhils.so")

HILS_F32, HILS_BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
          3: "workspace missing or too small", 4: "CUDA error", 5: "device-side check failed",
          6: "bounded on-chip wait timed out"}


class HilsError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, STATUS.get(status, "?"), status))


class Params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hkv", ctypes.c_int64),
                ("N_q", ctypes.c_int64), ("N_kv", ctypes.c_int64), ("d", ctypes.c_int64),
                ("q_pos0", ctypes.c_int64), ("S", ctypes.c_int32), ("K_top", ctypes.c_int32),
                ("W", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class PrologueParams(ctypes.Structure):
    """hils_prologue_params (include/hils.h)."""
    _fields_ = [("d_model", ctypes.c_int64), ("r", ctypes.c_int32),
                ("rope_base", ctypes.c_double), ("train_len", ctypes.c_double)]


class Rope(ctypes.Structure):
    """hils_rope (include/hils.h): the rotary position code of a model, made by rope()."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("freq", ctypes.c_double * 128)]


_Strides = ctypes.c_int64 * 3


class QkParams(ctypes.Structure):
    """hils_qk_params (include/hils.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "N", "Hq", "Hkv", "d", "pos0")] + [
        (n, _Strides) for n in ("q_str", "k_str", "v_str", "qo_str", "ko_str", "dq_str",
                                "dk_str")] + [
        ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("norm", ctypes.c_int32),
        ("eps", ctypes.c_float)]


class PagedParams(ctypes.Structure):
    """hils_paged_params (include/hils.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "B", "Hq", "Hkv", "d", "n_pages",
                                              "max_pages")] + [
        ("c_str", _Strides), ("page_size", ctypes.c_int32), ("window", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


# every function the header declares, with its ctypes signature
_P = ctypes.POINTER(Params)
_V = ctypes.c_void_p
SIGNATURES = {
    "hils_workspace_size": (ctypes.c_size_t, [_P]),
    "hils_forward": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V, _V, _V, _V, _V, ctypes.c_size_t, _V]),
    "hils_forward_timed": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V, _V, _V, _V, _V,
                                          ctypes.c_size_t, _V, ctypes.POINTER(_V), ctypes.c_int]),
    "hils_forward_phases": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_char_p), ctypes.c_int]),
    "hils_select": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V, ctypes.c_size_t, _V]),
    "hils_select_noalloc": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V]),
    "hils_select_noalloc_max_bytes": (ctypes.c_size_t, []),
    "hils_select_noalloc_status": (ctypes.c_int, [_V, ctypes.POINTER(ctypes.c_int32)]),
    "hils_landmarks": (ctypes.c_int, [_P, _V, _V, _V, _V, _V]),
    "hils_decode_step": (ctypes.c_int, [_P] + [_V] * 13 + [ctypes.c_size_t, _V]),
    "hils_wait_check": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_int, _V, ctypes.c_size_t, _V]),
    "hils_backward_workspace_size": (ctypes.c_size_t, [_P]),
    "hils_qcal_workspace_size": (ctypes.c_size_t, [_P, ctypes.POINTER(PrologueParams)]),
    "hils_qcal_hope": (ctypes.c_int, [_P, ctypes.POINTER(PrologueParams)] + [_V] * 7 +
                       [ctypes.c_size_t, _V]),
    "hils_hope_rotate": (ctypes.c_int, [_P, ctypes.POINTER(PrologueParams), ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _V, _V,
                                        _V]),
    "hils_backward": (ctypes.c_int, [_P] + [_V] * 16 + [ctypes.c_size_t, _V]),
    "hils_rope_init": (ctypes.c_int, [ctypes.POINTER(Rope)] + [ctypes.c_int32] * 3 +
                       [ctypes.c_double] * 5),
    # (parameter structures of these calls: packed bytes or a structure by reference)
    "hils_qk_norm_rope": (ctypes.c_int, [_V] * 10),
    "hils_qk_backward_workspace_size": (ctypes.c_size_t, [_V]),
    "hils_qk_norm_rope_backward": (ctypes.c_int, [_V] * 14 + [ctypes.c_size_t, _V]),
    "hils_paged_workspace_size": (ctypes.c_size_t, [_V]),
    "hils_paged_plan": (ctypes.c_int, [_V] * 13 + [ctypes.c_size_t, _V]),
    "hils_paged_append": (ctypes.c_int, [_V] * 14 + [ctypes.c_size_t, _V]),
    "hils_paged_attn": (ctypes.c_int, [_V] * 10 + [ctypes.c_size_t, _V]),
    "hils_chunk_attn": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V, _V]),
    "hils_fuse": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _V]),
    "hils_workspace_init": (ctypes.c_int, [_V, ctypes.c_size_t, _V]),
    "hils_device_status": (ctypes.c_int, [_V, _V, ctypes.POINTER(ctypes.c_int32)]),
    "hils_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "hils_version": (ctypes.c_char_p, []),
}

_lib = None
_lock = threading.Lock()


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        "libhils.so is not built (%s); run `python -m "
                        "hierarchical_chunk_sparse_scoring_b200.build`" % LIB_PATH)
                l = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    f = getattr(l, name)
                    f.restype = res
                    f.argtypes = args
                _lib = l
    return _lib


def _dtype_code(t):
    if t == torch.float32:
        return HILS_F32
    if t == torch.bfloat16:
        return HILS_BF16
    raise TypeError("HiLS tensors must be float32 or bfloat16, got %s" % t)


def make_params(B, Hq, Hkv, N_q, N_kv, d, *, S, K_top, W, q_pos0=0, dtype=torch.bfloat16,
                scale=0.0):
    return Params(B, Hq, Hkv, N_q, N_kv, d, q_pos0, S, K_top, W, _dtype_code(dtype), float(scale))


def params_for(q, K, *, S, K_top, W, q_pos0=0, scale=0.0):
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = K.shape
    return make_params(B, Hq, Hkv, N_q, N_kv, d, S=S, K_top=K_top, W=W, q_pos0=q_pos0,
                       dtype=q.dtype, scale=scale)


def workspace_size(p):
    return int(lib().hils_workspace_size(ctypes.byref(p)))


def _ptr(t):
    return None if t is None or t.numel() == 0 else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, where):
    if status != 0:
        raise HilsError(status, where)


def _need(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must live on a CUDA device (there is no CPU path)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


_ws_cache = {}


def workspace(p, device, stream=None):
    """A workspace of at least workspace_size(p) bytes for `device`, reused across calls made
    from the same stream."""
    need = workspace_size(p)
    if need == 0:
        # invalid or unsupported parameters: the library call reports which, before any launch
        return torch.empty(0, dtype=torch.uint8, device=device)
    st = stream if stream is not None else torch.cuda.current_stream(device)
    key = (torch.device(device).index, st.cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.empty(need, dtype=torch.uint8, device=device)
        _check(lib().hils_workspace_init(_ptr(buf), buf.numel(), _stream(st)), "hils_workspace_init")
        _ws_cache[key] = buf
    return buf


def forward(q, q_cal, K, V, k_lm, b_lm, *, S, K_top, W, q_pos0=0, scale=0.0, out=None,
            lse=None, idx=None, ws=None, stream=None):
    """The whole HiLS forward (steps 1-4).  Returns (out, lse, idx)."""
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = K.shape
    C = N_kv // S
    dt = q.dtype
    _need(q, "q", dt)
    _need(q_cal, "q_cal", dt, q.shape)
    _need(K, "K", dt)
    _need(V, "V", dt, K.shape)
    _need(k_lm, "k_lm", dt, (B, Hkv, C, d))
    _need(b_lm, "b_lm", torch.float32, (B, Hkv, C))
    p = params_for(q, K, S=S, K_top=K_top, W=W, q_pos0=q_pos0, scale=scale)
    out = torch.empty_like(q) if out is None else _need(out, "out", dt, q.shape)
    if lse is None:
        lse = torch.empty((B, Hq, N_q), dtype=torch.float32, device=q.device)
    if idx is None:
        idx = torch.empty((B, Hkv, N_q, K_top), dtype=torch.int32, device=q.device)
    ws = workspace(p, q.device, stream) if ws is None else ws
    st = lib().hils_forward(ctypes.byref(p), _ptr(q), _ptr(q_cal), _ptr(K), _ptr(V), _ptr(k_lm),
                            _ptr(b_lm), _ptr(out), _ptr(lse), _ptr(idx), _ptr(ws), ws.numel(),
                            _stream(stream))
    _check(st, "hils_forward")
    return out, lse, idx


def select(q_cal, k_lm, b_lm, *, N_kv, Hkv, S, K_top, W, q_pos0=0, scale=0.0, stream=None):
    """Steps 1-2.  Returns (idx [B,Hkv,N_q,K] int32, s_sel [B,Hq,N_q,K] fp32)."""
    B, Hq, N_q, d = q_cal.shape
    _need(q_cal, "q_cal")
    _need(k_lm, "k_lm", q_cal.dtype, (B, Hkv, N_kv // S, d))
    _need(b_lm, "b_lm", torch.float32, (B, Hkv, N_kv // S))
    p = make_params(B, Hq, Hkv, N_q, N_kv, d, S=S, K_top=K_top, W=W, q_pos0=q_pos0,
                    dtype=q_cal.dtype, scale=scale)
    idx = torch.empty((B, Hkv, N_q, K_top), dtype=torch.int32, device=q_cal.device)
    s_sel = torch.empty((B, Hq, N_q, K_top), dtype=torch.float32, device=q_cal.device)
    ws = workspace(p, q_cal.device, stream)
    _check(lib().hils_select(ctypes.byref(p), _ptr(q_cal), _ptr(k_lm), _ptr(b_lm), _ptr(idx),
                             _ptr(s_sel), _ptr(ws), ws.numel(), _stream(stream)), "hils_select")
    return idx, s_sel


def chunk_attn(q, K, V, idx, *, S, K_top, W, q_pos0=0, scale=0.0, stream=None):
    """Step 3.  Returns (unit_o [B,Hq,N_q,K+1,d] fp32, unit_lse [B,Hq,N_q,K+1] fp32)."""
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = K.shape
    _need(q, "q")
    _need(K, "K", q.dtype)
    _need(V, "V", q.dtype, K.shape)
    _need(idx, "idx", torch.int32, (B, Hkv, N_q, K_top))
    p = params_for(q, K, S=S, K_top=K_top, W=W, q_pos0=q_pos0, scale=scale)
    unit_o = torch.empty((B, Hq, N_q, K_top + 1, d), dtype=torch.float32, device=q.device)
    unit_lse = torch.empty((B, Hq, N_q, K_top + 1), dtype=torch.float32, device=q.device)
    _check(lib().hils_chunk_attn(ctypes.byref(p), _ptr(q), _ptr(K), _ptr(V), _ptr(idx),
                                 _ptr(unit_o), _ptr(unit_lse), _stream(stream)), "hils_chunk_attn")
    return unit_o, unit_lse


def fuse(s_sel, unit_o, unit_lse, *, Hkv, N_kv, S, K_top, W, q_pos0=0, dtype=torch.bfloat16,
         stream=None):
    """Step 4.  Returns (out [B,Hq,N_q,d] dtype, lse [B,Hq,N_q] fp32)."""
    B, Hq, N_q, _, d = unit_o.shape
    _need(s_sel, "s_sel", torch.float32, (B, Hq, N_q, K_top))
    _need(unit_o, "unit_o", torch.float32, (B, Hq, N_q, K_top + 1, d))
    _need(unit_lse, "unit_lse", torch.float32, (B, Hq, N_q, K_top + 1))
    p = make_params(B, Hq, Hkv, N_q, N_kv, d, S=S, K_top=K_top, W=W, q_pos0=q_pos0, dtype=dtype)
    out = torch.empty((B, Hq, N_q, d), dtype=dtype, device=unit_o.device)
    lse = torch.empty((B, Hq, N_q), dtype=torch.float32, device=unit_o.device)
    _check(lib().hils_fuse(ctypes.byref(p), _ptr(s_sel), _ptr(unit_o), _ptr(unit_lse), _ptr(out),
                           _ptr(lse), _stream(stream)), "hils_fuse")
    return out, lse


def device_status(ws, stream=None):
    code = ctypes.c_int32(0)
    _check(lib().hils_device_status(_ptr(ws), _stream(stream), ctypes.byref(code)),
           "hils_device_status")
    return int(code.value)


def landmarks(q_lm, K, *, S, scale=0.0, k_lm=None, b_lm=None, stream=None):
    """Landmark construction: q_lm [B,Hkv,C,d] landmark queries, K [B,Hkv,N_kv,d] keys with
    C = N_kv // S.  Returns (k_lm [B,Hkv,C,d] in K's dtype, b_lm [B,Hkv,C] fp32)."""
    B, Hkv, N_kv, d = K.shape
    C = N_kv // S
    _need(K, "K")
    _need(q_lm, "q_lm", K.dtype, (B, Hkv, C, d))
    if k_lm is None:
        k_lm = torch.empty((B, Hkv, C, d), dtype=K.dtype, device=K.device)
    if b_lm is None:
        b_lm = torch.empty((B, Hkv, C), dtype=torch.float32, device=K.device)
    _need(k_lm, "k_lm", K.dtype, (B, Hkv, C, d))
    _need(b_lm, "b_lm", torch.float32, (B, Hkv, C))
    p = make_params(B, Hkv, Hkv, 0, N_kv, d, S=S, K_top=0, W=1, dtype=K.dtype, scale=scale)
    _check(lib().hils_landmarks(ctypes.byref(p), _ptr(q_lm), _ptr(K), _ptr(k_lm), _ptr(b_lm),
                                _stream(stream)), "hils_landmarks")
    return k_lm, b_lm


def decode_step(q, q_cal, k_new, v_new, q_lm_new, K, V, k_lm, b_lm, *, pos, S, K_top, W,
                scale=0.0, out=None, lse=None, idx=None, ws=None, stream=None):
    """One decode step over a cache of capacity K.shape[2]: appends (k_new, v_new) at `pos`,
    builds the landmark of the chunk the token completes (q_lm_new, may be None otherwise) and
    runs the forward for the query at `pos`.  Returns (out, lse, idx)."""
    B, Hq, N_q, d = q.shape
    _, Hkv, N_cap, _ = K.shape
    p = make_params(B, Hq, Hkv, N_q, N_cap, d, S=S, K_top=K_top, W=W, q_pos0=pos,
                    dtype=q.dtype, scale=scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N_q), dtype=torch.float32, device=q.device)
    if idx is None:
        idx = torch.empty((B, Hkv, N_q, K_top), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = workspace(p, q.device, stream)
    _check(lib().hils_decode_step(ctypes.byref(p), _ptr(q), _ptr(q_cal), _ptr(k_new),
                                  _ptr(v_new), _ptr(q_lm_new) if q_lm_new is not None else None,
                                  _ptr(K), _ptr(V), _ptr(k_lm), _ptr(b_lm), _ptr(out), _ptr(lse),
                                  _ptr(idx), _ptr(ws), ws.numel(), _stream(stream)),
           "hils_decode_step")
    return out, lse, idx


def qcal_hope(q, hidden, W_down, W_up, *, rope_base, train_len, q_pos0=0, q_out=None,
              q_cal_out=None, ws=None, stream=None):
    """hils_qcal_hope: (HoPE(q), HoPE(q + W_up W_down hidden)) for query i at q_pos0 + i.
    q [B,Hq,N_q,d] and W_up [Hq,d,r] in the model dtype; hidden [B,N_q,d_model] and W_down
    [Hq,r,d_model] bf16 (W_down / W_up may be None for r = 0)."""
    B, Hq, N_q, d = q.shape
    _need(q, "q")
    r = 0 if W_down is None else W_down.shape[1]
    d_model = 0 if hidden is None else hidden.shape[2]
    if r > 0:
        _need(hidden, "hidden", torch.bfloat16, (B, N_q, d_model))
        _need(W_down, "W_down", torch.bfloat16, (Hq, r, d_model))
        _need(W_up, "W_up", q.dtype, (Hq, d, r))
    p = make_params(B, Hq, Hq, N_q, max(N_q + q_pos0, 1), d, S=1, K_top=0, W=1, q_pos0=q_pos0,
                    dtype=q.dtype)
    c = PrologueParams(d_model, r, float(rope_base), float(train_len))
    if q_out is None:
        q_out = torch.empty_like(q)
    if q_cal_out is None:
        q_cal_out = torch.empty_like(q)
    if ws is None:
        need = int(lib().hils_qcal_workspace_size(ctypes.byref(p), ctypes.byref(c)))
        ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib().hils_qcal_hope(ctypes.byref(p), ctypes.byref(c), _ptr(q), _ptr(hidden),
                                _ptr(W_down), _ptr(W_up), _ptr(q_out), _ptr(q_cal_out), _ptr(ws),
                                ws.numel(), _stream(stream)), "hils_qcal_hope")
    return q_out, q_cal_out


def hope_rotate(x, *, rope_base, train_len, pos0=0, out=None, stream=None):
    """hils_hope_rotate: HoPE of x [B,H,N,d], token n at position pos0 + n."""
    B, H, N, d = x.shape
    _need(x, "x")
    p = make_params(1, 1, 1, 1, 1, d, S=1, K_top=0, W=1, dtype=x.dtype)
    c = PrologueParams(0, 0, float(rope_base), float(train_len))
    if out is None:
        out = torch.empty_like(x)
    _check(lib().hils_hope_rotate(ctypes.byref(p), ctypes.byref(c), B, H, N, pos0, _ptr(x),
                                  _ptr(out), _stream(stream)), "hils_hope_rotate")
    return out


def backward_workspace(p, device):
    need = int(lib().hils_backward_workspace_size(ctypes.byref(p)))
    if need == 0:
        return None   # invalid or unsupported: hils_backward says which
    return torch.empty(need, dtype=torch.uint8, device=device)


def backward(q, q_cal, K, V, k_lm, b_lm, idx, dout, dlse=None, *, S, K_top, W, q_pos0=0,
             scale=0.0, ws=None, out=None, stream=None):
    """hils_backward: gradients of sum(dout * out) + sum(dlse * lse) with the selection `idx`
    held fixed.  Returns a dict of fp32 tensors dq, dq_cal, dK, dV, dk_lm, db_lm."""
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = K.shape
    C = N_kv // S
    _need(q, "q")
    _need(q_cal, "q_cal", q.dtype, q.shape)
    _need(K, "K", q.dtype)
    _need(V, "V", q.dtype, K.shape)
    _need(k_lm, "k_lm", q.dtype, (B, Hkv, C, d))
    _need(b_lm, "b_lm", torch.float32, (B, Hkv, C))
    _need(idx, "idx", torch.int32, (B, Hkv, N_q, K_top))
    _need(dout, "dout", q.dtype, q.shape)
    if dlse is not None:
        _need(dlse, "dlse", torch.float32, (B, Hq, N_q))
    p = make_params(B, Hq, Hkv, N_q, N_kv, d, S=S, K_top=K_top, W=W, q_pos0=q_pos0,
                    dtype=q.dtype, scale=scale)
    if ws is None:
        ws = backward_workspace(p, q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    g = out if out is not None else {
        "dq": torch.empty(q.shape, **f32), "dq_cal": torch.empty(q.shape, **f32),
        "dK": torch.empty(K.shape, **f32), "dV": torch.empty(K.shape, **f32),
        "dk_lm": torch.empty(k_lm.shape, **f32), "db_lm": torch.empty(b_lm.shape, **f32)}
    _check(lib().hils_backward(ctypes.byref(p), _ptr(q), _ptr(q_cal), _ptr(K), _ptr(V),
                               _ptr(k_lm), _ptr(b_lm), _ptr(idx), _ptr(dout), _ptr(dlse),
                               _ptr(g["dq"]), _ptr(g["dq_cal"]), _ptr(g["dK"]), _ptr(g["dV"]),
                               _ptr(g["dk_lm"]), _ptr(g["db_lm"]), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(stream)),
           "hils_backward")
    return g


def select_noalloc(q_cal, k_lm, b_lm, *, N_kv, Hkv, S, K_top, W, q_pos0=0, scale=0.0,
                   stream=None):
    """hils_select_noalloc: steps 1-2 with the library's fixed scratch array (no workspace).
    Returns (idx, s_sel)."""
    B, Hq, N_q, d = q_cal.shape
    p = make_params(B, Hq, Hkv, N_q, N_kv, d, S=S, K_top=K_top, W=W, q_pos0=q_pos0,
                    dtype=q_cal.dtype, scale=scale)
    idx = torch.empty((B, Hkv, N_q, K_top), dtype=torch.int32, device=q_cal.device)
    s_sel = torch.empty((B, Hq, N_q, K_top), dtype=torch.float32, device=q_cal.device)
    _check(lib().hils_select_noalloc(ctypes.byref(p), _ptr(q_cal), _ptr(k_lm), _ptr(b_lm),
                                     _ptr(idx), _ptr(s_sel), _stream(stream)),
           "hils_select_noalloc")
    return idx, s_sel


def select_noalloc_status(stream=None):
    """Reads and clears this device's hils_select_noalloc status word."""
    code = ctypes.c_int32(0)
    _check(lib().hils_select_noalloc_status(_stream(stream), ctypes.byref(code)),
           "hils_select_noalloc_status")
    return int(code.value)


def wait_check(polls, complete, ws, stream=None):
    """hils_wait_check: one bounded mbarrier wait on the device (see include/hils.h)."""
    _check(lib().hils_wait_check(int(polls), int(bool(complete)), _ptr(ws), ws.numel(),
                                 _stream(stream)), "hils_wait_check")


# ------------------------------------------------- norms, rotary positions and the paged cache

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "hope": 4}


def rope(rot_dim, *, layout="half", scaling="plain", base=10000.0, factor=1.0, train_len=0.0,
         beta_fast=32.0, beta_slow=1.0, freq=None, mscale=None):
    """The rotary position code of a model (hils_rope_init): pairs of the first rot_dim
    dimensions, "half" or "interleaved", under the scaling rule "plain", "linear", "ntk", "yarn"
    or "hope".  `freq` (rot_dim / 2 radians per position) and `mscale` replace the rule's.  (The
    ramp of "yarn" runs over the turns a pair makes in the trained length, as in the paper; a
    checkpoint whose ramp runs over the pair's index needs its `freq`.)"""
    if layout not in _LAYOUTS or scaling not in _SCALINGS:
        raise ValueError("layout is one of %s, scaling one of %s" %
                         (sorted(_LAYOUTS), sorted(_SCALINGS)))
    r = Rope()
    _check(lib().hils_rope_init(ctypes.byref(r), rot_dim, _LAYOUTS[layout], _SCALINGS[scaling],
                                base, factor, train_len, beta_fast, beta_slow), "hils_rope_init")
    if freq is not None:
        if len(freq) != rot_dim // 2:
            raise ValueError("freq has %d entries, expected %d" % (len(freq), rot_dim // 2))
        r.freq[:rot_dim // 2] = [float(f) for f in freq]
    if mscale is not None:
        r.mscale = float(mscale)
    return r


# hils_qk_params and hils_paged_params, packed: these calls are made once per layer and step of a
# serving loop, where building a ctypes structure field by field would cost as much as the launch
_QK = struct.Struct("<27q3if")
_PAGED = struct.Struct("<10q3if")
assert _QK.size == ctypes.sizeof(QkParams) and _PAGED.size == ctypes.sizeof(PagedParams)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _run(device, stream, used, go):
    """go(stream handle) with `device` current and outputs and workspaces allocated on `stream`
    (default: the device's current stream); the caller's tensors `used` are kept from reuse until
    the work given to `stream` is done."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return go(_raw_stream(device.index))
        with torch.cuda.device(device):
            return go(_raw_stream(device.index))
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        for u in used:
            if u is not None:
                u.record_stream(stream)
        return go(stream.cuda_stream)


def _addr(t):
    return None if t is None else t.data_ptr()     # (of an empty tensor: 0)


def _refuse(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must live on the CUDA device %s (there is no CPU path)" %
                         (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    raise ValueError("%s must be contiguous in its last dimension" % name)


def _rows(t, name, dtype, shape, device):
    """Strides of a tensor [..., d] whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or \
            t.device != device:
        _refuse(t, name, dtype, shape, device)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel():
        _refuse(t, name, dtype, shape, device)
    return st


def _out_rows(t, name, dtype, shape, device):
    """The same of an output: no two of its rows overlap."""
    st = _rows(t, name, dtype, shape, device)
    if not t.is_contiguous() and t.numel():
        span = shape[-1]
        for step, n in sorted((a, b) for a, b in zip(st[:-1], shape[:-1]) if b > 1):
            if step < span:      # (from the innermost stride out: past all the ones inside)
                raise ValueError("rows of %s overlap" % name)
            span = step * n
    return st


def _same_strides(a, b, shape):
    if a != b and any(x != y for x, y, n in zip(a, b, shape) if n > 1):
        raise ValueError("K and V must have the same strides")


def _ints(t, name, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.shape != shape or \
            t.device != device or not t.is_contiguous():
        _refuse(t, name, torch.int32, shape, device)


_NONE = (0, 0, 0, 0)


def _qk_setup(q, k, w_q, w_k, pos):
    """Checks q [B,Hq,N,d], k [B,Hkv,N,d] (either may be None) and what goes with them."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if not x.is_cuda:
        raise ValueError("tensors must live on a CUDA device (there is no CPU path)")
    dev, dt = x.device, x.dtype
    B, Hq, N, d = x.shape
    Hkv = 0
    sq = sk = _NONE
    if q is not None:
        sq = _rows(q, "q", dt, (B, Hq, N, d), dev)
    else:
        Hq = 0
    if k is not None:
        Hkv = k.shape[1]
        sk = _rows(k, "k", dt, (B, Hkv, N, d), dev)
    if w_q is not None:
        _rows(w_q, "w_q", dt, (d,), dev)
    if w_k is not None:
        _rows(w_k, "w_k", dt, (d,), dev)
    if pos is not None:
        _ints(pos, "pos", (B, N), dev)
    return dev, dt, (B, N, Hq, Hkv, d), sq[:3], sk[:3]


def _contiguous_like(x, dtype=None):
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def qk_norm_rope(q, k, w_q, w_k, rope, *, pos=None, pos0=0, eps=1e-6, norm=True, q_out=None,
                 k_out=None, stream=None):
    """hils_qk_norm_rope: RMS norm (weights w_q, w_k [d] or None) and rotation of q [B,Hq,N,d] and
    k [B,Hkv,N,d] (either may be None) at positions pos [B,N] int32 or pos0 + n.  Any strides over
    a contiguous head dim; outputs default to contiguous tensors, q_out may be q.  norm=False
    only rotates.  Returns (q_out, k_out)."""
    dev, dt, dims, sq, sk = _qk_setup(q, k, w_q, w_k, pos)

    def go(st):
        qo = ko = None
        so = sko = _NONE
        if q is not None:
            qo = _contiguous_like(q) if q_out is None else q_out
            so = _out_rows(qo, "q_out", dt, q.shape, dev)
        if k is not None:
            ko = _contiguous_like(k) if k_out is None else k_out
            sko = _out_rows(ko, "k_out", dt, k.shape, dev)
        code = _dtype_code(dt)
        p = _QK.pack(*dims, pos0, *sq, *sk, 0, 0, 0, *so[:3], *sko[:3], 0, 0, 0, 0, 0, 0, code,
                     code, int(bool(norm)), eps)
        _check(lib().hils_qk_norm_rope(p, ctypes.byref(rope), _addr(q), _addr(k), _addr(w_q),
                                       _addr(w_k), _addr(pos), _addr(qo), _addr(ko), st),
               "hils_qk_norm_rope")
        return qo, ko

    return _run(dev, stream, (q, k, w_q, w_k, pos, q_out, k_out), go)


def qk_norm_rope_backward(q, k, w_q, w_k, dq_out, dk_out, rope, *, pos=None, pos0=0, eps=1e-6,
                          norm=True, dq=None, dk=None, stream=None):
    """hils_qk_norm_rope_backward: the gradients of qk_norm_rope's inputs from those of its
    outputs (fp32, as backward() returns them, or q's dtype; any strides).  Returns a dict of dq,
    dk (in the gradients' dtype; dq may be dq_out) and dw_q, dw_k (fp32 [d], None where there is
    no weight)."""
    dev, dt, dims, sq, sk = _qk_setup(q, k, w_q, w_k, pos)
    for x, dy, n in ((q, dq_out, "dq_out"), (k, dk_out, "dk_out")):
        if x is not None and not isinstance(dy, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % n)
    gt = (dq_out if q is not None else dk_out).dtype

    def go(st):
        gq = gk = None
        sgq = sgk = sdq = sdk = _NONE
        if q is not None:
            sgq = _rows(dq_out, "dq_out", gt, q.shape, dev)
            gq = _contiguous_like(q, gt) if dq is None else dq
            sdq = _out_rows(gq, "dq", gt, q.shape, dev)
        if k is not None:
            sgk = _rows(dk_out, "dk_out", gt, k.shape, dev)
            gk = _contiguous_like(k, gt) if dk is None else dk
            sdk = _out_rows(gk, "dk", gt, k.shape, dev)
        p = _QK.pack(*dims, pos0, *sq, *sk, 0, 0, 0, *sgq[:3], *sgk[:3], *sdq[:3], *sdk[:3],
                     _dtype_code(dt), _dtype_code(gt), int(bool(norm)), eps)
        dw_q = dw_k = ws = None
        need = 0
        if w_q is not None or w_k is not None:
            need = lib().hils_qk_backward_workspace_size(p)
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            if w_q is not None:
                dw_q = _contiguous_like(w_q, torch.float32)
            if w_k is not None:
                dw_k = _contiguous_like(w_k, torch.float32)
        _check(lib().hils_qk_norm_rope_backward(
            p, ctypes.byref(rope), _addr(q), _addr(k), _addr(w_q), _addr(w_k), _addr(pos),
            _addr(dq_out) if q is not None else None, _addr(dk_out) if k is not None else None,
            _addr(gq), _addr(gk), _addr(dw_q), _addr(dw_k), _addr(ws), need, st),
            "hils_qk_norm_rope_backward")
        return {"dq": gq, "dk": gk, "dw_q": dw_q, "dw_k": dw_k}

    return _run(dev, stream, (q, k, w_q, w_k, pos, dq_out, dk_out, dq, dk), go)


def paged_workspace(q=None, K=None, *, device=None, stream=None):
    """A workspace for the paged calls (its status word, read with device_status, zeroed): of any
    size for plan and append, with q [T,Hq,d] and K for attention of their heads too.  Calls that
    overlap on the GPU (streams, replayed graphs) need one each."""
    n = 256
    if q is not None:
        c = PagedParams(T=0, B=0, Hq=q.shape[1], Hkv=K.shape[1], d=q.shape[2], page_size=1)
        n = int(lib().hils_paged_workspace_size(ctypes.byref(c)))
        device = q.device
    device = torch.device(device)
    if device.index is None:
        device = torch.device(device.type, torch.cuda.current_device())

    def go(st):
        buf = torch.empty(n, dtype=torch.uint8, device=device)
        _check(lib().hils_workspace_init(_addr(buf), n, st), "hils_workspace_init")
        return buf

    return _run(device, stream, (), go)


# workspaces of the paged calls made without one: (device index, stream handle) -> workspace
_paged_ws = {}


def _workspace_of(ws, device, n, st):
    """The caller's workspace, or the one kept for such calls on this device and stream `st`."""
    if ws is not None:
        if ws.device != device or ws.dtype != torch.uint8 or not ws.is_contiguous():
            _refuse(ws, "ws", torch.uint8, ws.shape, device)
        return ws
    n = max(n, 256)
    if torch.cuda.is_current_stream_capturing():   # a graph may run beside this stream's calls
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:256].zero_()
        return ws
    ws = _paged_ws.get((device.index, st))
    if ws is None or ws.numel() < n:
        new = torch.empty(n, dtype=torch.uint8, device=device)
        if ws is None:
            _check(lib().hils_workspace_init(_addr(new), n, st), "hils_workspace_init")
        else:
            new[:256].copy_(ws[:256])              # what is recorded so far
        _paged_ws[device.index, st] = ws = new
    return ws


def paged_status(stream=None):
    """Reads and clears what the paged calls made without `ws` on this stream (default: the current
    one of the current device) recorded: 0, or 5 if a length, page, slot or position was refused.
    A call captured in a graph without `ws` has a workspace that nothing reads: give it one."""
    if stream is None:
        stream = torch.cuda.current_stream()
    ws = _paged_ws.get((stream.device.index, stream.cuda_stream))
    if ws is None:
        return 0
    with torch.cuda.device(stream.device):
        return device_status(ws, stream)


def paged_plan(kv_len, new_len, block_table, free_pages, n_free, *, page_size, T_cap,
               kv_len_out=None, n_free_out=None, ws=None, stream=None):
    """hils_paged_plan: the slots, positions and sequences of a step's new tokens, with the pages
    they need taken from the free stack (free_pages [n_pages], n_free [1]) and entered in
    block_table [B,max_pages] (in place).  T_cap bounds the tokens.  kv_len_out and n_free_out may
    be kv_len and n_free.  Returns a dict: slot, pos, seq [T_cap], cu [B+1], kv_len [B],
    n_free [1], all int32.  Refused sequences and bad pages are recorded in ws (device_status), or,
    without it, for paged_status."""
    B, M = block_table.shape
    P = free_pages.numel()
    dev = block_table.device
    if not block_table.is_cuda:
        _refuse(block_table, "block_table", torch.int32, (B, M), dev)
    _ints(block_table, "block_table", (B, M), dev)
    _ints(kv_len, "kv_len", (B,), dev)
    _ints(new_len, "new_len", (B,), dev)
    _ints(free_pages, "free_pages", (P,), dev)
    _ints(n_free, "n_free", (1,), dev)
    if kv_len_out is not None:
        _ints(kv_len_out, "kv_len_out", (B,), dev)
    if n_free_out is not None:
        _ints(n_free_out, "n_free_out", (1,), dev)
    if T_cap < 0:
        raise ValueError("T_cap must not be negative")

    def go(st):
        # (one allocation: these live and die together)
        slot, pos, seq, cu, kv, nf = block_table.new_empty(3 * T_cap + 2 * B + 2).split_with_sizes(
            [T_cap, T_cap, T_cap, B + 1, B, 1])
        if kv_len_out is not None:
            kv = kv_len_out
        if n_free_out is not None:
            nf = n_free_out
        w = _workspace_of(ws, dev, 256, st)
        p = _PAGED.pack(T_cap, B, 0, 0, 0, P, M, 0, 0, 0, page_size, 0, 0, 0.0)
        _check(lib().hils_paged_plan(p, _addr(kv_len), _addr(new_len), _addr(block_table),
                                     _addr(free_pages), _addr(n_free), _addr(kv), _addr(nf),
                                     _addr(cu), _addr(slot), _addr(pos), _addr(seq), _addr(w),
                                     w.numel(), st), "hils_paged_plan")
        return {"slot": slot, "pos": pos, "seq": seq, "cu": cu, "kv_len": kv, "n_free": nf}

    return _run(dev, stream, (kv_len, new_len, block_table, free_pages, n_free, kv_len_out,
                              n_free_out, ws), go)


def paged_append(q, k, v, w_q, w_k, rope, K, V, pos, slot, *, eps=1e-6, norm=True, q_out=None,
                 ws=None, stream=None):
    """hils_paged_append: qk_norm_rope of a step's tokens q [T,Hq,d], k, v [T,Hkv,d] (any strides)
    at pos [T], keys and values written to slot [T] of the pools K, V [n_pages,Hkv,page_size,d]
    (any strides; a [n_pages,page_size,Hkv,d] pool as its transpose).  Returns q_out, whose
    padding rows (slot < 0) are left as they were (zero where it is allocated here).  Slots past
    the pool are recorded in ws (device_status), or, without it, for paged_status."""
    if not q.is_cuda:
        raise ValueError("tensors must live on a CUDA device (there is no CPU path)")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    P, _, ps, _ = K.shape
    dev, dt = q.device, q.dtype
    sq = _rows(q, "q", dt, (T, Hq, d), dev)
    sk = _rows(k, "k", dt, (T, Hkv, d), dev)
    sv = _rows(v, "v", dt, (T, Hkv, d), dev)
    for w, n in ((w_q, "w_q"), (w_k, "w_k")):
        if w is not None:
            _rows(w, n, dt, (d,), dev)
    sc = _out_rows(K, "K", dt, (P, Hkv, ps, d), dev)
    _same_strides(sc, _out_rows(V, "V", dt, (P, Hkv, ps, d), dev), K.shape)
    _ints(pos, "pos", (T,), dev)
    _ints(slot, "slot", (T,), dev)

    def go(st):
        out = torch.zeros_like(q, memory_format=torch.contiguous_format) if q_out is None \
            else q_out
        so = _out_rows(out, "q_out", dt, (T, Hq, d), dev)
        w = _workspace_of(ws, dev, 256, st)
        code = _dtype_code(dt)
        p = _QK.pack(1, T, Hq, Hkv, d, 0, 0, sq[1], sq[0], 0, sk[1], sk[0], 0, sv[1], sv[0], 0,
                     so[1], so[0], 0, 0, 0, 0, 0, 0, 0, 0, 0, code, code, int(bool(norm)), eps)
        c = _PAGED.pack(T, 0, Hq, Hkv, d, P, 0, *sc[:3], ps, 0, code, 0.0)
        _check(lib().hils_paged_append(p, ctypes.byref(rope), c, _addr(q), _addr(k), _addr(v),
                                       _addr(w_q), _addr(w_k), _addr(pos), _addr(slot),
                                       _addr(out), _addr(K), _addr(V), _addr(w), w.numel(), st),
               "hils_paged_append")
        return out

    return _run(dev, stream, (q, k, v, w_q, w_k, K, V, pos, slot, q_out, ws), go)


def paged_attn(q, K, V, block_table, pos, *, seq=None, window=0, scale=0.0, out=None, lse=None,
               ws=None, stream=None):
    """hils_paged_attn: row t of q [T,Hq,d] attends to tokens 0 .. pos[t] (the last `window` of
    them, if given) of sequence seq[t] (default t) in the pools K, V [n_pages,Hkv,page_size,d]
    (any strides; d = 64 or 128, at most 16 heads per KV head) through block_table [B,max_pages].
    Returns (out [T,Hq,d], lse [T,Hq] fp32); padding rows (seq < 0) are left as they were (zero
    where `out` is allocated here).  Bad positions, sequences and pages are recorded in ws
    (device_status), or, without it, for paged_status."""
    if not q.is_cuda:
        raise ValueError("tensors must live on a CUDA device (there is no CPU path)")
    T, Hq, d = q.shape
    P, Hkv, ps, _ = K.shape
    B, M = block_table.shape
    dev, dt = q.device, q.dtype
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    sc = _rows(K, "K", dt, (P, Hkv, ps, d), dev)
    _same_strides(sc, _rows(V, "V", dt, (P, Hkv, ps, d), dev), K.shape)
    _ints(block_table, "block_table", (B, M), dev)
    _ints(pos, "pos", (T,), dev)
    if seq is not None:
        _ints(seq, "seq", (T,), dev)
    if out is not None and not _need(out, "out", dt, (T, Hq, d)).device == dev:
        raise ValueError("out must live on %s" % dev)
    if lse is not None and not _need(lse, "lse", torch.float32, (T, Hq)).device == dev:
        raise ValueError("lse must live on %s" % dev)

    def go(st):
        o, z = out, lse
        if o is None:
            o = torch.empty_like(q) if seq is None else torch.zeros_like(q)
        if z is None:
            z = q.new_empty((T, Hq), dtype=torch.float32) if seq is None else \
                q.new_zeros((T, Hq), dtype=torch.float32)
        c = _PAGED.pack(T, B, Hq, Hkv, d, P, M, *sc[:3], ps, window, _dtype_code(dt), scale)
        w = _workspace_of(ws, dev, 0 if ws is not None else lib().hils_paged_workspace_size(c), st)
        _check(lib().hils_paged_attn(c, _addr(q), _addr(K), _addr(V), _addr(block_table),
                                     _addr(seq), _addr(pos), _addr(o), _addr(z), _addr(w),
                                     w.numel(), st), "hils_paged_attn")
        return o, z

    return _run(dev, stream, (q, K, V, block_table, pos, seq, out, lse, ws), go)


def version():
    return lib().hils_version().decode()


def phases(p):
    """Names of the kernels hils_forward launches for params p, in launch order."""
    n = lib().hils_forward_phases(ctypes.byref(p), None, 0)
    if n < 0:
        raise HilsError(1, "hils_forward_phases")
    arr = (ctypes.c_char_p * max(n, 1))()
    lib().hils_forward_phases(ctypes.byref(p), arr, n)
    return [arr[i].decode() for i in range(n)]


def forward_raw(p, q, q_cal, K, V, k_lm, b_lm, out, lse, idx, ws, stream=None, events=None):
    """hils_forward on preallocated tensors (no Python-side checks).  `events`: torch.cuda.Event
    objects already recorded once (so their CUDA handles exist); the library records them before
    the first kernel and after each kernel."""
    if events is None:
        st = lib().hils_forward(ctypes.byref(p), _ptr(q), _ptr(q_cal), _ptr(K), _ptr(V),
                                _ptr(k_lm), _ptr(b_lm), _ptr(out), _ptr(lse), _ptr(idx),
                                _ptr(ws), ws.numel(), _stream(stream))
    else:
        handles = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        st = lib().hils_forward_timed(ctypes.byref(p), _ptr(q), _ptr(q_cal), _ptr(K), _ptr(V),
                                      _ptr(k_lm), _ptr(b_lm), _ptr(out), _ptr(lse), _ptr(idx),
                                      _ptr(ws), ws.numel(), _stream(stream), handles,
                                      len(events))
    _check(st, "hils_forward")
