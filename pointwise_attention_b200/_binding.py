"""ctypes binding of libhstu (include/hstu.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
only checks tensor placement, builds the ``hstu_problem_t`` struct, allocates
outputs and workspace with torch (device memory is plumbing) and forwards
raw pointers.  There is no fallback: if libhstu.so is missing, or a tensor is
not on a CUDA device, the call raises.

``stream=`` takes a torch.cuda.Stream: the call runs on it, and what it
allocates or clears belongs to it.  The inputs have to be ready there; the
caller's stream waits for it before it reads the outputs.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# HSTU_DEBUG_BOUNDS=1 in the environment selects the build with device-side
# index checks (python -m pointwise_attention_b200.build --debug-bounds).
LIB_PATH = os.path.join(_HERE, "libhstu_debug.so" if os.environ.get("HSTU_DEBUG_BOUNDS") == "1"
                        else "libhstu.so")

HSTU_OK, HSTU_ERR_INVALID_ARG, HSTU_ERR_UNSUPPORTED = 0, 1, 2
HSTU_ERR_CUDA, HSTU_ERR_TIMEOUT, HSTU_ERR_WORKSPACE, HSTU_ERR_BOUNDS = 3, 4, 5, 6
HSTU_F32, HSTU_BF16 = 0, 1

EXPORTED = ("hstu_attn_workspace_size", "hstu_attn_fwd", "hstu_attn_bwd", "hstu_attn_check",
            "hstu_status_string", "hstu_time_bucket_thresholds", "hstu_selftest_wait_timeout",
            "hstu_attn_bwd_noalloc", "hstu_uvqk_fwd", "hstu_out_fwd", "hstu_cand_workspace_size",
            "hstu_cand_fwd", "hstu_rmsnorm_fwd", "hstu_rmsnorm_bwd",
            "hstu_rmsnorm_bwd_workspace_size", "hstu_quant_rows", "hstu_uvqk_fp8_fwd",
            "hstu_rab_bucket_fwd", "hstu_rab_bucket_bwd", "hstu_pos_bucket_thresholds",
            "hstu_kv4_pack", "hstu_kv4_unpack", "hstu_cand_kv4_workspace_size",
            "hstu_cand_kv4_fwd")


class HSTUError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s: %s" % (what, status_string(code)))


class hstu_problem_t(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("batch", ctypes.c_int32),
        ("total_tokens", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("offsets", ctypes.c_void_p),
        ("offsets_host", ctypes.c_void_p),
        ("timestamps", ctypes.c_void_p),
        ("rab_pos", ctypes.c_void_p),
        ("rab_pos_len", ctypes.c_int32),
        ("rab_time", ctypes.c_void_p),
        ("num_time_buckets", ctypes.c_int32),
        ("norm_len", ctypes.c_int32),
        ("ln_eps", ctypes.c_float),
        ("ln_weight", ctypes.c_void_p),
        ("ln_bias", ctypes.c_void_p),
    ]


_lib = None


def load_library():
    """Loads libhstu.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libhstu.so is not built (%s); run `python -m "
                           "pointwise_attention_b200.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(hstu_problem_t)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.hstu_attn_workspace_size.argtypes = [P, ctypes.c_int]
    lib.hstu_attn_workspace_size.restype = sz
    lib.hstu_attn_fwd.argtypes = [P] + [vp] * 5 + [vp] * 3 + [vp, sz, vp]
    lib.hstu_attn_fwd.restype = ctypes.c_int
    lib.hstu_attn_bwd.argtypes = [P] + [vp] * 5 + [vp] * 3 + [vp] * 4 + [vp] * 4 + [vp, sz, vp]
    lib.hstu_attn_bwd.restype = ctypes.c_int
    lib.hstu_attn_check.argtypes = [vp, vp]
    lib.hstu_attn_check.restype = ctypes.c_int
    lib.hstu_status_string.argtypes = [ctypes.c_int]
    lib.hstu_status_string.restype = ctypes.c_char_p
    lib.hstu_time_bucket_thresholds.argtypes = [vp, ctypes.c_int32]
    lib.hstu_time_bucket_thresholds.restype = ctypes.c_int32
    lib.hstu_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
    lib.hstu_selftest_wait_timeout.restype = ctypes.c_int
    lib.hstu_attn_bwd_noalloc.argtypes = [P] + [vp] * 5 + [vp] * 3 + [vp] * 4 + [vp] * 4 + [vp]
    lib.hstu_attn_bwd_noalloc.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.hstu_uvqk_fwd.argtypes = [i32] * 6 + [vp] * 7 + [vp, sz, vp]
    lib.hstu_uvqk_fwd.restype = ctypes.c_int
    lib.hstu_out_fwd.argtypes = [i32] * 3 + [vp] * 6 + [ctypes.c_float] + [vp] * 3 + [vp, sz, vp]
    lib.hstu_out_fwd.restype = ctypes.c_int
    lib.hstu_cand_workspace_size.argtypes = [P, i32, i32]
    lib.hstu_cand_workspace_size.restype = sz
    lib.hstu_cand_fwd.argtypes = [P, vp, vp, vp, i32, i32] + [vp] * 6 + [vp, sz, vp]
    lib.hstu_cand_fwd.restype = ctypes.c_int
    f32, it = ctypes.c_float, ctypes.c_int
    lib.hstu_rmsnorm_fwd.argtypes = [it, i32, i32, vp, vp, vp, f32] + [vp] * 6
    lib.hstu_rmsnorm_fwd.restype = it
    lib.hstu_quant_rows.argtypes = [it, i32, i32] + [vp] * 4
    lib.hstu_quant_rows.restype = it
    lib.hstu_rmsnorm_bwd_workspace_size.argtypes = [i32, i32]
    lib.hstu_rmsnorm_bwd_workspace_size.restype = sz
    lib.hstu_rmsnorm_bwd.argtypes = [it, i32, i32] + [vp] * 8 + [sz, vp]
    lib.hstu_rmsnorm_bwd.restype = it
    lib.hstu_uvqk_fp8_fwd.argtypes = [i32] * 6 + [vp] * 10 + [sz, vp]
    lib.hstu_uvqk_fp8_fwd.restype = it
    for f in (lib.hstu_rab_bucket_fwd, lib.hstu_rab_bucket_bwd):
        f.argtypes = [i32, i32, i32] + [vp] * 4
        f.restype = it
    lib.hstu_pos_bucket_thresholds.argtypes = [vp, i32, i32, i32]
    lib.hstu_pos_bucket_thresholds.restype = i32
    lib.hstu_kv4_pack.argtypes = [i32, i32, vp, vp, vp, i32] + [vp] * 5 + [sz, vp]
    lib.hstu_kv4_pack.restype = it
    lib.hstu_kv4_unpack.argtypes = [i32, i32] + [vp] * 5 + [i32] + [vp] * 3 + [sz, vp]
    lib.hstu_kv4_unpack.restype = it
    lib.hstu_cand_kv4_workspace_size.argtypes = [i32] * 5
    lib.hstu_cand_kv4_workspace_size.restype = sz
    lib.hstu_cand_kv4_fwd.argtypes = [P] + [vp] * 4 + [i32, vp, vp, i32, i32] + [vp] * 7 + [sz, vp]
    lib.hstu_cand_kv4_fwd.restype = it
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().hstu_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor (the library runs on the GPU only)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    return t


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_problem(q, v, offsets, max_seq_len, timestamps=None, rab_pos=None, rab_time=None,
                 norm_len=0, eps=1e-5, offsets_host=None, ln_weight=None, ln_bias=None):
    """hstu_problem_t for tensors q [T,H,dqk], v [T,H,dv] and int32 offsets [B+1];
    ln_weight, ln_bias: fp32 [H*dv] LayerNorm affine, or None (ones, zeros)."""
    if q.dtype == torch.bfloat16:
        dt = HSTU_BF16
    elif q.dtype == torch.float32:
        dt = HSTU_F32
    else:
        raise ValueError("q must be bf16 or fp32")
    T, H, dqk = q.shape
    p = hstu_problem_t()
    p.dtype = dt
    p.batch = offsets.numel() - 1
    p.total_tokens = T
    p.max_seq_len = int(max_seq_len)
    p.num_heads = H
    p.d_qk = dqk
    p.d_v = v.shape[-1]
    p.offsets = offsets.data_ptr()
    p.offsets_host = None if offsets_host is None else offsets_host.data_ptr()
    p.timestamps = None if timestamps is None else timestamps.data_ptr()
    p.rab_pos = None if rab_pos is None else rab_pos.data_ptr()
    p.rab_pos_len = 0 if rab_pos is None else (rab_pos.shape[-1] + 1) // 2
    p.rab_time = None if rab_time is None else rab_time.data_ptr()
    p.num_time_buckets = 0 if rab_time is None else rab_time.shape[-1]
    p.norm_len = int(norm_len)
    p.ln_eps = float(eps)
    p.ln_weight = None if ln_weight is None else ln_weight.data_ptr()
    p.ln_bias = None if ln_bias is None else ln_bias.data_ptr()
    return p


def hstu_attn_workspace_size(problem: hstu_problem_t, is_bwd: bool = False) -> int:
    return int(load_library().hstu_attn_workspace_size(ctypes.byref(problem), int(bool(is_bwd))))


def new_workspace(problem: hstu_problem_t, is_bwd: bool, device) -> torch.Tensor:
    n = hstu_attn_workspace_size(problem, is_bwd)
    if n == 0:
        raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_attn_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def hstu_attn_fwd(q, k, v, u, offsets, max_seq_len, *, timestamps=None, rab_pos=None,
                  rab_time=None, norm_len=0, eps=1e-5, ln_weight=None, ln_bias=None,
                  save_for_backward=False, offsets_host=None, y=None, saved=None,
                  workspace=None, stream=None):
    """Forward.  Returns (y, saved) with saved = (o_save, ln_mean, ln_rstd) or None."""
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v), ("u", u)):
        _dev(t, name, q.dtype)
    _dev(offsets, "offsets", torch.int32)
    _dev(timestamps, "timestamps", torch.int64)
    _dev(rab_pos, "rab_pos", torch.float32)
    _dev(rab_time, "rab_time", torch.float32)
    _dev(ln_weight, "ln_weight", torch.float32)
    _dev(ln_bias, "ln_bias", torch.float32)
    T, H, _ = q.shape
    D = H * v.shape[-1]
    p = make_problem(q, v, offsets, max_seq_len, timestamps, rab_pos, rab_time, norm_len, eps,
                     offsets_host, ln_weight, ln_bias)
    new_y, new_saved = y is None, save_for_backward and saved is None
    with _on(q, stream=stream):
        if y is None:
            y = torch.empty((T, D), dtype=q.dtype, device=q.device)
        _dev(y, "y", q.dtype)
        if save_for_backward and saved is None:
            saved = (torch.empty((T, D), dtype=torch.float32, device=q.device),
                     torch.empty((T,), dtype=torch.float32, device=q.device),
                     torch.empty((T,), dtype=torch.float32, device=q.device))
        if not save_for_backward:
            saved = None
        if workspace is None:
            workspace = new_workspace(p, False, q.device)
        o_save, mean, rstd = saved if saved is not None else (None, None, None)
        rc = lib.hstu_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(y),
                               _ptr(o_save), _ptr(mean), _ptr(rstd), _ptr(workspace),
                               workspace.numel(), _stream_of(q, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_attn_fwd")
    _hand_over(stream, y if new_y else None, *(saved if new_saved else ()))
    return y, saved


def hstu_attn_bwd(dy, q, k, v, u, offsets, max_seq_len, saved, *, timestamps=None,
                  rab_pos=None, rab_time=None, norm_len=0, eps=1e-5, ln_weight=None,
                  ln_bias=None, offsets_host=None, need_rab_grads=True, grads=None,
                  workspace=None, stream=None):
    """Backward.  Returns dict dq, dk, dv, du, d_rab_pos, d_rab_time, d_ln_weight,
    d_ln_bias (the table gradients None where the table is absent)."""
    lib = load_library()
    for name, t in (("dy", dy), ("q", q), ("k", k), ("v", v), ("u", u)):
        _dev(t, name, q.dtype)
    _dev(offsets, "offsets", torch.int32)
    o_save, mean, rstd = saved
    for name, t in (("o_save", o_save), ("ln_mean", mean), ("ln_rstd", rstd)):
        _dev(t, name, torch.float32)
    _dev(ln_weight, "ln_weight", torch.float32)
    _dev(ln_bias, "ln_bias", torch.float32)
    p = make_problem(q, v, offsets, max_seq_len, timestamps, rab_pos, rab_time, norm_len, eps,
                     offsets_host, ln_weight, ln_bias)
    new = grads is None
    with _on(q, stream=stream):
        if grads is None:
            grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                         du=torch.empty_like(u),
                         d_rab_pos=(torch.empty_like(rab_pos)
                                    if (rab_pos is not None and need_rab_grads) else None),
                         d_rab_time=(torch.empty_like(rab_time)
                                     if (rab_time is not None and need_rab_grads) else None),
                         d_ln_weight=(torch.empty_like(ln_weight)
                                      if (ln_weight is not None and need_rab_grads) else None),
                         d_ln_bias=(torch.empty_like(ln_bias)
                                    if (ln_bias is not None and need_rab_grads) else None))
        grads.setdefault("d_ln_weight", None)
        grads.setdefault("d_ln_bias", None)
        if workspace is None:
            workspace = new_workspace(p, True, q.device)
        rc = lib.hstu_attn_bwd(ctypes.byref(p), _ptr(dy), _ptr(q), _ptr(k), _ptr(v), _ptr(u),
                               _ptr(o_save), _ptr(mean), _ptr(rstd), _ptr(grads["dq"]),
                               _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["du"]),
                               _ptr(grads["d_rab_pos"]), _ptr(grads["d_rab_time"]),
                               _ptr(grads["d_ln_weight"]), _ptr(grads["d_ln_bias"]),
                               _ptr(workspace), workspace.numel(), _stream_of(q, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_attn_bwd")
    if new:
        _hand_over(stream, *grads.values())
    return grads


def hstu_attn_check(workspace, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status word."""
    return int(load_library().hstu_attn_check(_ptr(workspace), _stream_ptr(stream)))


def hstu_time_bucket_thresholds(num_buckets: int = 128):
    import numpy as np
    out = np.zeros(max(num_buckets - 1, 1), dtype=np.int64)
    n = load_library().hstu_time_bucket_thresholds(out.ctypes.data_as(ctypes.c_void_p),
                                                   int(num_buckets))
    if n < 0:
        raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_time_bucket_thresholds")
    return out[:n]


def hstu_selftest_wait_timeout(workspace, budget_ns: int = 50_000_000, stream=None) -> int:
    """Runs the bounded-wait self-test kernel; returns the launch status."""
    return int(load_library().hstu_selftest_wait_timeout(_ptr(workspace), int(budget_ns),
                                                         _stream_ptr(stream)))


def _status_workspace(device):
    return torch.zeros(256, dtype=torch.uint8, device=device)


def hstu_uvqk_fwd(x, w, num_heads: int, d_qk: int, d_v: int, *, bias=None, act: int = 0,
                  out=None, workspace=None, stream=None):
    """UVQK projection act(x w^T + bias) of x [T, E] by w [H(2dv+2dqk), E] (bf16).

    Returns dict u [T, H*dv], v [T, H, dv], q [T, H, dqk], k [T, H, dqk] (bf16)."""
    lib = load_library()
    _dev(x, "x", torch.bfloat16)
    _dev(w, "w", torch.bfloat16)
    _dev(bias, "bias", torch.float32)
    T, E = x.shape
    H = int(num_heads)
    new = out is None
    with _on(x, stream=stream):
        if out is None:
            out = dict(u=torch.empty((T, H * d_v), dtype=x.dtype, device=x.device),
                       v=torch.empty((T, H, d_v), dtype=x.dtype, device=x.device),
                       q=torch.empty((T, H, d_qk), dtype=x.dtype, device=x.device),
                       k=torch.empty((T, H, d_qk), dtype=x.dtype, device=x.device))
        for n in ("u", "v", "q", "k"):
            _dev(out[n], n, x.dtype)
        if workspace is None:
            workspace = _status_workspace(x.device)
        rc = lib.hstu_uvqk_fwd(int(T), int(E), H, int(d_qk), int(d_v), int(act), _ptr(x), _ptr(w),
                               _ptr(bias), _ptr(out["u"]), _ptr(out["v"]), _ptr(out["q"]),
                               _ptr(out["k"]), _ptr(workspace), workspace.numel(),
                               _stream_of(x, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_uvqk_fwd")
    if new:
        _hand_over(stream, *out.values())
    return out


def hstu_out_fwd(y, w, x, *, bias=None, ln_weight=None, ln_bias=None, eps: float = 1e-5,
                 save_stats: bool = False, z=None, workspace=None, stream=None):
    """Z = LayerNorm(x + y w^T + bias) * ln_weight + ln_bias for y [T, D], w [E, D],
    x [T, E] (bf16).  Returns (z, (mean, rstd) or None)."""
    lib = load_library()
    _dev(y, "y", torch.bfloat16)
    _dev(w, "w", torch.bfloat16)
    _dev(x, "x", torch.bfloat16)
    for n, t in (("bias", bias), ("ln_weight", ln_weight), ("ln_bias", ln_bias)):
        _dev(t, n, torch.float32)
    T, D = y.shape
    E = x.shape[1]
    new = z is None
    with _on(x, stream=stream):
        if z is None:
            z = torch.empty((T, E), dtype=x.dtype, device=x.device)
        _dev(z, "z", x.dtype)
        stats = None
        if save_stats:
            stats = (torch.empty(T, dtype=torch.float32, device=x.device),
                     torch.empty(T, dtype=torch.float32, device=x.device))
        if workspace is None:
            workspace = _status_workspace(x.device)
        mean, rstd = stats if stats is not None else (None, None)
        rc = lib.hstu_out_fwd(int(T), int(E), int(D), _ptr(y), _ptr(w), _ptr(x), _ptr(bias),
                              _ptr(ln_weight), _ptr(ln_bias), float(eps), _ptr(z), _ptr(mean),
                              _ptr(rstd), _ptr(workspace), workspace.numel(), _stream_of(x, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_out_fwd")
    _hand_over(stream, z if new else None, *(stats or ()))
    return z, stats


def hstu_cand_fwd(k_hist, v_hist, offsets, max_seq_len, q, k, v, u, cand_offsets,
                  max_cands: int, *, timestamps=None, cand_timestamps=None, rab_pos=None,
                  rab_time=None, norm_len=0, eps=1e-5, ln_weight=None, ln_bias=None,
                  offsets_host=None, y=None, workspace=None, stream=None):
    """Candidate scoring against cached histories (M-FALCON): every candidate
    of user b attends to b's history (k_hist, v_hist [T_h, H, 128], offsets)
    and to itself.  q, k, v [C, H, 128], u [C, H*128] (bf16); cand_offsets
    int32 [B+1].  Returns y [C, H*128]."""
    lib = load_library()
    for name, t in (("k_hist", k_hist), ("v_hist", v_hist), ("q", q), ("k", k), ("v", v),
                    ("u", u)):
        _dev(t, name, torch.bfloat16)
    _dev(offsets, "offsets", torch.int32)
    _dev(cand_offsets, "cand_offsets", torch.int32)
    _dev(timestamps, "timestamps", torch.int64)
    _dev(cand_timestamps, "cand_timestamps", torch.int64)
    for name, t in (("rab_pos", rab_pos), ("rab_time", rab_time), ("ln_weight", ln_weight),
                    ("ln_bias", ln_bias)):
        _dev(t, name, torch.float32)
    p = make_problem(k_hist, v_hist, offsets, max_seq_len, timestamps, rab_pos, rab_time,
                     norm_len, eps, offsets_host, ln_weight, ln_bias)
    C, H, _ = q.shape
    new = y is None
    with _on(q, stream=stream):
        if y is None:
            y = torch.empty((C, H * v.shape[-1]), dtype=q.dtype, device=q.device)
        _dev(y, "y", q.dtype)
        if workspace is None:
            n = int(lib.hstu_cand_workspace_size(ctypes.byref(p), int(C), int(max_cands)))
            if n == 0:
                raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_cand_workspace_size")
            workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
        rc = lib.hstu_cand_fwd(ctypes.byref(p), _ptr(k_hist), _ptr(v_hist), _ptr(cand_offsets),
                               int(C), int(max_cands), _ptr(cand_timestamps), _ptr(q), _ptr(k),
                               _ptr(v), _ptr(u), _ptr(y), _ptr(workspace), workspace.numel(),
                               _stream_of(q, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_cand_fwd")
    _hand_over(stream, y if new else None)
    return y


_BF16, _F32, _F8, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.float8_e4m3fn,
                                     torch.int32, torch.int64, torch.uint8)
_ROWS = {_BF16: HSTU_BF16, _F32: HSTU_F32}
_STAY = contextlib.nullcontext()


def _rows_dtype(t, name):
    """The library's name of the rows' type; t must be [T, E]."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _ROWS:
        raise ValueError("%s must be a bf16 or fp32 tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be [T, E]" % name)
    return _ROWS[t.dtype]


def _arg(t, name, dtype, *shape):
    """Placement, layout, type and shape of one argument (None passes); its address."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()
            and (not shape or t.shape == shape)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library runs on the GPU only)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))


def _on(ref, *tensors, stream=None):
    """A context in which ref's device and the given stream are current; every
    tensor must be there.  What a call allocates and clears in it (outputs,
    workspace) is then ordered with its kernels, and is not handed out again
    before them."""
    at = ref.get_device()
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError("all tensors must be on one device (%s and %s)" % (ref.device, t.device))
    if stream is not None:
        if stream.device.index != at:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, ref.device))
        return torch.cuda.stream(stream)
    return _STAY if torch._C._cuda_getDevice() == at else torch.cuda.device(at)


def _hand_over(stream, *outputs):
    """Outputs allocated on the given stream, for the caller's: their memory waits
    for what the caller's stream has done with them when they are let go of."""
    if stream is not None:
        mine = torch.cuda.current_stream(stream.device)
        for t in outputs:
            if t is not None and mine != stream:
                t.record_stream(mine)


def _stream_of(ref, stream):
    """The given stream, else the current one of ref's device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(ref.get_device())


def _room(workspace, ref):
    """A workspace's address and bytes (a status word's worth when None)."""
    if workspace is None:
        workspace = _status_workspace(ref.device)
    elif not workspace.is_cuda or workspace.dtype != _U8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor")
    return workspace, workspace.data_ptr(), workspace.numel()


def hstu_rmsnorm_fwd(x, *, residual=None, weight=None, eps: float = 1e-6, quant: bool = False,
                     save_rstd: bool = False, out=None, stream=None):
    """Root-mean-square norm of the rows of x + residual (x [T, E], bf16 or fp32).

    Returns a dict: h = round(x + residual) (None without a residual); y, or with
    quant q8 (e4m3) and scale (fp32 [T]); rstd (fp32 [T], None unless save_rstd).
    ``out`` may hold any of these tensors to write to."""
    lib = load_library()
    dt = _rows_dtype(x, "x")
    T, E = x.shape
    xp = _arg(x, "x", x.dtype)
    rp = _arg(residual, "residual", x.dtype, T, E)
    wp = _arg(weight, "weight", _F32, E)
    h = y = q8 = scale = rstd = None
    hp = yp = qp = sp = np_ = None
    if out is not None:
        h, y, q8, scale, rstd = (out.get(n) for n in ("h", "y", "q8", "scale", "rstd"))
        hp, yp = _arg(h, "h", x.dtype, T, E), _arg(y, "y", x.dtype, T, E)
        qp, sp = _arg(q8, "q8", _F8, T, E), _arg(scale, "scale", _F32, T)
        np_ = _arg(rstd, "rstd", _F32, T)
        _on(x, h, y, q8, scale, rstd)
    given = (h, y, q8, scale, rstd)
    with _on(x, residual, weight, stream=stream):
        if residual is not None and h is None:
            h = torch.empty_like(x)
            hp = h.data_ptr()
        if quant:
            if q8 is None:
                q8 = torch.empty_like(x, dtype=_F8)
                qp = q8.data_ptr()
            if scale is None:
                scale = x.new_empty(T, dtype=_F32)
                sp = scale.data_ptr()
        elif y is None:
            y = torch.empty_like(x)
            yp = y.data_ptr()
        if save_rstd and rstd is None:
            rstd = x.new_empty(T, dtype=_F32)
            np_ = rstd.data_ptr()
        rc = lib.hstu_rmsnorm_fwd(dt, T, E, xp, rp, wp, float(eps), hp, yp, qp, sp, np_,
                                  _stream_of(x, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_rmsnorm_fwd")
    if stream is not None:
        _hand_over(stream, *(t for t, g in zip((h, y, q8, scale, rstd), given) if t is not g))
    return dict(h=h, y=y, q8=q8, scale=scale, rstd=rstd)


def hstu_rmsnorm_bwd(dy, h, rstd, *, weight=None, d_residual=None, need_weight_grad=True,
                     dx=None, workspace=None, stream=None):
    """Backward of hstu_rmsnorm_fwd from its h (x without a residual) and rstd.
    Returns (dx, d_weight fp32 [E] or None); dx is the residual's gradient too."""
    lib = load_library()
    dt = _rows_dtype(dy, "dy")
    T, E = dy.shape
    args = (_arg(dy, "dy", dy.dtype), _arg(h, "h", dy.dtype, T, E), _arg(rstd, "rstd", _F32, T),
            _arg(weight, "weight", _F32, E), _arg(d_residual, "d_residual", dy.dtype, T, E))
    dxp = _arg(dx, "dx", dy.dtype, T, E)
    new = dx is None
    with _on(dy, h, rstd, weight, d_residual, dx, workspace, stream=stream):
        if dx is None:
            dx = torch.empty_like(dy)
            dxp = dx.data_ptr()
        dw, wp, wn = None, None, 0
        if need_weight_grad:
            dw = dy.new_empty(E, dtype=_F32)
            if workspace is None:
                wn = max(lib.hstu_rmsnorm_bwd_workspace_size(T, E), 256)
                workspace = dy.new_empty(wn, dtype=_U8)
                wp = workspace.data_ptr()
            else:
                workspace, wp, wn = _room(workspace, dy)
        rc = lib.hstu_rmsnorm_bwd(dt, T, E, *args, dxp,
                                  None if dw is None else dw.data_ptr(), wp, wn,
                                  _stream_of(dy, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_rmsnorm_bwd")
    _hand_over(stream, dx if new else None, dw)
    return dx, dw


def hstu_quant_rows(x, *, stream=None):
    """Rows of x [T, E] (bf16 or fp32) as e4m3 bytes with one scale each.
    Returns (q8 [T, E] float8_e4m3fn, scale fp32 [T])."""
    lib = load_library()
    dt = _rows_dtype(x, "x")
    T, E = x.shape
    xp = _arg(x, "x", x.dtype)
    with _on(x, stream=stream):
        q8 = torch.empty_like(x, dtype=_F8)
        scale = x.new_empty(T, dtype=_F32)
        rc = lib.hstu_quant_rows(dt, T, E, xp, q8.data_ptr(), scale.data_ptr(),
                                 _stream_of(x, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_quant_rows")
    _hand_over(stream, q8, scale)
    return q8, scale


def hstu_uvqk_fp8_fwd(x8, x_scale, w8, w_scale, num_heads: int, d_qk: int, d_v: int, *, bias=None,
                      act: int = 0, out=None, workspace=None, stream=None):
    """UVQK projection act(x w^T + bias) of 8-bit rows: x8 [T, E], w8 [N, E]
    (float8_e4m3fn) with fp32 scales per row.  Returns the dict of hstu_uvqk_fwd."""
    lib = load_library()
    xp = _arg(x8, "x8", _F8)
    T, E = x8.shape
    H, d_qk, d_v = int(num_heads), int(d_qk), int(d_v)
    N = 2 * H * (d_qk + d_v)
    args = (xp, _arg(x_scale, "x_scale", _F32, T), _arg(w8, "w8", _F8, N, E),
            _arg(w_scale, "w_scale", _F32, N), _arg(bias, "bias", _F32, N))
    shapes = (T, H * d_v), (T, H, d_v), (T, H, d_qk), (T, H, d_qk)
    if out is not None:
        outs = out["u"], out["v"], out["q"], out["k"]
        ptrs = [_arg(t, n, _BF16, *sh) for t, n, sh in zip(outs, "uvqk", shapes)]
        _on(x8, *outs)
    new = out is None
    with _on(x8, x_scale, w8, w_scale, bias, workspace, stream=stream):
        if out is None:
            u = x8.new_empty(shapes[0], dtype=_BF16)
            v = x8.new_empty(shapes[1], dtype=_BF16)
            q = torch.empty_like(v) if d_qk == d_v else x8.new_empty(shapes[2], dtype=_BF16)
            k = torch.empty_like(q)
            out = dict(u=u, v=v, q=q, k=k)
            ptrs = u.data_ptr(), v.data_ptr(), q.data_ptr(), k.data_ptr()
        workspace, wp, wn = _room(workspace, x8)
        rc = lib.hstu_uvqk_fp8_fwd(T, E, H, d_qk, d_v, int(act), *args, *ptrs, wp, wn,
                                   _stream_of(x8, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_uvqk_fp8_fwd")
    if new:
        _hand_over(stream, *out.values())
    return out


def hstu_pos_bucket_thresholds(num_buckets: int, max_exact: int, max_distance: int):
    """int32 CPU tensor [num_buckets - 1]: the smallest distance of each bucket
    from 1 on, exact up to max_exact, then logarithmic up to max_distance."""
    out = torch.zeros(max(int(num_buckets) - 1, 1), dtype=_I32)
    n = load_library().hstu_pos_bucket_thresholds(
        out.data_ptr() if 1 <= num_buckets <= 128 else None, int(num_buckets), int(max_exact),
        int(max_distance))
    if n < 0:
        raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_pos_bucket_thresholds")
    return out[:n]


def _thresholds(thr, nb):
    if (not isinstance(thr, torch.Tensor) or thr.is_cuda or thr.dtype != _I32
            or thr.shape != (nb - 1,) or not thr.is_contiguous()):
        raise ValueError("thresholds must be a contiguous int32 CPU tensor [%d]" % (nb - 1))
    return thr.data_ptr()


def hstu_rab_bucket_fwd(table, length: int, thresholds, *, out=None, stream=None):
    """Position-bias table rab_pos [H, 2 length - 1] (fp32) from table [H, NB] and
    the buckets' thresholds (int32 CPU tensor [NB - 1])."""
    lib = load_library()
    tp = _arg(table, "table", _F32)
    H, NB = table.shape
    thr = _thresholds(thresholds, NB)
    length = int(length)
    if length < 1:
        raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_rab_bucket_fwd")
    new = out is None
    with _on(table, out, stream=stream):
        if out is None:
            out = table.new_empty((H, 2 * length - 1))
            op = out.data_ptr()
        else:
            op = _arg(out, "out", _F32, H, 2 * length - 1)
        rc = lib.hstu_rab_bucket_fwd(H, length, NB, thr, tp, op, _stream_of(table, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_rab_bucket_fwd")
    _hand_over(stream, out if new else None)
    return out


def hstu_rab_bucket_bwd(d_rab_pos, num_buckets: int, thresholds, *, out=None, stream=None):
    """Gradient [H, num_buckets] of hstu_rab_bucket_fwd's table from that of
    rab_pos [H, 2L - 1] (hstu_attn_bwd's d_rab_pos)."""
    lib = load_library()
    gp = _arg(d_rab_pos, "d_rab_pos", _F32)
    H, W = d_rab_pos.shape
    if W % 2 != 1:
        raise ValueError("d_rab_pos must be [H, 2L - 1]")
    NB = int(num_buckets)
    thr = _thresholds(thresholds, NB)
    new = out is None
    with _on(d_rab_pos, out, stream=stream):
        if out is None:
            out = d_rab_pos.new_empty((H, NB))
        rc = lib.hstu_rab_bucket_bwd(H, (W + 1) // 2, NB, thr, gp, _arg(out, "out", _F32, H, NB),
                                     _stream_of(d_rab_pos, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_rab_bucket_bwd")
    _hand_over(stream, out if new else None)
    return out


def hstu_kv4_cache(cache_rows: int, num_heads: int, device):
    """An empty 4-bit cache: (k_codes, k_scales, v_codes, v_scales), codes uint8
    [cache_rows, H, 64], scales bf16 [cache_rows, H, 4]; it reads as zeros."""
    R, H = int(cache_rows), int(num_heads)
    codes = lambda: torch.full((R, H, 64), 0x88, dtype=_U8, device=device)
    scales = lambda: torch.zeros((R, H, 4), dtype=_BF16, device=device)
    return codes(), scales(), codes(), scales()


def _cache_args(cache):
    """Rows, heads and the four addresses of a cache."""
    kc, ks, vc, vs = cache
    R, H = kc.shape[0], kc.shape[1]
    return R, H, (_arg(kc, "k_codes", _U8, R, H, 64), _arg(ks, "k_scales", _BF16, R, H, 4),
                  _arg(vc, "v_codes", _U8, R, H, 64), _arg(vs, "v_scales", _BF16, R, H, 4))


def hstu_kv4_pack(k, v, *, cache=None, rows=None, workspace=None, stream=None):
    """Writes keys and values [T, H, 128] (bf16) to a 4-bit cache: to the rows
    ``rows`` (int32 [T], distinct, -1 skips), else to rows 0..T-1.  Without
    ``cache`` a new one of T rows.  Returns the cache."""
    lib = load_library()
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a [T, H, 128] tensor")
    T, H = k.shape[0], k.shape[1]
    kp, vp = _arg(k, "k", _BF16, T, H, 128), _arg(v, "v", _BF16, T, H, 128)
    rp = _arg(rows, "rows", _I32, T)
    new = cache is None
    with _on(k, v, rows, workspace, *(cache or ()), stream=stream):
        if cache is None:
            if rows is not None:
                raise ValueError("rows need a cache")
            cache = (k.new_empty((T, H, 64), dtype=_U8), k.new_empty((T, H, 4)),
                     k.new_empty((T, H, 64), dtype=_U8), k.new_empty((T, H, 4)))
        R, HC, ptrs = _cache_args(cache)
        if HC != H:
            raise ValueError("the cache has %d heads, k has %d" % (HC, H))
        wp, wn = None, 0
        if rows is not None or workspace is not None:
            workspace, wp, wn = _room(workspace, k)
        rc = lib.hstu_kv4_pack(T, H, kp, vp, rp, R, *ptrs, wp, wn, _stream_of(k, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_kv4_pack")
    if new:
        _hand_over(stream, *cache)
    return cache


def hstu_kv4_unpack(cache, *, rows=None, out=None, workspace=None, stream=None):
    """Keys and values [T, H, 128] (bf16) of a 4-bit cache's rows ``rows``
    (int32 [T]; a token of row -1 keeps what ``out`` holds), else of all rows."""
    lib = load_library()
    R, H, ptrs = _cache_args(cache)
    rp = _arg(rows, "rows", _I32)
    T = R if rows is None else rows.numel()
    ref = cache[0]
    new = out is None
    with _on(ref, *cache, rows, workspace, *(out or ()), stream=stream):
        if out is None:
            make = ref.new_empty if rows is None else ref.new_zeros
            out = make((T, H, 128), dtype=_BF16), make((T, H, 128), dtype=_BF16)
        k, v = out
        kp, vp = _arg(k, "k", _BF16, T, H, 128), _arg(v, "v", _BF16, T, H, 128)
        wp, wn = None, 0
        if rows is not None or workspace is not None:
            workspace, wp, wn = _room(workspace, ref)
        rc = lib.hstu_kv4_unpack(T, H, *ptrs, rp, R, kp, vp, wp, wn, _stream_of(ref, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_kv4_unpack")
    if new:
        _hand_over(stream, k, v)
    return k, v


def hstu_cand_kv4_workspace(batch: int, num_heads: int, max_seq_len: int, total_cands: int,
                            max_cands: int, device):
    """Workspace of hstu_cand_kv4_fwd for these sizes; with as many heads it serves
    every call of no larger ones."""
    n = int(load_library().hstu_cand_kv4_workspace_size(int(batch), int(num_heads),
                                                        int(max_seq_len), int(total_cands),
                                                        int(max_cands)))
    if n == 0:
        raise HSTUError(HSTU_ERR_INVALID_ARG, "hstu_cand_kv4_workspace_size")
    return torch.zeros(n, dtype=_U8, device=device)


def hstu_cand_kv4_fwd(cache, offsets, max_seq_len: int, q, k, v, u, cand_offsets, max_cands: int, *,
                      first_rows=None, total_tokens=None, timestamps=None, cand_timestamps=None,
                      rab_pos=None, rab_time=None, norm_len=0, eps=1e-5, ln_weight=None,
                      ln_bias=None, offsets_host=None, y=None, workspace=None, stream=None):
    """hstu_cand_fwd against histories in a 4-bit cache (hstu_kv4_pack): user b's
    history is the cache rows first_rows[b].. (int32 [B]), or, without
    first_rows, the rows offsets[b]..offsets[b+1]-1.  total_tokens bounds
    offsets[B] (default: the timestamps' length and, without first_rows, the
    cache's rows).  q, k, v, u may be longer than cand_offsets[B] and timestamps
    than offsets[B]; rows of y that belong to no user stay as they were.  Returns
    y [C, H*128]."""
    lib = load_library()
    R, HC, ptrs = _cache_args(cache)
    qp = _arg(q, "q", _BF16)
    C, H, _ = q.shape
    B = offsets.numel() - 1
    if H != HC:
        raise ValueError("the cache has %d heads, q has %d" % (HC, H))
    if rab_pos is not None and (rab_pos.dim() != 2 or rab_pos.shape[1] % 2 != 1):
        raise ValueError("rab_pos must be [H, 2L - 1]")
    if timestamps is not None and timestamps.dim() != 1:
        raise ValueError("timestamps must be [T]")
    W = 0 if rab_pos is None else rab_pos.shape[1]
    NB = 0 if rab_time is None else rab_time.shape[-1]
    limit = timestamps.numel() if timestamps is not None else 2 ** 31 - 1
    if offsets_host is not None:
        if (offsets_host.is_cuda or offsets_host.dtype != _I32 or offsets_host.shape != (B + 1,)
                or not offsets_host.is_contiguous()):
            raise ValueError("offsets_host must be a contiguous int32 CPU tensor [B + 1]")
        total_tokens = int(offsets_host[-1])
    max_seq_len, max_cands = int(max_seq_len), int(max_cands)
    if total_tokens is None:
        # (no users, or a cache without rows: no history either)
        total_tokens = (min(limit, R) if first_rows is None else limit) if B > 0 and R > 0 else 0
    elif timestamps is not None and total_tokens > limit:
        raise ValueError("total_tokens exceeds the timestamps' length")
    new = y is None
    with _on(q, *cache, offsets, k, v, u, cand_offsets, first_rows, timestamps, cand_timestamps,
             rab_pos, rab_time, ln_weight, ln_bias, y, workspace, stream=stream):
        p = hstu_problem_t(HSTU_BF16, B, int(total_tokens), max_seq_len, H, 128, 128,
                           _arg(offsets, "offsets", _I32, B + 1),
                           None if offsets_host is None else offsets_host.data_ptr(),
                           _arg(timestamps, "timestamps", _I64),
                           _arg(rab_pos, "rab_pos", _F32, H, W), (W + 1) // 2,
                           _arg(rab_time, "rab_time", _F32, H, NB), NB, int(norm_len), float(eps),
                           _arg(ln_weight, "ln_weight", _F32, H * 128),
                           _arg(ln_bias, "ln_bias", _F32, H * 128))
        if rab_time is not None and timestamps is not None and total_tokens == 0:
            p.timestamps = p.rab_time   # nothing to read; an empty tensor has no address
        if y is None:
            y = torch.empty_like(u)
        if workspace is None:
            workspace = hstu_cand_kv4_workspace(B, H, max_seq_len, C, max_cands, q.device)
        workspace, wp, wn = _room(workspace, q)
        rc = lib.hstu_cand_kv4_fwd(
            ctypes.byref(p), *ptrs, R, _arg(first_rows, "first_rows", _I32, B),
            _arg(cand_offsets, "cand_offsets", _I32, B + 1), C, max_cands,
            _arg(cand_timestamps, "cand_timestamps", _I64, C), _arg(q, "q", _BF16, C, H, 128),
            _arg(k, "k", _BF16, C, H, 128), _arg(v, "v", _BF16, C, H, 128),
            _arg(u, "u", _BF16, C, H * 128), _arg(y, "y", _BF16, C, H * 128), wp, wn,
            _stream_of(q, stream))
    if rc != HSTU_OK:
        raise HSTUError(rc, "hstu_cand_kv4_fwd")
    _hand_over(stream, y if new else None)
    return y
