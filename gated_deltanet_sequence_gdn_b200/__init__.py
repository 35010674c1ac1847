"""Python binding of libgdn.so, the B200 (sm_100a) Gated DeltaNet hot path.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libgdn.so, called through its C ABI (include/gdn.h) with ctypes.
PyTorch provides device memory and the current stream.  There is no CPU or
Python fallback: importing this module fails if the library is not built, and
every call raises if the library reports an error.

Entry points (same names as the C ABI):
    gdn_gate_prep, gdn_chunk_fwd, gdn_chunk_workspace_bytes, gdn_chunk_fwd_noalloc,
    gdn_recurrent_step, gdn2_chunk_fwd, gdn_check_status
and, with the vector state, gdn_linrec_fwd, gdn_linrec_bwd, gdn_linrec_step; for q and k,
gdn_qk_norm_rope, gdn_qk_norm_rope_bwd.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

__all__ = ["gdn_gate_prep", "gdn_chunk_fwd", "gdn_chunk_workspace_bytes", "gdn_recurrent_step",
           "gdn_conv_prefill", "gdn_rmsnorm_gated", "gdn_kda_chunk_fwd",
           "gdn_kda_chunk_workspace_bytes", "gdn_chunk_fwd_varlen",
           "gdn_chunk_varlen_workspace_bytes",
           "gdn2_chunk_fwd", "gdn2_chunk_workspace_bytes", "gdn_chunk_fwd_noalloc",
           "gdn_chunk_fwd_gated_norm", "gdn_recurrent_step_gated_norm",
           "gdn_chunk_bwd", "gdn_chunk_bwd_workspace_bytes",
           "gdn_linrec_fwd", "gdn_linrec_bwd", "gdn_linrec_step", "gdn_linrec_chunks",
           "gdn_linrec_workspace_bytes", "gdn_linrec_bwd_workspace_bytes",
           "gdn_qk_norm_rope", "gdn_qk_norm_rope_bwd", "gdn_qk_norm_rope_bwd_workspace_bytes",
           "gdn_check_status", "gdn_status", "gdn_test_set_wait_fault", "GDNError",
           "LIB_PATH", "lib", "F32", "BF16",
           "QK_L2NORM", "GATES_PRECOMPUTED", "OUT_F32", "LINREC_TIED", "LINREC_UNIT",
           "GRAD_F32", "QK_RMSNORM", "ROPE_INTERLEAVED", "LINREC_CHUNK"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python gated_deltanet_sequence_gdn_b200/build.py`"
        " (nvcc, sm_100a). There is no fallback implementation.")

lib = ctypes.CDLL(LIB_PATH)

F32, BF16 = 0, 1
QK_L2NORM, GATES_PRECOMPUTED, OUT_F32 = 1, 2, 4
LINREC_TIED, LINREC_UNIT, GRAD_F32, QK_RMSNORM, ROPE_INTERLEAVED = 8, 16, 32, 64, 128
LINREC_CHUNK = 64
_STATUS = {0: "GDN_OK", -1: "GDN_ERR_INVALID_ARG", -2: "GDN_ERR_UNSUPPORTED",
           -3: "GDN_ERR_CUDA", -4: "GDN_ERR_TIMEOUT", -5: "GDN_ERR_WORKSPACE",
           -6: "GDN_ERR_RANGE"}

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
lib.gdn_gate_prep.argtypes = [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                              _vp, _vp, _vp, _vp, _vp]
lib.gdn_chunk_fwd.argtypes = [_vp] * 8 + [_i] * 7 + [_f, _i, _vp, _vp, _vp, _sz, _vp]
lib.gdn2_chunk_fwd.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _i, _vp, _vp, _vp, _sz, _vp]
lib.gdn_chunk_fwd_noalloc.argtypes = [_vp] * 8 + [_i] * 7 + [_f, _i, _vp, _vp, _vp]
lib.gdn_chunk_fwd_host.argtypes = [_vp] * 8 + [_i] * 7 + [_f, _i, _vp, _vp, _i, _vp, _sz, _vp]
lib.gdn_chunk_fwd_host_workspace_bytes.argtypes = [_i] * 9
lib.gdn_chunk_fwd_host_workspace_bytes.restype = _sz
lib.gdn_recurrent_step.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _i, _vp]
lib.gdn_conv_prefill.argtypes = [_vp] * 6 + [_i] * 7 + [_vp]
lib.gdn_rmsnorm_gated.argtypes = [_vp] * 4 + [ctypes.c_long, _i, _i, _f, _vp]
lib.gdn_chunk_fwd_varlen.argtypes = ([_vp] * 8 + [ctypes.POINTER(ctypes.c_longlong)] + [_i] * 6
                                     + [_f, _i, _vp, _vp, _vp, _sz, _vp])
lib.gdn_chunk_varlen_workspace_bytes.argtypes = [ctypes.POINTER(ctypes.c_longlong)] + [_i] * 6
lib.gdn_chunk_varlen_workspace_bytes.restype = _sz
lib.gdn_kda_chunk_fwd.argtypes = [_vp] * 8 + [_i] * 6 + [_f, _i, _vp, _vp, _vp, _sz, _vp]
lib.gdn_kda_chunk_workspace_bytes.argtypes = [_i] * 7
lib.gdn_kda_chunk_workspace_bytes.restype = _sz
lib.gdn_chunk_workspace_bytes.argtypes = [_i] * 7
lib.gdn2_chunk_workspace_bytes.argtypes = [_i] * 6
lib.gdn_chunk_workspace_bytes.restype = _sz
lib.gdn2_chunk_workspace_bytes.restype = _sz
lib.gdn_chunk_fwd_gated_norm.argtypes = [_vp] * 10 + [_f] + [_i] * 7 + [_f, _i, _vp, _vp, _vp,
                                                                       _sz, _vp]
lib.gdn_recurrent_step_gated_norm.argtypes = [_vp] * 10 + [_f, _vp] + [_i] * 6 + [_f, _i, _vp]
lib.gdn_chunk_bwd.argtypes = [_vp] * 10 + [_i] * 7 + [_f, _i] + [_vp] * 9 + [_sz, _vp]
lib.gdn_chunk_bwd_workspace_bytes.argtypes = [_i] * 6
lib.gdn_chunk_bwd_workspace_bytes.restype = _sz
lib.gdn_linrec_fwd.argtypes = ([_vp] * 7 + [_i] * 3 + [_ll] * 3 + [_i, _i, _vp, _ll] + [_vp] * 3
                               + [_sz, _vp])
lib.gdn_linrec_bwd.argtypes = ([_vp] * 7 + [_i] * 3 + [_ll] * 3 + [_vp, _ll, _vp, _vp, _i, _i]
                               + [_vp, _ll] * 3 + [_vp] * 4 + [_sz, _vp])
lib.gdn_linrec_step.argtypes = [_vp] * 6 + [_i] * 2 + [_ll] * 3 + [_i, _i, _vp, _ll, _vp]
lib.gdn_linrec_workspace_bytes.argtypes = [_vp, _i, _i, _i]
lib.gdn_linrec_workspace_bytes.restype = _sz
lib.gdn_linrec_bwd_workspace_bytes.argtypes = [_vp, _i, _i, _i, _i, _i]
lib.gdn_linrec_bwd_workspace_bytes.restype = _sz
lib.gdn_qk_norm_rope.argtypes = ([_vp] * 6 + [_ll] + [_i] * 4 + [_ll] * 2 + [_i, _i, _f, _f]
                                 + [_vp, _ll] * 2 + [_vp])
lib.gdn_qk_norm_rope_bwd.argtypes = ([_vp] * 6 + [_ll] + [_i] * 4 + [_ll] * 2 + [_vp, _ll] * 2
                                     + [_i, _i, _f, _f] + [_vp, _ll] * 2 + [_vp] * 3
                                     + [_sz, _vp])
lib.gdn_qk_norm_rope_bwd_workspace_bytes.argtypes = [_ll] + [_i] * 4
lib.gdn_qk_norm_rope_bwd_workspace_bytes.restype = _sz
lib.gdn_check_status.argtypes = [_vp]
lib.gdn_test_set_wait_fault.argtypes = [_i, ctypes.c_uint]
lib.gdn_test_set_wait_fault.restype = _i
lib.gdn_status_string.argtypes = [_i]
lib.gdn_status_string.restype = ctypes.c_char_p
lib.gdn_version.argtypes = []
for _fn in (lib.gdn_gate_prep, lib.gdn_chunk_fwd, lib.gdn_chunk_fwd_noalloc, lib.gdn_chunk_fwd_host,
            lib.gdn_chunk_fwd_gated_norm, lib.gdn_recurrent_step_gated_norm,
            lib.gdn2_chunk_fwd,
            lib.gdn_recurrent_step, lib.gdn_conv_prefill, lib.gdn_rmsnorm_gated,
            lib.gdn_kda_chunk_fwd, lib.gdn_chunk_fwd_varlen,
            lib.gdn_linrec_fwd, lib.gdn_linrec_bwd, lib.gdn_linrec_step,
            lib.gdn_qk_norm_rope, lib.gdn_qk_norm_rope_bwd,
            lib.gdn_check_status, lib.gdn_version):
    _fn.restype = _i


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


def _check(status: int, where: str):
    if status != 0:
        raise GDNError(status, where)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t}; expected bfloat16 or float32")


def _p(t):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _ph(t):
    """Host pointer of a contiguous CPU tensor (None -> NULL); page-locked memory
    (tensor.pin_memory()) gives asynchronous copies."""
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("tensor must live in host memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def gdn_gate_prep(q, k, a, b, A_log, dt_bias, *, scale=None, q_out=None, k_out=None,
                  g_out=None, beta_out=None, stream=None):
    """Gate + L2-norm prologue. Returns (q_hat, k_hat, g, beta)."""
    B, T, Hk, d = q.shape
    Hv = a.shape[2]
    dt = q.dtype
    scale = d ** -0.5 if scale is None else scale
    q_out = torch.empty_like(q) if q_out is None else q_out
    k_out = torch.empty_like(k) if k_out is None else k_out
    g_out = torch.empty((B, T, Hv), device=q.device, dtype=torch.float32) if g_out is None else g_out
    beta_out = torch.empty_like(g_out) if beta_out is None else beta_out
    _need(k, dt, q.shape, "k")
    _need(a, dt, (B, T, Hv), "a")
    _need(b, dt, (B, T, Hv), "b")
    _check(lib.gdn_gate_prep(_p(q), _p(k), _dtype_code(dt), _p(a), _p(b), _p(A_log),
                             _p(dt_bias), B, T, Hk, Hv, d, float(scale), _p(q_out), _p(k_out),
                             _p(g_out), _p(beta_out), _stream(stream)), "gdn_gate_prep")
    return q_out, k_out, g_out, beta_out


def gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv, dtype) -> int:
    """Bytes of device workspace gdn_chunk_fwd needs for these sizes (0 = none)."""
    return int(lib.gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv, _dtype_code(dtype)))


def gdn_chunk_fwd(q, k, v, a, b, A_log=None, dt_bias=None, h0=None, *, scale=None,
                  l2norm=True, gates_precomputed=False, out_f32=False, o=None, ht=None,
                  want_ht=True, workspace=None, stream=None):
    """Chunkwise GDN prefill. q, k [B,T,Hk,dk]; v [B,T,Hv,dv]; a, b [B,T,Hv]
    (float32 g, beta with gates_precomputed); A_log, dt_bias [Hv] float32;
    h0 [B,Hv,dk,dv] float32 or None.  Returns (o [B,T,Hv,dv], ht or None);
    o has the input dtype, or float32 with out_f32.  workspace: a uint8 CUDA
    tensor of at least gdn_chunk_workspace_bytes(...) bytes, allocated here
    when None."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    gdt = torch.float32 if gates_precomputed else dt
    _need(a, gdt, (B, T, Hv), "a")
    _need(b, gdt, (B, T, Hv), "b")
    if h0 is not None:
        _need(h0, torch.float32, (B, Hv, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, Hv, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (B, T, Hv, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    ws_need = gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_chunk_fwd(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias), _p(h0),
                             B, T, Hk, Hv, dk, dv, _dtype_code(dt), float(scale), flags, _p(o),
                             _p(ht), _p(workspace), ws_bytes, _stream(stream)), "gdn_chunk_fwd")
    return o, ht


def gdn_chunk_fwd_gated_norm(q, k, v, a, b, A_log, dt_bias, h0, z, norm_weight, *, eps=1e-6,
                             scale=None, l2norm=True, gates_precomputed=False, out_f32=False,
                             o=None, ht=None, want_ht=True, workspace=None, stream=None):
    """gdn_chunk_fwd with the gated RMSNorm of the output stage applied to o:
    o = core / sqrt(mean(core^2) + eps) * norm_weight * SiLU(z) per (token, value
    head); z [B,T,Hv,dv] in the input dtype, norm_weight [dv] float32.  Fused into
    the scan's output store on the bf16 d = 128 path.  Returns (o, ht)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    gdt = torch.float32 if gates_precomputed else dt
    _need(a, gdt, (B, T, Hv), "a")
    _need(b, gdt, (B, T, Hv), "b")
    _need(z, dt, (B, T, Hv, dv), "z")
    _need(norm_weight, torch.float32, (dv,), "norm_weight")
    if h0 is not None:
        _need(h0, torch.float32, (B, Hv, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, Hv, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (B, T, Hv, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    ws_need = gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_chunk_fwd_gated_norm(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log),
                                        _p(dt_bias), _p(h0), _p(z), _p(norm_weight),
                                        float(eps), B, T, Hk, Hv, dk, dv, _dtype_code(dt),
                                        float(scale), flags, _p(o), _p(ht), _p(workspace),
                                        ws_bytes, _stream(stream)), "gdn_chunk_fwd_gated_norm")
    return o, ht


def gdn_chunk_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv):
    return lib.gdn_chunk_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv)


def gdn_chunk_bwd(q, k, v, a, b, A_log, dt_bias, h0, do, dht=None, *, scale=None, l2norm=True,
                  gates_precomputed=False, want_dh0=True, workspace=None, stream=None):
    """Gradients of sum(o * do) + sum(ht * dht) for gdn_chunk_fwd's (o, ht) on the same
    inputs (see include/gdn.h).  Returns a dict of float32 tensors dq, dk [B,T,Hk,dk],
    dv [B,T,Hv,dv], da, db [B,T,Hv] (with gates_precomputed: with respect to g and
    beta), dA_log, ddt_bias [Hv] (None with gates_precomputed) and dh0 [B,Hv,dk,dv]
    (None unless want_dh0)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    _need(do, dt, (B, T, Hv, dv), "do")
    gdt = torch.float32 if gates_precomputed else dt
    _need(a, gdt, (B, T, Hv), "a")
    _need(b, gdt, (B, T, Hv), "b")
    if h0 is not None:
        _need(h0, torch.float32, (B, Hv, dk, dv), "h0")
    if dht is not None:
        _need(dht, torch.float32, (B, Hv, dk, dv), "dht")
    f32 = dict(device=q.device, dtype=torch.float32)
    out = {"dq": torch.empty((B, T, Hk, dk), **f32), "dk": torch.empty((B, T, Hk, dk), **f32),
           "dv": torch.empty((B, T, Hv, dv), **f32), "da": torch.empty((B, T, Hv), **f32),
           "db": torch.empty((B, T, Hv), **f32),
           "dA_log": None if gates_precomputed else torch.empty((Hv,), **f32),
           "ddt_bias": None if gates_precomputed else torch.empty((Hv,), **f32),
           "dh0": torch.empty((B, Hv, dk, dv), **f32) if want_dh0 else None}
    flags = (QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
    ws_need = gdn_chunk_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_chunk_bwd(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias), _p(h0),
                             _p(do), _p(dht), B, T, Hk, Hv, dk, dv, _dtype_code(dt),
                             float(scale), flags, _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                             _p(out["da"]), _p(out["db"]), _p(out["dA_log"]),
                             _p(out["ddt_bias"]), _p(out["dh0"]), _p(workspace), ws_bytes,
                             _stream(stream)), "gdn_chunk_bwd")
    return out


def gdn_chunk_fwd_noalloc(q, k, v, a, b, A_log=None, dt_bias=None, h0=None, *, scale=None,
                          l2norm=True, gates_precomputed=False, out_f32=False, o=None, ht=None,
                          want_ht=True, stream=None):
    """gdn_chunk_fwd with the library's fixed 64 MiB device scratch instead of a
    workspace (raises GDNError(GDN_ERR_WORKSPACE) when the sizes need more)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    gdt = torch.float32 if gates_precomputed else dt
    _need(a, gdt, (B, T, Hv), "a")
    _need(b, gdt, (B, T, Hv), "b")
    if h0 is not None:
        _need(h0, torch.float32, (B, Hv, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, Hv, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (B, T, Hv, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    _check(lib.gdn_chunk_fwd_noalloc(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias),
                                     _p(h0), B, T, Hk, Hv, dk, dv, _dtype_code(dt), float(scale),
                                     flags, _p(o), _p(ht), _stream(stream)),
           "gdn_chunk_fwd_noalloc")
    return o, ht


def gdn_chunk_fwd_host_workspace_bytes(B, T, Hk, Hv, dk, dv, dtype, *, l2norm=True,
                                       gates_precomputed=False, out_f32=False,
                                       piece_tokens=0) -> int:
    """Bytes of device scratch gdn_chunk_fwd_host needs for these sizes."""
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    return int(lib.gdn_chunk_fwd_host_workspace_bytes(B, T, Hk, Hv, dk, dv, _dtype_code(dtype),
                                                      flags, piece_tokens))


def gdn_chunk_fwd_host(q, k, v, a, b, A_log=None, dt_bias=None, h0=None, *, scale=None,
                       l2norm=True, gates_precomputed=False, out_f32=False, o=None, ht=None,
                       want_ht=True, piece_tokens=0, dev_workspace=None, device=None,
                       stream=None, sync=True):
    """gdn_chunk_fwd for host (CPU) tensors: the library copies the sequence to the
    device piece by piece, overlapping the copies in, the compute and the copies
    out.  Arguments as gdn_chunk_fwd, all CPU tensors (pin_memory() for
    asynchronous copies); o / ht are CPU tensors (page-locked when allocated
    here).  dev_workspace: a uint8 CUDA tensor of at least
    gdn_chunk_fwd_host_workspace_bytes(...) bytes, allocated here when None.
    Returns (o, ht); with sync=True (the default) once the stream has completed, so
    that they hold the results; with sync=False as soon as the work is enqueued (the
    host buffers are written asynchronously until the stream completes, and a
    dev_workspace allocated here must not be reused before then)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    gdt = torch.float32 if gates_precomputed else dt
    _need(a, gdt, (B, T, Hv), "a")
    _need(b, gdt, (B, T, Hv), "b")
    if h0 is not None:
        _need(h0, torch.float32, (B, Hv, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, Hv, dv), dtype=odt).pin_memory() if o is None else o
    _need(o, odt, (B, T, Hv, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), dtype=torch.float32).pin_memory()
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    need = lib.gdn_chunk_fwd_host_workspace_bytes(B, T, Hk, Hv, dk, dv, _dtype_code(dt), flags,
                                                  piece_tokens)
    if dev_workspace is None and need > 0:
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        dev_workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if dev_workspace is None else dev_workspace.numel() * dev_workspace.element_size()
    st = _stream(stream)
    _check(lib.gdn_chunk_fwd_host(_ph(q), _ph(k), _ph(v), _ph(a), _ph(b), _ph(A_log),
                                  _ph(dt_bias), _ph(h0), B, T, Hk, Hv, dk, dv, _dtype_code(dt),
                                  float(scale), flags, _ph(o), _ph(ht), int(piece_tokens),
                                  _p(dev_workspace), ws_bytes, st), "gdn_chunk_fwd_host")
    if sync:
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return o, ht


def gdn2_chunk_workspace_bytes(B, T, H, dk, dv, dtype) -> int:
    """Bytes of device workspace gdn2_chunk_fwd needs for these sizes (0 = none)."""
    return int(lib.gdn2_chunk_workspace_bytes(B, T, H, dk, dv, _dtype_code(dtype)))


def gdn2_chunk_fwd(q, k, v, a, b_logit, w_logit, A_log=None, dt_bias=None, h0=None, *,
                   scale=None, l2norm=True, gates_precomputed=False, out_f32=False, o=None,
                   ht=None, want_ht=True, workspace=None, stream=None):
    """Chunkwise Gated DeltaNet-2 forward. q, k, a, b_logit [B,T,H,dk]; v, w_logit
    [B,T,H,dv]; A_log, dt_bias [H,dk] float32; h0 [B,H,dk,dv] or None.  With
    gates_precomputed, a is the per-channel log-decay and b_logit / w_logit are
    the gate values (float32).  workspace as for gdn_chunk_fwd."""
    B, T, H, dk = q.shape
    dv = v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    gdt = torch.float32 if gates_precomputed else dt
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, H, dv), "v")
    _need(a, gdt, (B, T, H, dk), "a")
    _need(b_logit, gdt, (B, T, H, dk), "b_logit")
    _need(w_logit, gdt, (B, T, H, dv), "w_logit")
    if h0 is not None:
        _need(h0, torch.float32, (B, H, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, H, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (B, T, H, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, H, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    ws_need = gdn2_chunk_workspace_bytes(B, T, H, dk, dv, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn2_chunk_fwd(_p(q), _p(k), _p(v), _p(a), _p(b_logit), _p(w_logit), _p(A_log),
                              _p(dt_bias), _p(h0), B, T, H, dk, dv, _dtype_code(dt),
                              float(scale), flags, _p(o), _p(ht), _p(workspace), ws_bytes,
                              _stream(stream)),
           "gdn2_chunk_fwd")
    return o, ht


def gdn_chunk_varlen_workspace_bytes(cu_seqlens, Hk, Hv, dk, dv, dtype) -> int:
    """Device workspace bytes gdn_chunk_fwd_varlen needs for these N + 1 token
    offsets (0 when the call needs none)."""
    cu = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    if len(cu) < 2:
        return 0
    arr = (ctypes.c_longlong * len(cu))(*cu)
    return int(lib.gdn_chunk_varlen_workspace_bytes(arr, len(cu) - 1, Hk, Hv, dk, dv,
                                                    _dtype_code(dtype)))


def gdn_chunk_fwd_varlen(q, k, v, a, b, A_log, dt_bias, h0, cu_seqlens, *, scale=None,
                         l2norm=True, gates_precomputed=False, out_f32=False, o=None, ht=None,
                         want_ht=True, workspace=None, stream=None):
    """Chunkwise GDN prefill over a packed batch: q, k [T_total, Hk, dk]; v
    [T_total, Hv, dv]; a, b [T_total, Hv]; cu_seqlens: N + 1 token offsets (a list
    or a CPU int64 tensor, first 0); h0 [N, Hv, dk, dv] or None.  Returns
    (o [T_total, Hv, dv], ht [N, Hv, dk, dv] or None)."""
    cu = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    N = len(cu) - 1
    Tt, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    gdt = torch.float32 if gates_precomputed else dt
    _need(k, dt, q.shape, "k")
    _need(v, dt, (Tt, Hv, dv), "v")
    _need(a, gdt, (Tt, Hv), "a")
    _need(b, gdt, (Tt, Hv), "b")
    if N < 0 or cu[0] != 0 or cu[-1] != Tt:
        raise ValueError("cu_seqlens must start at 0 and end at the packed token count")
    if h0 is not None:
        _need(h0, torch.float32, (N, Hv, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((Tt, Hv, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (Tt, Hv, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((N, Hv, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    cu_arr = (ctypes.c_longlong * len(cu))(*cu)
    ws_need = gdn_chunk_varlen_workspace_bytes(cu, Hk, Hv, dk, dv, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_chunk_fwd_varlen(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias),
                                    _p(h0), cu_arr, N, Hk, Hv, dk, dv, _dtype_code(dt),
                                    float(scale), flags, _p(o), _p(ht), _p(workspace), ws_bytes,
                                    _stream(stream)),
           "gdn_chunk_fwd_varlen")
    return o, ht


def gdn_kda_chunk_workspace_bytes(B, T, H, dk, dv, dtype, gates_precomputed=False) -> int:
    """Bytes of device workspace gdn_kda_chunk_fwd needs (the tiled gates included)."""
    return int(lib.gdn_kda_chunk_workspace_bytes(B, T, H, dk, dv, _dtype_code(dtype),
                                                 GATES_PRECOMPUTED if gates_precomputed else 0))


def gdn_kda_chunk_fwd(q, k, v, a, beta, A_log=None, dt_bias=None, h0=None, *, scale=None,
                      l2norm=True, gates_precomputed=False, out_f32=False, o=None, ht=None,
                      want_ht=True, workspace=None, stream=None):
    """Chunkwise KDA forward: Gated DeltaNet-2 with one beta per (token, head) for
    the erase and the write.  q, k, a [B,T,H,dk]; v [B,T,H,dv]; beta [B,T,H] (the
    logit, or beta in float32 with gates_precomputed, a then the per-channel
    log-decay); A_log, dt_bias [H,dk] float32; h0 [B,H,dk,dv] or None."""
    B, T, H, dk = q.shape
    dv = v.shape[3]
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    gdt = torch.float32 if gates_precomputed else dt
    _need(k, dt, q.shape, "k")
    _need(v, dt, (B, T, H, dv), "v")
    _need(a, gdt, (B, T, H, dk), "a")
    _need(beta, gdt, (B, T, H), "beta")
    if h0 is not None:
        _need(h0, torch.float32, (B, H, dk, dv), "h0")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((B, T, H, dv), device=q.device, dtype=odt) if o is None else o
    _need(o, odt, (B, T, H, dv), "o")
    if ht is None and want_ht:
        ht = torch.empty((B, H, dk, dv), device=q.device, dtype=torch.float32)
    flags = ((QK_L2NORM if l2norm else 0) | (GATES_PRECOMPUTED if gates_precomputed else 0)
             | (OUT_F32 if out_f32 else 0))
    ws_need = gdn_kda_chunk_workspace_bytes(B, T, H, dk, dv, dt, gates_precomputed)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_kda_chunk_fwd(_p(q), _p(k), _p(v), _p(a), _p(beta), _p(A_log), _p(dt_bias),
                                 _p(h0), B, T, H, dk, dv, _dtype_code(dt), float(scale), flags,
                                 _p(o), _p(ht), _p(workspace), ws_bytes, _stream(stream)),
           "gdn_kda_chunk_fwd")
    return o, ht


def gdn_recurrent_step(x, conv_w, conv_state, a, b, A_log, dt_bias, state, *, Hk, Hv, dk,
                       dv, scale=None, out_f32=False, o=None, stream=None):
    """One fused conv1d + GDN decode step for N sequences; conv_state and state
    are updated in place.  x [N, 2*Hk*dk + Hv*dv]; returns o [N, Hv, dv]."""
    N = x.shape[0]
    dt = x.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(x, dt, (N, 2 * Hk * dk + Hv * dv), "x")
    _need(a, dt, (N, Hv), "a")
    _need(b, dt, (N, Hv), "b")
    _need(state, torch.float32, (N, Hv, dk, dv), "state")
    if conv_w is not None:
        _need(conv_w, torch.float32, (x.shape[1], 4), "conv_w")
        _need(conv_state, dt, (N, x.shape[1], 3), "conv_state")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((N, Hv, dv), device=x.device, dtype=odt) if o is None else o
    _need(o, odt, (N, Hv, dv), "o")
    _check(lib.gdn_recurrent_step(_p(x), _p(conv_w), _p(conv_state), _p(a), _p(b), _p(A_log),
                                  _p(dt_bias), _p(state), _p(o), N, Hk, Hv, dk, dv,
                                  _dtype_code(dt), float(scale), OUT_F32 if out_f32 else 0,
                                  _stream(stream)),
           "gdn_recurrent_step")
    return o


def gdn_recurrent_step_gated_norm(x, conv_w, conv_state, a, b, A_log, dt_bias, state, z,
                                  norm_weight, *, Hk, Hv, dk, dv, eps=1e-6, scale=None,
                                  out_f32=False, o=None, stream=None):
    """gdn_recurrent_step with the gated RMSNorm of the output stage fused into the
    store of o; z [N, Hv, dv] in the input dtype, norm_weight [dv] float32."""
    N = x.shape[0]
    dt = x.dtype
    scale = dk ** -0.5 if scale is None else scale
    _need(x, dt, (N, 2 * Hk * dk + Hv * dv), "x")
    _need(a, dt, (N, Hv), "a")
    _need(b, dt, (N, Hv), "b")
    _need(state, torch.float32, (N, Hv, dk, dv), "state")
    _need(z, dt, (N, Hv, dv), "z")
    _need(norm_weight, torch.float32, (dv,), "norm_weight")
    if conv_w is not None:
        _need(conv_w, torch.float32, (x.shape[1], 4), "conv_w")
        _need(conv_state, dt, (N, x.shape[1], 3), "conv_state")
    odt = torch.float32 if out_f32 else dt
    o = torch.empty((N, Hv, dv), device=x.device, dtype=odt) if o is None else o
    _need(o, odt, (N, Hv, dv), "o")
    _check(lib.gdn_recurrent_step_gated_norm(_p(x), _p(conv_w), _p(conv_state), _p(a), _p(b),
                                             _p(A_log), _p(dt_bias), _p(state), _p(z),
                                             _p(norm_weight), float(eps), _p(o), N, Hk, Hv, dk,
                                             dv, _dtype_code(dt), float(scale),
                                             OUT_F32 if out_f32 else 0, _stream(stream)),
           "gdn_recurrent_step_gated_norm")
    return o


def gdn_conv_prefill(x, conv_w, conv_state, *, Hk, Hv, dk, dv, q=None, k=None, v=None,
                     stream=None):
    """Causal conv1d (kernel 4) + SiLU over a prefill of the mixed stream
    x [B, T, 2*Hk*dk + Hv*dv]; conv_state [B, Cc, 3] (or None: a zero window) is
    read and then overwritten in place with the last three inputs.  Returns
    (q [B,T,Hk,dk], k [B,T,Hk,dk], v [B,T,Hv,dv]), not normalised."""
    B, T = x.shape[0], x.shape[1]
    dt = x.dtype
    Cc = 2 * Hk * dk + Hv * dv
    _need(x, dt, (B, T, Cc), "x")
    _need(conv_w, torch.float32, (Cc, 4), "conv_w")
    if conv_state is not None:
        _need(conv_state, dt, (B, Cc, 3), "conv_state")
    q = torch.empty((B, T, Hk, dk), device=x.device, dtype=dt) if q is None else q
    k = torch.empty((B, T, Hk, dk), device=x.device, dtype=dt) if k is None else k
    v = torch.empty((B, T, Hv, dv), device=x.device, dtype=dt) if v is None else v
    _need(q, dt, (B, T, Hk, dk), "q")
    _need(k, dt, (B, T, Hk, dk), "k")
    _need(v, dt, (B, T, Hv, dv), "v")
    _check(lib.gdn_conv_prefill(_p(x), _p(conv_w), _p(conv_state), _p(q), _p(k), _p(v), B, T,
                                Hk, Hv, dk, dv, _dtype_code(dt), _stream(stream)),
           "gdn_conv_prefill")
    return q, k, v


def gdn_rmsnorm_gated(o, z, weight, *, eps=1e-6, y=None, stream=None):
    """Gated RMSNorm of the core output over its last axis (d_v):
    y = o / sqrt(mean(o^2) + eps) * weight * SiLU(z).  o, z [..., dv] (same shape
    and dtype); weight [dv] float32.  y may be o or z (in place)."""
    dt = o.dtype
    dv = o.shape[-1]
    _need(z, dt, tuple(o.shape), "z")
    _need(weight, torch.float32, (dv,), "weight")
    y = torch.empty_like(o) if y is None else y
    _need(y, dt, tuple(o.shape), "y")
    rows = o.numel() // dv if dv else 0
    _check(lib.gdn_rmsnorm_gated(_p(o), _p(z), _p(weight), _p(y), rows, dv, _dtype_code(dt),
                                 float(eps), _stream(stream)),
           "gdn_rmsnorm_gated")
    return y


# ---- the gated linear recurrence and the norm-and-rotation of q and k ----------------------


def _on_device(fn):
    """Runs an entry point on its first argument's device and on `stream` (default: that
    device's current stream); what it allocates then belongs to that stream."""
    sig = inspect.signature(fn)
    name = next(iter(sig.parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{fn.__name__}: {name} must be a tensor")
        index = first.get_device()
        if index < 0:
            raise ValueError("tensor must live on a CUDA device")
        if stream is None and index == torch.cuda.current_device():
            return fn(*args, **kw)
        dev = first.device
        if stream is not None and stream.device != dev:
            raise ValueError(f"stream of {stream.device} for tensors of {dev}")
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return fn(*args, **kw)

    if "stream" not in sig.parameters:
        more = inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)
        call.__signature__ = sig.replace(parameters=[*sig.parameters.values(), more])
    return call


def _here(dev):
    """The handle of a device's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _new(t, dtype):
    """A contiguous tensor of t's shape (the call that does it in the least host time)."""
    if t.dtype is not dtype:
        return t.new_empty(t.shape, dtype=dtype)
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _like(t, dtype, shape, dev, name):
    """Raises unless the tensor has this dtype, shape and device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev.index:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")


def _dense(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of this dtype, shape and device (None -> NULL)."""
    if t is None:
        return None
    _like(t, dtype, shape, dev, name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _strided(t, dtype, shape, dev, name, tail=1):
    """(pointer, elements from one token to the next) of a tensor of one or two token axes
    and `tail` dense axes: a view whose tokens are a fixed distance apart, at least a
    token's elements (None -> (NULL, 0))."""
    if t is None:
        return None, 0
    _like(t, dtype, shape, dev, name)
    row = shape[-1] if tail == 1 else shape[-1] * shape[-2]
    if t.is_contiguous():
        return t.data_ptr(), row
    st = t.stride()
    if (st[-1] != 1 and shape[-1] > 1) or (tail == 2 and st[-2] != shape[-1] and shape[-2] > 1):
        raise ValueError(f"{name}: the elements of a token must be contiguous")
    if len(st) == tail + 1:
        ld = st[0] if shape[0] > 1 else row
    elif shape[1] > 1:
        ld = st[1]
        if shape[0] > 1 and st[0] != ld * shape[1]:
            raise ValueError(f"{name}: the tokens must be a fixed distance apart")
    else:
        ld = st[0] if shape[0] > 1 else row
    if ld < row:
        raise ValueError(f"{name}: tokens overlap (a broadcast view?)")
    return t.data_ptr(), ld


_SCALES = {"none": 0, "tied": LINREC_TIED, "unit": LINREC_UNIT}


def _host_offsets(cu_seqlens):
    """(ctypes int64 array or None, sequences)."""
    if cu_seqlens is None:
        return None, 0
    if hasattr(cu_seqlens, "tolist"):
        cu_seqlens = cu_seqlens.tolist()
    n = len(cu_seqlens)
    if n < 1:
        raise ValueError("cu_seqlens must hold the sequences' offsets and their end")
    return (_ll * n)(*cu_seqlens), n - 1


def gdn_linrec_chunks(B, T, cu_seqlens=None) -> int:
    """Rows of `states`: the chunks of LINREC_CHUNK tokens of all sequences."""
    if cu_seqlens is None:
        return B * (-(-T // LINREC_CHUNK))
    cu = cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens
    return sum(-(-(int(b) - int(a)) // LINREC_CHUNK) for a, b in zip(cu, cu[1:]))


def gdn_linrec_workspace_bytes(B, T, D, cu_seqlens=None) -> int:
    """Bytes of device workspace gdn_linrec_fwd needs (with cu_seqlens T is all packed tokens
    and B the offsets' number of sequences, whatever is passed)."""
    cu, n = _host_offsets(cu_seqlens)
    return int(lib.gdn_linrec_workspace_bytes(cu, B if cu is None else n, T, D))


def gdn_linrec_bwd_workspace_bytes(B, T, D, cu_seqlens=None, *, states_given=False,
                                   gates_precomputed=False) -> int:
    """Bytes of device workspace gdn_linrec_bwd needs (B and T as above)."""
    cu, n = _host_offsets(cu_seqlens)
    return int(lib.gdn_linrec_bwd_workspace_bytes(
        cu, B if cu is None else n, T, D, int(states_given),
        GATES_PRECOMPUTED if gates_precomputed else 0))


def _workspace(workspace, need, like, dev):
    """(tensor to keep, pointer, bytes) of a call's workspace, allocated here when None."""
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous and on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _linrec_inputs(x, a, b, A_log, dt_bias, gates_precomputed, input_scale):
    """Checked (arguments, flags) that the recurrence's entry points share."""
    dt, dev, shape = x.dtype, x.device, x.shape
    D = shape[-1]
    if input_scale not in _SCALES:
        raise ValueError(f"input_scale: expected one of {sorted(_SCALES)}, got {input_scale!r}")
    gdt = torch.float32 if gates_precomputed else dt
    px, ldx = _strided(x, dt, shape, dev, "x")
    pa, lda = _strided(a, gdt, shape, dev, "a")
    pb, ldb = _strided(b, gdt, shape, dev, "b")
    pA = pt = None
    if not gates_precomputed:
        pA = _dense(A_log, torch.float32, (D,), dev, "A_log")
        pt = _dense(dt_bias, torch.float32, (D,), dev, "dt_bias")
    flags = _SCALES[input_scale] | (GATES_PRECOMPUTED if gates_precomputed else 0)
    return (px, pa, pb, pA, pt), (ldx, lda, ldb), flags


def _linrec_sizes(x, cu_seqlens):
    """(host offsets or None, B, T, D)."""
    cu, n = _host_offsets(cu_seqlens)
    if x.dim() != (3 if cu is None else 2):
        raise ValueError("x: expected [B, T, D], or [T, D] with cu_seqlens")
    return (cu, n, x.shape[0], x.shape[1]) if cu is not None else (None, *x.shape)


def _clear_rest(cu, T, *outs):
    """Zeros in the tokens behind the last packed sequence, which the library leaves alone."""
    if cu is not None and cu[-1] < T:
        for t in outs:
            if t is not None:
                t[cu[-1]:].zero_()


@_on_device
def gdn_linrec_fwd(x, a, b=None, A_log=None, dt_bias=None, h0=None, *, cu_seqlens=None,
                   input_scale="none", gates_precomputed=False, out_f32=False, h=None, ht=None,
                   want_ht=True, want_states=False, states=None, workspace=None):
    """Gated linear recurrence h_t = alpha_t h_{t-1} + s(alpha_t) beta_t x_t per channel, with
    the delta rules' gates (alpha_t = exp(-exp(A_log) softplus(a_t + dt_bias)), beta_t =
    sigmoid(b_t), 1 without b) and s = 1, 1 - alpha or sqrt(1 - alpha^2) by input_scale
    ("none", "tied", "unit").  x, a, b [B,T,D], or [T,D] packed with cu_seqlens (N + 1 token
    offsets: a list or a CPU int64 tensor); they may be slices of one projection's output.
    With gates_precomputed a is log alpha and b is beta, float32.  A_log, dt_bias [D], h0 [B,D]
    float32.  Returns (h, ht), or (h, ht, states) with want_states: the float32 state before
    each chunk of LINREC_CHUNK tokens [gdn_linrec_chunks(...), D], for gdn_linrec_bwd.  h has
    the input dtype, or float32 with out_f32, and may be x; tokens behind the last packed
    sequence are zeros in an h that is allocated here, and stay as they are in the caller's.
    stream: as everywhere."""
    cu, B, T, D = _linrec_sizes(x, cu_seqlens)
    ins, lds, flags = _linrec_inputs(x, a, b, A_log, dt_bias, gates_precomputed, input_scale)
    dev, f32 = x.device, torch.float32
    odt = f32 if out_f32 else x.dtype
    own = h is None
    if own:
        h = _new(x, odt)
        ph, ldh = h.data_ptr(), D
    else:
        ph, ldh = _strided(h, odt, x.shape, dev, "h")
    if ht is None and want_ht:
        ht = x.new_empty((B, D), dtype=f32) if h0 is None else torch.empty_like(h0)
    if want_states or states is not None:
        shape = (gdn_linrec_chunks(B, T, cu), D)
        if states is None:
            states = x.new_empty(shape, dtype=f32)
        want_states = True
        ps = _dense(states, f32, shape, dev, "states")
    else:
        ps = None
    # a dense batch needs none
    need = 0 if cu is None else lib.gdn_linrec_workspace_bytes(cu, B, T, D)
    keep, ws, ws_bytes = _workspace(workspace, need, x, dev)
    _check(lib.gdn_linrec_fwd(*ins, _dense(h0, f32, (B, D), dev, "h0"), cu, B, T, D, *lds,
                              _dtype_code(x.dtype), flags | (OUT_F32 if out_f32 else 0), ph, ldh,
                              _dense(ht, f32, (B, D), dev, "ht"), ps, ws, ws_bytes,
                              _here(dev)), "gdn_linrec_fwd")
    if own:
        _clear_rest(cu, T, h)
    return (h, ht, states) if want_states else (h, ht)


@_on_device
def gdn_linrec_bwd(x, a, b, A_log, dt_bias, h0, dh, dht=None, *, cu_seqlens=None,
                   input_scale="none", gates_precomputed=False, grad_f32=False, states=None,
                   want_dh0=True, workspace=None):
    """Gradients of sum(h * dh) + sum(ht * dht) for gdn_linrec_fwd's (h, ht) on the same inputs
    (see include/gdn.h).  dh in the input dtype (float32 with grad_f32), states: the forward's
    (None: recomputed here).  Returns a dict: dx, da, db in dh's dtype (da, db float32 with
    gates_precomputed, with respect to log alpha and beta; db None without b), dA_log,
    ddt_bias [D] float32 (None with gates_precomputed), dh0 [B,D] float32 (None unless
    want_dh0).  The gradients of tokens behind the last packed sequence are zeros."""
    cu, B, T, D = _linrec_sizes(x, cu_seqlens)
    ins, lds, flags = _linrec_inputs(x, a, b, A_log, dt_bias, gates_precomputed, input_scale)
    dev, f32 = x.device, torch.float32
    ddt = f32 if grad_f32 else x.dtype
    gdt = f32 if gates_precomputed else ddt
    pdh, lddh = _strided(dh, ddt, x.shape, dev, "dh")
    out = {"dx": _new(x, ddt), "da": _new(x, gdt), "db": None if b is None else _new(x, gdt),
           "dA_log": None, "ddt_bias": None,
           "dh0": x.new_empty((B, D), dtype=f32) if want_dh0 else None}
    if not gates_precomputed:
        out["dA_log"], out["ddt_bias"] = torch.empty_like(A_log), torch.empty_like(dt_bias)
    ps = None
    if states is not None:
        ps = _dense(states, f32, (gdn_linrec_chunks(B, T, cu), D), dev, "states")
    keep, ws, ws_bytes = _workspace(
        workspace, lib.gdn_linrec_bwd_workspace_bytes(cu, B, T, D, int(states is not None), flags),
        x, dev)
    ptr = {k: None if v is None else v.data_ptr() for k, v in out.items()}
    _check(lib.gdn_linrec_bwd(*ins, _dense(h0, f32, (B, D), dev, "h0"), cu, B, T, D, *lds, pdh,
                              lddh, _dense(dht, f32, (B, D), dev, "dht"), ps,
                              _dtype_code(x.dtype), flags | (GRAD_F32 if grad_f32 else 0),
                              ptr["dx"], D, ptr["da"], D, ptr["db"], D, ptr["dA_log"],
                              ptr["ddt_bias"], ptr["dh0"], ws, ws_bytes,
                              _here(dev)), "gdn_linrec_bwd")
    _clear_rest(cu, T, out["dx"], out["da"], out["db"])
    return out


@_on_device
def gdn_linrec_step(x, a, b, A_log, dt_bias, state, *, input_scale="none",
                    gates_precomputed=False, out_f32=False, h=None):
    """One token of gdn_linrec_fwd for N sequences: x, a, b [N, D] (b None: beta = 1), state
    [N, D] float32 updated in place.  Returns h [N, D], which may be x."""
    if x.dim() != 2:
        raise ValueError("x: expected [N, D]")
    N, D = x.shape
    ins, lds, flags = _linrec_inputs(x, a, b, A_log, dt_bias, gates_precomputed, input_scale)
    odt = torch.float32 if out_f32 else x.dtype
    dev = x.device
    if h is None:
        h = _new(x, odt)
        ph, ldh = h.data_ptr(), D
    else:
        ph, ldh = _strided(h, odt, x.shape, dev, "h")
    _check(lib.gdn_linrec_step(*ins, _dense(state, torch.float32, x.shape, dev, "state"), N, D,
                               *lds, _dtype_code(x.dtype), flags | (OUT_F32 if out_f32 else 0),
                               ph, ldh, _here(dev)), "gdn_linrec_step")
    return h


_NORMS = {None: 0, "none": 0, "l2": QK_L2NORM, "rms": QK_RMSNORM}


def _norm_flag(norm):
    if norm not in _NORMS:
        raise ValueError(f"norm: expected 'rms', 'l2' or None, got {norm!r}")
    return _NORMS[norm]


def _rope_inputs(q, k, positions, inv_freq, q_weight, k_weight, norm, interleaved):
    """Checked arguments that both entry points share."""
    some = _either(q, k)
    dt, dev, lead, d = some.dtype, some.device, some.shape[:-2], some.shape[-1]
    if len(lead) not in (1, 2):
        raise ValueError("q, k: expected [T, H, d] or [B, T, H, d]")
    flags = _norm_flag(norm) | (ROPE_INTERLEAVED if interleaved else 0)
    Hq, Hk = (0 if t is None else t.shape[-2] for t in (q, k))
    tokens = lead.numel()
    pq, ldq = _strided(q, dt, (*lead, Hq, d), dev, "q", 2)
    pk, ldk = _strided(k, dt, (*lead, Hk, d), dev, "k", 2)
    rot = 0
    pp = pf = None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        pf = _dense(inv_freq, torch.float32, (rot // 2,), dev, "inv_freq")
        pp = _dense(positions, torch.int64, lead, dev, "positions")
    pw = [_dense(w, torch.float32, (d,), dev, n)
          for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight"))]
    return (pq, pk, pp, pf, *pw, tokens, Hq, Hk, d, rot, ldq, ldk), flags, dt, dev, lead


def _either(q, k):
    """The tensor whose device a call runs on."""
    if q is None and k is None:
        raise ValueError("one of q and k must be given")
    return q if q is not None else k


def _rope_out(t, out, dt, dev, name):
    """(output like t, pointer, elements from token to token)."""
    if t is None:
        if out is not None:
            raise ValueError(f"{name}: given without its input")
        return None, None, 0
    if out is None:
        out = _new(t, dt)
        return out, out.data_ptr(), t.shape[-1] * t.shape[-2]
    return out, *_strided(out, dt, t.shape, dev, name, 2)


def gdn_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, *, norm="rms",
                     eps=1e-6, scale=1.0, interleaved=False, q_out=None, k_out=None,
                     stream=None):
    """Norm of every head of q [..., Hq, d] and k [..., Hk, d] ("rms" with the weights [d]
    float32, "l2", or None) and the rotation of its first 2 * len(inv_freq) channels by
    positions [...] (int64) * inv_freq (float32; None: no rotation), in one pass; queries are
    multiplied by scale.  The leading axes are [T] or [B, T]; q and k may be slices of one
    projection's output, and one of them None.  Returns (q_out, k_out), which may be q and k."""
    return _rope_fwd(_either(q, k), q, k, positions, inv_freq, q_weight, k_weight,
                     norm, eps, scale, interleaved, q_out, k_out, stream=stream)


@_on_device
def _rope_fwd(_, q, k, positions, inv_freq, q_weight, k_weight, norm, eps, scale, interleaved,
              q_out, k_out):
    args, flags, dt, dev, lead = _rope_inputs(q, k, positions, inv_freq, q_weight, k_weight,
                                              norm, interleaved)
    q_out, *po = _rope_out(q, q_out, dt, dev, "q_out")
    k_out, *ko = _rope_out(k, k_out, dt, dev, "k_out")
    _check(lib.gdn_qk_norm_rope(*args, _dtype_code(dt), flags, eps, scale, *po, *ko,
                                _here(dev)), "gdn_qk_norm_rope")
    return q_out, k_out


def gdn_qk_norm_rope_bwd_workspace_bytes(tokens, Hq, Hk, d, norm="rms") -> int:
    """Bytes of device workspace gdn_qk_norm_rope_bwd needs for the weights' gradients."""
    return int(lib.gdn_qk_norm_rope_bwd_workspace_bytes(tokens, Hq, Hk, d, _norm_flag(norm)))


def gdn_qk_norm_rope_bwd(q, k, positions, inv_freq, q_weight, k_weight, dq_out, dk_out, *,
                         norm="rms", eps=1e-6, scale=1.0, interleaved=False, grad_f32=False,
                         workspace=None, stream=None):
    """Gradients of gdn_qk_norm_rope at its inputs q, k and weights, from those at its outputs
    (the input dtype, or float32 with grad_f32).  Returns a dict: dq, dk in the gradients'
    dtype, dq_weight, dk_weight [d] float32 (None where the weight is)."""
    return _rope_bwd(_either(q, k), q, k, positions, inv_freq, q_weight, k_weight,
                     dq_out, dk_out, norm, eps, scale, interleaved, grad_f32, workspace,
                     stream=stream)


@_on_device
def _rope_bwd(_, q, k, positions, inv_freq, q_weight, k_weight, dq_out, dk_out, norm, eps, scale,
              interleaved, grad_f32, workspace):
    args, flags, dt, dev, lead = _rope_inputs(q, k, positions, inv_freq, q_weight, k_weight,
                                              norm, interleaved)
    tokens, Hq, Hk, d = args[6:10]
    gdt = torch.float32 if grad_f32 else dt
    gq = _strided(dq_out, gdt, () if q is None else q.shape, dev, "dq_out", 2)
    gk = _strided(dk_out, gdt, () if k is None else k.shape, dev, "dk_out", 2)
    out = {"dq": None if q is None else _new(q, gdt), "dk": None if k is None else _new(k, gdt)}
    for name, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        out[name] = None if w is None else torch.empty_like(w)
    need = 0
    if q_weight is not None or k_weight is not None:
        need = lib.gdn_qk_norm_rope_bwd_workspace_bytes(tokens, Hq, Hk, d, flags)
    keep, ws, ws_bytes = _workspace(workspace, need, _either(q, k), dev)
    ptr = {n: None if v is None else v.data_ptr() for n, v in out.items()}
    _check(lib.gdn_qk_norm_rope_bwd(*args, *gq, *gk, _dtype_code(dt),
                                    flags | (GRAD_F32 if grad_f32 else 0), eps, scale,
                                    ptr["dq"], Hq * d, ptr["dk"], Hk * d, ptr["dq_weight"],
                                    ptr["dk_weight"], ws, ws_bytes,
                                    _here(dev)), "gdn_qk_norm_rope_bwd")
    return out


def gdn_check_status(stream=None):
    """Synchronise the stream and raise if a bounded device wait expired or an
    fp16 operand left its range since the last check."""
    _check(lib.gdn_check_status(_stream(stream)), "gdn_check_status")


def gdn_status(stream=None) -> int:
    """Synchronise the stream, read and clear the device status word: the raw
    gdn_check_status code (0 = GDN_OK, -4 = GDN_ERR_TIMEOUT, -6 = GDN_ERR_RANGE)."""
    return int(lib.gdn_check_status(_stream(stream)))


def gdn_test_set_wait_fault(site: int, spin_limit: int = 0):
    """Test hook: make the tensor-core chunk kernels leave one bounded wait to
    expire (site 1: the scan's first state hand-off, site 2: the prep's K / Q
    tiles, site 3: the chunk results in a cluster of the linear recurrence,
    site 4: its tiles; 0: none), with spin_limit polls per wait (0 = the default)."""
    _check(lib.gdn_test_set_wait_fault(int(site), int(spin_limit)), "gdn_test_set_wait_fault")
