"""Fused attention-distillation KL divergence for B200 (sm_100a).

Thin ctypes binding over the C ABI in ``include/streamkl.h`` (library
``libstreamkl.so`` next to this file).  Every step of the computation runs in
the library's CUDA kernels; this module only checks tensors, allocates outputs
with torch and passes raw pointers.  There is no CPU fallback: if the library
is missing or the device is not an sm_100 GPU, calls raise.

Functions keep the C names:
  streamkl_fwd(q_t, k_t, q_s, k_s, ...) -> (kl, lse_t, lse_s, loss_mean)
  streamkl_bwd(q_t, k_t, q_s, k_s, kl, lse_t, lse_s, ...) -> (dq_s, dk_s, dq_t, dk_t)
Keys may have fewer heads than the queries (grouped key heads: k_t
[B, H_kt, N_K, d_t], k_s [B, H_ks, N_K, d_s], each count dividing H), and
``kv_len`` (int32 [B] on the device) marks the keys at and past each batch
element's length as padding; either routes the call to the C ABI's
``streamkl_fwd_ex`` / ``streamkl_bwd_ex``.
Serving with a bounded key-value cache (bf16 or fp16, no gradients):
  streamkl_key_mass(q, k, lse, ...) -> (mass, lse): attention weight of every key
  streamkl_decode(q, k_pages, v_pages, page_table, seq_len, ...) -> (out, lse):
    one new token a sequence over a paged cache
  streamkl_evict(k_pages, v_pages, page_table, seq_len, mass, budget, ...) ->
    (new_len, mass, pos): keeps the tokens with the largest weight
The autograd wrapper with temperature scaling is in ``.autograd``
(``streamkl_loss``).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstreamkl.so")

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "device wait timeout",
          5: "workspace", 6: "access outside a tensor (bounds-checked build)"}


class StreamKLError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} (status {code})")
        self.code = code


_lib = None
_lock = threading.Lock()
_VP = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run `python -m attention_kl_divergence_attn_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            shape = [_I] * 6 + [_F, _F, _I]
            L.streamkl_fwd.argtypes = [_VP] * 4 + shape + [_VP] * 4 + [_VP, ctypes.c_size_t, _VP]
            L.streamkl_fwd.restype = _I
            L.streamkl_bwd.argtypes = ([_VP] * 4 + shape + [_VP] * 3 + [_VP, _F] + [_VP] * 4
                                       + [_VP, ctypes.c_size_t, _VP])
            L.streamkl_bwd.restype = _I
            L.streamkl_bwd_dk.argtypes = ([_VP] * 4 + shape + [_VP] * 3 + [_VP, _F] + [_VP] * 2
                                          + [_VP, ctypes.c_size_t, _VP])
            L.streamkl_bwd_dk.restype = _I
            L.streamkl_bwd_dq.argtypes = L.streamkl_bwd_dk.argtypes
            L.streamkl_bwd_dq.restype = _I
            L.streamkl_bwd_dloss_device.argtypes = ([_VP] * 4 + shape + [_VP] * 3 + [_VP, _VP, _F] + [_VP] * 4
                                                    + [_VP, ctypes.c_size_t, _VP])
            L.streamkl_bwd_dloss_device.restype = _I
            L.streamkl_loss_mean.argtypes = [_VP, ctypes.c_longlong, _VP, _VP]
            L.streamkl_loss_mean.restype = _I
            L.streamkl_loss_reduce.argtypes = [_VP, ctypes.c_longlong, ctypes.c_double, _VP, _VP]
            L.streamkl_loss_reduce.restype = _I
            shape_ex = [_I] * 8 + [_F, _F, _I, _VP]            # B, H, H_kt, H_ks, N_Q, N_K, d_t, d_s, ..., kv_len
            L.streamkl_fwd_ex.argtypes = [_VP] * 4 + shape_ex + [_VP] * 4 + [_VP, ctypes.c_size_t, _VP]
            L.streamkl_fwd_ex.restype = _I
            L.streamkl_bwd_ex.argtypes = ([_VP] * 4 + shape_ex + [_VP] * 3 + [_VP, _F, _VP] + [_VP] * 4 + [_I]
                                          + [_VP, ctypes.c_size_t, _VP])
            L.streamkl_bwd_ex.restype = _I
            L.streamkl_workspace_size_ex.argtypes = [_I] * 10
            L.streamkl_workspace_size_ex.restype = ctypes.c_size_t
            L.streamkl_key_mass.argtypes = ([_VP] * 4 + [_I] * 7 + [_F, _I] + [_VP] * 2 + [_I, _VP, _I]
                                            + [_VP, ctypes.c_size_t] * 2 + [_VP])
            L.streamkl_key_mass.restype = _I
            L.streamkl_key_mass_scratch_size.argtypes = [_I] * 7
            L.streamkl_key_mass_scratch_size.restype = ctypes.c_size_t
            L.streamkl_decode.argtypes = ([_VP] * 6 + [_I] * 7 + [_VP, _I, ctypes.c_longlong, _VP, _F]
                                          + [_VP] * 4 + [_I] + [_VP, ctypes.c_size_t] * 2 + [_VP])
            L.streamkl_decode.restype = _I
            L.streamkl_decode_scratch_size.argtypes = [_I] * 8
            L.streamkl_decode_scratch_size.restype = ctypes.c_size_t
            L.streamkl_evict.argtypes = ([_VP] * 4 + [_I] * 5 + [_VP, _I, ctypes.c_longlong] + [_VP] * 4 + [_I] * 3
                                         + [_VP] * 3 + [_VP, ctypes.c_size_t] * 2 + [_VP])
            L.streamkl_evict.restype = _I
            L.streamkl_evict_scratch_size.argtypes = [_I] * 7
            L.streamkl_evict_scratch_size.restype = ctypes.c_size_t
            L.streamkl_fwd_noalloc.argtypes = ([_VP] * 4 + shape + [_VP] * 4 + [_VP, ctypes.POINTER(ctypes.c_uint)])
            L.streamkl_fwd_noalloc.restype = _I
            L.streamkl_workspace_size.argtypes = [_I] * 7
            L.streamkl_workspace_size.restype = ctypes.c_size_t
            L.streamkl_workspace_init.argtypes = [_VP, ctypes.c_size_t, _VP]
            L.streamkl_workspace_init.restype = _I
            L.streamkl_check.argtypes = [_VP, _VP, ctypes.POINTER(ctypes.c_uint)]
            L.streamkl_check.restype = _I
            L.streamkl_selftest_timeout.argtypes = [_VP, ctypes.c_size_t, ctypes.c_ulonglong, _VP]
            L.streamkl_selftest_timeout.restype = _I
            L.streamkl_strerror.argtypes = [_I]
            L.streamkl_strerror.restype = ctypes.c_char_p
            L.streamkl_version.argtypes = []
            L.streamkl_version.restype = _I
            _lib = L
    return _lib


_workspaces: dict = {}
_ws_sizes: dict = {}
_STATUS_BYTES = 256


def workspace(device=None, nbytes=None) -> torch.Tensor:
    """This device's workspace, created and cleared on first use.

    Its first 256 bytes are the library's device status word.  ``nbytes``
    (from ``workspace_size``) grows it for problems whose kernels split key
    ranges; growing keeps the status word.  Calls through this module run on
    the current stream, so they are ordered and may share it.
    """
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index)
    need = max(int(nbytes or 0), _STATUS_BYTES)
    ws = _workspaces.get(dev.index)
    if ws is None or ws.numel() < need:
        new = torch.zeros(need, dtype=torch.uint8, device=dev)
        if ws is not None:
            new[:_STATUS_BYTES].copy_(ws[:_STATUS_BYTES])
        ws = new
        _workspaces[dev.index] = ws
    return ws


def workspace_size(B, H, N_Q, N_K, d_t, d_s, causal, H_kt=None, H_ks=None, teacher_grads=False) -> int:
    """streamkl_workspace_size(_ex) for this problem on the current device (cached)."""
    H_kt = H if H_kt is None else H_kt
    H_ks = H if H_ks is None else H_ks
    key = (torch.cuda.current_device(), B, H, H_kt, H_ks, N_Q, N_K, d_t, d_s, int(bool(causal)),
           int(bool(teacher_grads)))
    n = _ws_sizes.get(key)
    if n is None:
        if H_kt == H and H_ks == H:
            n = int(lib().streamkl_workspace_size(B, H, N_Q, N_K, d_t, d_s, int(bool(causal))))
        else:
            n = int(lib().streamkl_workspace_size_ex(B, H, H_kt, H_ks, N_Q, N_K, d_t, d_s, int(bool(causal)),
                                                     int(bool(teacher_grads))))
        _ws_sizes[key] = n
    return n


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_inputs(q_t, k_t, q_s, k_s):
    for name, t in (("q_t", q_t), ("k_t", k_t), ("q_s", q_s), ("k_s", k_s)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA bf16 tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    B, H, N_Q, d_t = q_t.shape
    H_kt, N_K = k_t.shape[1], k_t.shape[2]
    d_s = q_s.shape[3]
    H_ks = k_s.shape[1]
    if k_t.shape != (B, H_kt, N_K, d_t) or q_s.shape != (B, H, N_Q, d_s) or k_s.shape != (B, H_ks, N_K, d_s):
        raise ValueError("inconsistent shapes of q_t, k_t, q_s, k_s")
    if H_kt < 1 or H_ks < 1 or H % H_kt or H % H_ks:
        raise ValueError("the key heads of k_t and k_s must each divide the query heads")
    return B, H, N_Q, N_K, d_t, d_s, H_kt, H_ks


def _check_lengths(kv_len, B, device):
    if kv_len is None:
        return None
    if (not isinstance(kv_len, torch.Tensor) or kv_len.dtype != torch.int32 or kv_len.device != device
            or kv_len.numel() != B or not kv_len.is_contiguous()):
        raise ValueError("kv_len must be a contiguous int32 tensor of B lengths on the inputs' device")
    return kv_len


def streamkl_fwd(q_t, k_t, q_s, k_s, scale_t=None, scale_s=None, causal=False, *, loss_mean=True,
                 out=None, stream=None, kv_len=None):
    """Per-row KL(P_teacher || Q_student), both log-sum-exps and the mean loss.

    Returns (kl, lse_t, lse_s, loss) with kl/lse_* fp32 [B, H, N_Q] and loss a
    0-d fp32 device tensor (None if loss_mean=False).  ``out`` may supply the
    three per-row buffers (and optionally a 4th, the loss scalar).  A row with
    no visible key (all keys padding) gets KL = 0 and LSE = -inf.
    """
    B, H, N_Q, N_K, d_t, d_s, H_kt, H_ks = _check_inputs(q_t, k_t, q_s, k_s)
    kv_len = _check_lengths(kv_len, B, q_t.device)
    scale_t = 1.0 / math.sqrt(d_t) if scale_t is None else float(scale_t)
    scale_s = 1.0 / math.sqrt(d_s) if scale_s is None else float(scale_s)
    dev = q_t.device
    if out is None:
        kl = torch.empty(B, H, N_Q, dtype=torch.float32, device=dev)
        lse_t = torch.empty_like(kl)
        lse_s = torch.empty_like(kl)
        loss = torch.empty((), dtype=torch.float32, device=dev) if loss_mean else None
    else:
        kl, lse_t, lse_s = out[:3]
        loss = (out[3] if len(out) > 3 else torch.empty((), dtype=torch.float32, device=dev)) if loss_mean else None
    ws = workspace(dev, workspace_size(B, H, N_Q, N_K, d_t, d_s, causal))
    if H_kt == H and H_ks == H and kv_len is None:
        rc = lib().streamkl_fwd(_ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, N_Q, N_K, d_t, d_s,
                                scale_t, scale_s, int(bool(causal)), _ptr(kl), _ptr(lse_t), _ptr(lse_s),
                                _ptr(loss), _ptr(ws), ws.numel(), _stream(stream))
        if rc:
            raise StreamKLError("streamkl_fwd", rc)
        return kl, lse_t, lse_s, loss
    rc = lib().streamkl_fwd_ex(_ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, H_kt, H_ks, N_Q, N_K, d_t, d_s,
                               scale_t, scale_s, int(bool(causal)), _ptr(kv_len), _ptr(kl), _ptr(lse_t),
                               _ptr(lse_s), _ptr(loss), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise StreamKLError("streamkl_fwd_ex", rc)
    return kl, lse_t, lse_s, loss


_PART_DK, _PART_DQ = 1, 2


def _bwd_ex(parts, q_t, k_t, q_s, k_s, kl, lse_t, lse_s, shape, scale_t, scale_s, causal, kv_len, dkl,
            dloss, dloss_scale, grads, stream):
    """streamkl_bwd_ex: grouped key heads and/or padding (grads = dq_s, dk_s, dq_t, dk_t)."""
    B, H, N_Q, N_K, d_t, d_s, H_kt, H_ks = shape
    teacher = grads[2] is not None or grads[3] is not None
    ws = workspace(q_t.device, workspace_size(B, H, N_Q, N_K, d_t, d_s, causal, H_kt, H_ks, teacher))
    if isinstance(dloss, torch.Tensor):
        if dloss.dtype != torch.float32 or dloss.numel() != 1 or dloss.device != q_t.device:
            raise ValueError("a tensor dloss must be a one-element fp32 tensor on the inputs' device")
        scale, dev_ptr = (1.0 / (B * H * N_Q) if dloss_scale is None else float(dloss_scale)), _ptr(dloss)
    else:
        if dloss_scale is not None:
            raise ValueError("dloss_scale applies to a device-tensor dloss only")
        scale, dev_ptr = float(dloss), None
    rc = lib().streamkl_bwd_ex(_ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, H_kt, H_ks, N_Q, N_K, d_t, d_s,
                               scale_t, scale_s, int(bool(causal)), _ptr(kv_len), _ptr(kl), _ptr(lse_t),
                               _ptr(lse_s), _ptr(dkl), scale, dev_ptr, *[_ptr(g) for g in grads], parts,
                               _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise StreamKLError("streamkl_bwd_ex", rc)


def streamkl_bwd(q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t=None, scale_s=None, causal=False, *,
                 dkl=None, dloss=1.0, dloss_scale=None, teacher_grads=False, out=None, stream=None, kv_len=None):
    """Gradients of sum_i g_i KL_i with g = dkl, or of dloss * mean(KL) if dkl is None.

    ``dloss`` is a number or a 0-d CUDA fp32 tensor; a tensor stays on the
    device (streamkl_bwd_dloss_device) and then g = dloss_scale * dloss, with
    dloss_scale defaulting to 1 / (B*H*N_Q).  Returns (dq_s, dk_s, dq_t,
    dk_t), fp32, the teacher pair None unless teacher_grads.  ``out`` may
    supply the four buffers.  With grouped key heads dk_s, dk_t have the key
    tensors' shapes (each key head's gradient sums over its query heads).
    """
    shape = _check_inputs(q_t, k_t, q_s, k_s)
    B, H, N_Q, N_K, d_t, d_s, H_kt, H_ks = shape
    kv_len = _check_lengths(kv_len, B, q_t.device)
    scale_t = 1.0 / math.sqrt(d_t) if scale_t is None else float(scale_t)
    scale_s = 1.0 / math.sqrt(d_s) if scale_s is None else float(scale_s)
    for name, t in (("kl", kl), ("lse_t", lse_t), ("lse_s", lse_s)) + ((("dkl", dkl),) if dkl is not None else ()):
        if t.dtype != torch.float32 or t.numel() != B * H * N_Q or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 [B, H, N_Q] tensor")
    dev = q_t.device
    if out is None:
        dq_s = torch.empty(B, H, N_Q, d_s, dtype=torch.float32, device=dev)
        dk_s = torch.empty(B, H_ks, N_K, d_s, dtype=torch.float32, device=dev)
        dq_t = torch.empty(B, H, N_Q, d_t, dtype=torch.float32, device=dev) if teacher_grads else None
        dk_t = torch.empty(B, H_kt, N_K, d_t, dtype=torch.float32, device=dev) if teacher_grads else None
    else:
        dq_s, dk_s, dq_t, dk_t = out
    if H_kt != H or H_ks != H or kv_len is not None:
        _bwd_ex(_PART_DK | _PART_DQ, q_t, k_t, q_s, k_s, kl, lse_t, lse_s, shape, scale_t, scale_s, causal, kv_len,
                dkl, dloss, dloss_scale, (dq_s, dk_s, dq_t, dk_t), stream)
        return dq_s, dk_s, dq_t, dk_t
    ws = workspace(dev, workspace_size(B, H, N_Q, N_K, d_t, d_s, causal))
    if isinstance(dloss, torch.Tensor):
        if dloss.dtype != torch.float32 or dloss.numel() != 1 or dloss.device != dev:
            raise ValueError("a tensor dloss must be a one-element fp32 tensor on the inputs' device")
        scale = 1.0 / (B * H * N_Q) if dloss_scale is None else float(dloss_scale)
        rc = lib().streamkl_bwd_dloss_device(
            _ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, N_Q, N_K, d_t, d_s, scale_t, scale_s,
            int(bool(causal)), _ptr(kl), _ptr(lse_t), _ptr(lse_s), _ptr(dkl), _ptr(dloss), scale,
            _ptr(dq_s), _ptr(dk_s), _ptr(dq_t), _ptr(dk_t), _ptr(ws), ws.numel(), _stream(stream))
        if rc:
            raise StreamKLError("streamkl_bwd_dloss_device", rc)
        return dq_s, dk_s, dq_t, dk_t
    if dloss_scale is not None:
        raise ValueError("dloss_scale applies to a device-tensor dloss only")
    rc = lib().streamkl_bwd(_ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, N_Q, N_K, d_t, d_s,
                            scale_t, scale_s, int(bool(causal)), _ptr(kl), _ptr(lse_t), _ptr(lse_s),
                            _ptr(dkl), float(dloss), _ptr(dq_s), _ptr(dk_s), _ptr(dq_t), _ptr(dk_t),
                            _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise StreamKLError("streamkl_bwd", rc)
    return dq_s, dk_s, dq_t, dk_t


def _bwd_part(fn, which, q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t, scale_s, causal, dkl, dloss,
              teacher_grads, out, stream, kv_len=None):
    shape = _check_inputs(q_t, k_t, q_s, k_s)
    B, H, N_Q, N_K, d_t, d_s, H_kt, H_ks = shape
    kv_len = _check_lengths(kv_len, B, q_t.device)
    scale_t = 1.0 / math.sqrt(d_t) if scale_t is None else float(scale_t)
    scale_s = 1.0 / math.sqrt(d_s) if scale_s is None else float(scale_s)
    dev = q_t.device
    if out is None:
        n_s, n_t = (H_ks, H_kt) if which == "k" else (H, H)
        n = N_K if which == "k" else N_Q
        g_s = torch.empty(B, n_s, n, d_s, dtype=torch.float32, device=dev)
        g_t = torch.empty(B, n_t, n, d_t, dtype=torch.float32, device=dev) if teacher_grads else None
    else:
        g_s, g_t = out
    if H_kt != H or H_ks != H or kv_len is not None:
        grads = (None, g_s, None, g_t) if which == "k" else (g_s, None, g_t, None)
        _bwd_ex(_PART_DK if which == "k" else _PART_DQ, q_t, k_t, q_s, k_s, kl, lse_t, lse_s, shape, scale_t,
                scale_s, causal, kv_len, dkl, dloss, None, grads, stream)
        return g_s, g_t
    ws = workspace(dev, workspace_size(B, H, N_Q, N_K, d_t, d_s, causal))
    rc = getattr(lib(), fn)(_ptr(q_t), _ptr(k_t), _ptr(q_s), _ptr(k_s), B, H, N_Q, N_K, d_t, d_s,
                            scale_t, scale_s, int(bool(causal)), _ptr(kl), _ptr(lse_t), _ptr(lse_s),
                            _ptr(dkl), float(dloss), _ptr(g_s), _ptr(g_t), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise StreamKLError(fn, rc)
    return g_s, g_t


def streamkl_bwd_dk(q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t=None, scale_s=None, causal=False, *,
                    dkl=None, dloss=1.0, teacher_grads=False, out=None, stream=None, kv_len=None):
    """Key gradients only: (dk_s, dk_t), the teacher one None unless teacher_grads."""
    return _bwd_part("streamkl_bwd_dk", "k", q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t, scale_s, causal,
                     dkl, dloss, teacher_grads, out, stream, kv_len)


def streamkl_bwd_dq(q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t=None, scale_s=None, causal=False, *,
                    dkl=None, dloss=1.0, teacher_grads=False, out=None, stream=None, kv_len=None):
    """Query gradients only: (dq_s, dq_t), the teacher one None unless teacher_grads."""
    return _bwd_part("streamkl_bwd_dq", "q", q_t, k_t, q_s, k_s, kl, lse_t, lse_s, scale_t, scale_s, causal,
                     dkl, dloss, teacher_grads, out, stream, kv_len)


def streamkl_loss_mean(kl, out=None, stream=None):
    """Deterministic mean of a contiguous fp32 per-row KL tensor, as a 0-d device tensor."""
    if kl.dtype != torch.float32 or not kl.is_cuda or not kl.is_contiguous():
        raise TypeError("kl must be a contiguous CUDA fp32 tensor")
    out = torch.empty((), dtype=torch.float32, device=kl.device) if out is None else out
    rc = lib().streamkl_loss_mean(_ptr(kl), kl.numel(), _ptr(out), _stream(stream))
    if rc:
        raise StreamKLError("streamkl_loss_mean", rc)
    return out


def streamkl_loss_reduce(kl, factor, out=None, stream=None):
    """factor * sum(kl) (fixed order, fp64 accumulation) as a 0-d device tensor."""
    if kl.dtype != torch.float32 or not kl.is_cuda or not kl.is_contiguous():
        raise TypeError("kl must be a contiguous CUDA fp32 tensor")
    out = torch.empty((), dtype=torch.float32, device=kl.device) if out is None else out
    rc = lib().streamkl_loss_reduce(_ptr(kl), kl.numel(), float(factor), _ptr(out), _stream(stream))
    if rc:
        raise StreamKLError("streamkl_loss_reduce", rc)
    return out


# ---------------------------------------------------------------- cache operators
# Serving calls take a few microseconds on the GPU, so what a call's shapes,
# strides and types decide (the checks, the scratch size, the stride arrays) is
# worked out once for each combination and looked up after that.
_words: dict = {}
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _status_word(dev):
    """Address of the cache operators' status word on device index `dev`: 256 bytes that are never replaced,
    so that a captured graph's pointer to them stays good."""
    w = _words.get(dev)
    if w is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first cache operator on a device must run before a graph capture")
        with _lock:
            w = _words.get(dev)
            if w is None:
                w = torch.zeros(_STATUS_BYTES, dtype=torch.uint8, device=torch.device("cuda", dev))
                torch.cuda.current_stream(dev).synchronize()   # cleared before any stream uses it
                _words[dev] = w
    return w.data_ptr()


def _current_stream(dev):
    return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream


def _on(dev, stream):
    """Context that makes the call's device and stream current, or None when they are."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return None if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _sig(t):
    """What the checks of a tensor depend on (None, and what is not a tensor, stand for themselves)."""
    if t is None:
        return None
    try:
        return t.dtype, t.get_device(), t.shape, t.stride()
    except AttributeError:
        return type(t)


class _Meta:
    """A signature with a tensor's attributes, for the checks."""

    def __init__(self, sig):
        self.dtype, self.device, self.shape, self._stride = sig
        self.numel = math.prod(self.shape)

    def stride(self, i):
        return self._stride[i]

    def contiguous(self):
        n = 1
        for size, s in zip(reversed(self.shape), reversed(self._stride)):
            if size > 1 and s != n:
                return self.numel == 0
            n *= size
        return True


def _meta(sig):
    return _Meta(sig) if isinstance(sig, tuple) else None


def _check_rows(name, sig, ndim, like=None):
    """A CUDA 16-bit tensor whose rows (last dimension) are contiguous and 16-byte aligned."""
    t = _meta(sig)
    if t is None or t.dtype not in _DTYPES or t.device < 0:
        raise TypeError(f"{name} must be a CUDA bf16 or fp16 tensor")
    if len(t.shape) != ndim or (t.stride(-1) != 1 and t.numel > 0):
        raise ValueError(f"{name} must have {ndim} dimensions, the last one contiguous")
    if t.numel > 0 and any(n > 1 and (s % 8 or s <= 0) for n, s in zip(t.shape[:-1], t._stride)):
        raise ValueError(f"{name} must have strides in positive multiples of 8 (rows on 16-byte boundaries)")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must have the type and device of the other tensors")
    return t


def _check_vec(name, sig, dtype, shape, dev):
    t = _meta(sig)
    if t is None or t.dtype != dtype or t.device != dev or t.shape != torch.Size(shape) or not t.contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor {list(shape)} on the inputs' device")


def _check_pages(k_pages, v_pages, page_table, seq_len, like=None):
    k = _check_rows("k_pages", k_pages, 4, like)
    v = _check_rows("v_pages", v_pages, 4, k)
    if k.shape != v.shape:
        raise ValueError("k_pages and v_pages must have one shape [pages, H_k, page_size, d]")
    if k.shape[1] < 1 or k.shape[2] < 1:
        raise ValueError("k_pages must have a key head and a slot a page")
    t = _meta(page_table)
    if (t is None or t.dtype != torch.int32 or t.device != k.device or len(t.shape) != 2
            or (t.shape[1] > 1 and t.stride(1) != 1)):
        raise ValueError("page_table must be an int32 tensor [B, max_pages] with contiguous rows on the inputs' device")
    _check_vec("seq_len", seq_len, torch.int32, (t.shape[0],), k.device)
    return k, v, t


def _scratch_bytes(dev, fn, *args):
    with torch.cuda.device(dev):                               # (it depends on the device's size)
        return int(getattr(lib(), fn)(*args))


def _longs(s):
    return (ctypes.c_longlong * len(s))(*s)


def _span(t):
    """Addresses of the first byte and past the last (strides are positive here)."""
    p = t.data_ptr()
    if t.numel() == 0:
        return p, p
    return p, p + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _overlap(a, b):
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _refused(fn, rc, outs, ins, changed=()):
    """Raises for a call that the library refused; overlaps, which it looks for, are named here.  `changed`: tensors
    changed in place, which may lie between each other."""
    outs, ins, changed = [[t for t in x if t is not None] for x in (outs, ins, changed)]
    if rc == 1 and (any(_overlap(o, i) for o in outs + changed for i in ins)
                    or any(_overlap(o, t) for n, o in enumerate(outs) for t in outs[:n] + changed)):
        raise ValueError("outputs must not overlap inputs or each other")
    raise StreamKLError(fn, rc)


@functools.lru_cache(maxsize=4096)
def _key_mass_plan(q_sig, k_sig, lse_sig, len_sig, out_sig, accumulate):
    q = _check_rows("q", q_sig, 4)
    k = _check_rows("k", k_sig, 4, q)
    B, H, N_Q, d = q.shape
    H_k, N_K = k.shape[1], k.shape[2]
    if k.shape != (B, H_k, N_K, d):
        raise ValueError("inconsistent shapes of q and k")
    if H_k < 1 or H % H_k:
        raise ValueError("the key heads must divide the query heads")
    if accumulate and out_sig is None:
        raise ValueError("accumulate needs out, the sums to add to")
    dev = q.device
    if len_sig is not None:
        _check_vec("kv_len", len_sig, torch.int32, (B,), dev)
    if lse_sig is not None:
        _check_vec("lse", lse_sig, torch.float32, (B, H, N_Q), dev)
    if out_sig is not None:
        _check_vec("out", out_sig, torch.float32, (B, H_k, N_K), dev)
    given = int(lse_sig is not None)
    nbytes = _scratch_bytes(dev, "streamkl_key_mass_scratch_size", B, H, H_k, N_Q, N_K, d, given)
    return (dev, torch.device("cuda", dev), (B, H_k, N_K), (B, H, N_Q), nbytes, 1.0 / math.sqrt(max(d, 1)),
            _longs(q._stride[:3]), _longs(k._stride[:3]), (_DTYPES[q.dtype], B, H, H_k, N_Q, N_K, d))


def streamkl_key_mass(q, k, lse=None, scale=None, causal=False, *, kv_len=None, out=None, accumulate=False,
                      stream=None):
    """Attention weight that every key receives from the query rows: (mass, lse).

    q [B, H, N_Q, d], k [B, H_k, N_K, d] (bf16 or fp16, d in {64, 128}, H_k
    dividing H; rows contiguous, other strides free).  mass fp32 [B, H_k, N_K]
    = the column sums of softmax(scale q k^T), summed over each key head's
    query heads.  ``lse`` fp32 [B, H, N_Q] are the rows' log-sum-exps if they
    are at hand (lse_t of ``streamkl_fwd`` for the teacher's q and k, same
    scale, mask and lengths); otherwise they are computed and returned.
    ``causal`` and ``kv_len`` as in ``streamkl_fwd``; a row without a visible
    key adds nothing.  ``out`` supplies mass and must not overlap another
    tensor; with ``accumulate`` the call adds to it (the pieces of a long
    prompt).  Gradients do not flow.
    """
    dev, device, mass_shape, row_shape, nbytes, default, qs, ks, sizes = _key_mass_plan(
        _sig(q), _sig(k), _sig(lse), _sig(kv_len), _sig(out), bool(accumulate))
    on = _on(dev, stream)
    if on is not None:
        with on:
            return streamkl_key_mass(q, k, lse, scale, causal, kv_len=kv_len, out=out, accumulate=accumulate)
    word = _status_word(dev)
    mass = torch.empty(mass_shape, dtype=torch.float32, device=device) if out is None else out
    given = lse is not None
    if not given:
        lse = torch.empty(row_shape, dtype=torch.float32, device=device)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    rc = lib().streamkl_key_mass(q.data_ptr(), qs, k.data_ptr(), ks, *sizes, default if scale is None else float(scale),
                                 1 if causal else 0, None if kv_len is None else kv_len.data_ptr(), lse.data_ptr(),
                                 given, mass.data_ptr(), 1 if accumulate else 0, word, _STATUS_BYTES,
                                 None if scratch is None else scratch.data_ptr(), nbytes, _current_stream(dev))
    if rc:
        _refused("streamkl_key_mass", rc, (mass, None if given else lse), (q, k, kv_len, lse if given else None))
    return mass, lse


@functools.lru_cache(maxsize=4096)
def _decode_plan(q_sig, k_sig, v_sig, table_sig, len_sig, mass_sig, mass_out_sig, outs, o_sig, lse_sig):
    q = _check_rows("q", q_sig, 3)
    k, v, table = _check_pages(k_sig, v_sig, table_sig, len_sig, q)
    dev = q.device
    B, H, d = q.shape
    pages, H_k, page, dk = k.shape
    if dk != d or table.shape[0] != B:
        raise ValueError("inconsistent shapes of q, k_pages and page_table")
    if H % H_k:
        raise ValueError("the key heads must divide the query heads")
    cap = 0
    if mass_sig is not None:
        m = _meta(mass_sig)
        cap = m.shape[-1] if m is not None and len(m.shape) == 3 else 0
        _check_vec("mass", mass_sig, torch.float32, (B, H_k, cap), dev)
        if cap == 0 and table.shape[1] > 0:
            raise ValueError("mass must have a column for every slot that a sequence may use")
        if mass_out_sig is not None:
            _check_vec("mass_out", mass_out_sig, torch.float32, (B, H_k, cap), dev)
    elif mass_out_sig is not None:
        raise ValueError("mass_out needs mass")
    if outs:
        _check_vec("out[0]", o_sig, q.dtype, (B, H, d), dev)
        _check_vec("out[1]", lse_sig, torch.float32, (B, H), dev)
    max_pages = table.shape[1]
    nbytes = _scratch_bytes(dev, "streamkl_decode_scratch_size", B, H, H_k, page, max_pages, d,
                            int(mass_sig is not None), cap)
    return (dev, torch.device("cuda", dev), (B, H), nbytes, 1.0 / math.sqrt(max(d, 1)), _longs(q._stride[:2]),
            _longs(k._stride[:3]), _longs(v._stride[:3]), (_DTYPES[q.dtype], B, H, H_k, d, pages, page), max_pages,
            table.stride(0), cap)


def streamkl_decode(q, k_pages, v_pages, page_table, seq_len, scale=None, *, mass=None, mass_out=None, out=None,
                    stream=None):
    """Attention of one new token a sequence over a paged key-value cache: (out, lse).

    q [B, H, d]; k_pages, v_pages [pages, H_k, page_size, d] (bf16 or fp16,
    rows contiguous, other strides free: a token-major cache is its
    transposed view); page_table int32 [B, max_pages]; seq_len int32 [B].
    Slot t of sequence b is slot t % page_size of page page_table[b, t //
    page_size].  out [B, H, d] has q's type, lse is fp32 [B, H]; a sequence of
    length 0 gets 0 and -inf.  ``mass`` fp32 [B, H_k, n] accumulates the
    tokens' weights, summed over each key head's query heads: in place, or
    into ``mass_out`` (mass itself then stays as it was).  ``out`` may supply
    the (out, lse) buffers; no output may overlap another tensor.  Bad lengths
    and pages are reported by ``streamkl_check``.  Gradients do not flow.
    """
    o, lse = (None, None) if out is None else out
    dev, device, row_shape, nbytes, default, qs, ks, vs, sizes, max_pages, table_stride, cap = _decode_plan(
        _sig(q), _sig(k_pages), _sig(v_pages), _sig(page_table), _sig(seq_len), _sig(mass), _sig(mass_out),
        out is not None, _sig(o), _sig(lse))
    on = _on(dev, stream)
    if on is not None:
        with on:
            return streamkl_decode(q, k_pages, v_pages, page_table, seq_len, scale, mass=mass, mass_out=mass_out,
                                   out=out)
    mass_ptr = mass_out_ptr = None
    if mass is not None:
        mass_ptr = mass_out_ptr = mass.data_ptr()
        if mass_out is not None:
            mass_out_ptr = mass_out.data_ptr()
    word = _status_word(dev)
    if out is None:
        o, lse = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(row_shape, dtype=torch.float32,
                                                                                        device=device)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    rc = lib().streamkl_decode(q.data_ptr(), qs, k_pages.data_ptr(), ks, v_pages.data_ptr(), vs, *sizes,
                               page_table.data_ptr(), max_pages, table_stride, seq_len.data_ptr(),
                               default if scale is None else float(scale), o.data_ptr(), lse.data_ptr(), mass_ptr,
                               mass_out_ptr, cap, word, _STATUS_BYTES,
                               None if scratch is None else scratch.data_ptr(), nbytes, _current_stream(dev))
    if rc:
        _refused("streamkl_decode", rc, (o, lse, mass if mass_out is None else mass_out),
                 (q, k_pages, v_pages, page_table, seq_len, None if mass_out_ptr == mass_ptr else mass))
    return o, lse


@functools.lru_cache(maxsize=4096)
def _evict_plan(k_sig, v_sig, table_sig, len_sig, mass_sig, pos_sig, next_sig, out_sigs, budget, recent):
    k, v, table = _check_pages(k_sig, v_sig, table_sig, len_sig)
    dev = k.device
    pages, H_k, page, d = k.shape
    B, max_pages = table.shape
    if budget < 0 or recent < 0 or recent > budget:
        raise ValueError("budget and recent must satisfy 0 <= recent <= budget")
    budget, recent = min(budget, 0x7fffffff), min(recent, 0x7fffffff)
    m = _meta(mass_sig)
    cap = m.shape[-1] if m is not None and len(m.shape) == 3 else 0
    _check_vec("mass", mass_sig, torch.float32, (B, H_k, cap), dev)
    if pos_sig is not None:
        _check_vec("pos", pos_sig, torch.int32, (B, H_k, cap), dev)
    if next_sig is not None:
        _check_vec("next_pos", next_sig, torch.int32, (B,), dev)
    if recent > 0 and (pos_sig is None or next_sig is None):
        raise ValueError("recent needs pos and next_pos")
    if out_sigs is not None:
        _check_vec("out[0]", out_sigs[0], torch.int32, (B,), dev)
        _check_vec("out[1]", out_sigs[1], torch.float32, (B, H_k, cap), dev)
        if (out_sigs[2] is None) != (pos_sig is None):
            raise ValueError("out[2] goes with pos")
        if pos_sig is not None:
            _check_vec("out[2]", out_sigs[2], torch.int32, (B, H_k, cap), dev)
    nbytes = _scratch_bytes(dev, "streamkl_evict_scratch_size", B, H_k, pages, page, max_pages, cap, budget)
    return (dev, torch.device("cuda", dev), (B,), max(nbytes, 16), _longs(k._stride[:3]), _longs(v._stride[:3]),
            (B, H_k, d, pages, page), max_pages, table.stride(0), (cap, budget, recent))


def streamkl_evict(k_pages, v_pages, page_table, seq_len, mass, budget, *, recent=0, pos=None, next_pos=None,
                   out=None, stream=None):
    """Keeps min(seq_len, budget) tokens of every (sequence, key head): (new_len, mass, pos).

    The cache is ``streamkl_decode``'s and is changed in place; mass fp32
    [B, H_k, n] are the accumulated weights.  Kept are the ``recent`` newest
    tokens (pos >= next_pos - recent; pos int32 [B, H_k, n] holds the position
    of each slot's token, next_pos int32 [B] the next token's) and those with
    the largest weight, the lower slot first among equals.  Kept tokens past
    the new length move into the slots of evicted ones before it; mass and pos
    are returned in the new order (0 and -1 past new_len), as new tensors or
    in ``out`` = (new_len, mass, pos), which must not overlap another tensor.  pos
    is None if none is given.  A sequence that shares pages with another one
    is left as it is and reported by ``streamkl_check``.
    """
    dev, device, len_shape, nbytes, ks, vs, sizes, max_pages, table_stride, tail = _evict_plan(
        _sig(k_pages), _sig(v_pages), _sig(page_table), _sig(seq_len), _sig(mass), _sig(pos), _sig(next_pos),
        None if out is None else tuple(_sig(o) for o in out), int(budget), int(recent))
    on = _on(dev, stream)
    if on is not None:
        with on:
            return streamkl_evict(k_pages, v_pages, page_table, seq_len, mass, budget, recent=recent, pos=pos,
                                  next_pos=next_pos, out=out)
    if k_pages.data_ptr() == v_pages.data_ptr() and k_pages.numel():
        raise ValueError("k_pages and v_pages must be two tensors")
    word = _status_word(dev)
    if out is None:
        new_len = torch.empty(len_shape, dtype=torch.int32, device=device)
        mass_out = torch.empty_like(mass)
        pos_out = None if pos is None else torch.empty_like(pos)
    else:
        new_len, mass_out, pos_out = out
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=device)
    rc = lib().streamkl_evict(k_pages.data_ptr(), ks, v_pages.data_ptr(), vs, *sizes, page_table.data_ptr(),
                              max_pages, table_stride, seq_len.data_ptr(), mass.data_ptr(),
                              None if pos is None else pos.data_ptr(),
                              None if next_pos is None else next_pos.data_ptr(), *tail, new_len.data_ptr(),
                              mass_out.data_ptr(), None if pos_out is None else pos_out.data_ptr(), word,
                              _STATUS_BYTES, scratch.data_ptr(), nbytes, _current_stream(dev))
    if rc:
        _refused("streamkl_evict", rc, (new_len, mass_out, pos_out), (page_table, seq_len, mass, pos, next_pos),
                 (k_pages, v_pages))
    return new_len, mass_out, pos_out


def streamkl_check(stream=None, device=None) -> int:
    """Synchronises and raises if a kernel gave up on a bounded wait; returns the status word."""
    ws = workspace(device)
    codes = []
    for w in (ws, _words.get(ws.device.index)):
        if w is None:
            continue
        code = ctypes.c_uint(0)
        rc = lib().streamkl_check(_ptr(w), _stream(stream), ctypes.byref(code))
        codes.append((rc, code.value))
    for rc, _ in codes:
        if rc:
            raise StreamKLError("streamkl_check", rc)
    return codes[0][1] | codes[-1][1]
