"""Python binding of libgdn.so (C ABI in include/gdn.h), with the same entry-point names.

Argument marshalling only: every step of the operator runs in the HIP kernels of the
library. torch supplies device memory and the current stream. There is no CPU path: a
missing library, or a tensor that is not on a GPU, raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
_DTYPE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
CHUNK = 64

# (name, restype, argtypes) of every function declared in include/gdn.h
_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F = ctypes.c_int64, ctypes.c_float
_SIGNATURES = [
    ("gdn_version", _I, []),
    ("gdn_status_string", ctypes.c_char_p, [_I]),
    ("gdn_chunk_fwd_workspace_bytes", _SZ, [_I] * 9),
    ("gdn_chunk_fwd", _I, [_P] * 9 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_chunk_fwd_noalloc", _I, [_P] * 9 + [_I] * 9 + [_P]),
    ("gdn_chunk_prepare", _I, [_P] * 5 + [_I] * 8 + [_P, _SZ, _P]),
    ("gdn_chunk_propagate", _I, [_P] * 7 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_decode_step", _I, [_P] * 7 + [_I] * 6 + [_P]),
    ("gdn_chunk_bwd_workspace_bytes", _SZ, [_I] * 9),
    ("gdn_chunk_bwd", _I, [_P] * 15 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_kda_chunk_fwd_workspace_bytes", _SZ, [_I] * 9),
    ("gdn_kda_chunk_fwd", _I, [_P] * 9 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_kda_chunk_bwd_workspace_bytes", _SZ, [_I] * 9),
    ("gdn_kda_chunk_bwd", _I, [_P] * 15 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_kda_decode_step", _I, [_P] * 7 + [_I] * 6 + [_P]),
    ("gdn_decoupled_chunk_fwd", _I, [_P] * 10 + [_I] * 9 + [_P, _SZ, _P]),
    ("gdn_decoupled_decode_step", _I, [_P] * 8 + [_I] * 6 + [_P]),
    ("gdn_recurrent_fwd", _I, [_P] * 10 + [_I] * 7 + [_L] * 3 + [_I] * 3 + [_P]),
    ("gdn_qk_norm_fwd", _I, [_P] * 8 + [_I] * 4 + [_L] * 4 + [_I, _F, _I, _I, _F, _F, _I, _I, _P]),
    ("gdn_qk_norm_bwd_workspace_bytes", _SZ, [_I] * 4),
    ("gdn_qk_norm_bwd", _I, [_P] * 12 + [_I] * 4 + [_L] * 8 + [_I, _F, _I, _I, _F, _F, _I, _I, _P, _SZ, _P]),
    ("gdn_layer_norm_fwd", _I, [_P] * 6 + [_I] * 2 + [_L] * 2 + [_F] + [_I] * 3 + [_P]),
    ("gdn_layer_norm_bwd_workspace_bytes", _SZ, [_I] * 2),
    ("gdn_layer_norm_bwd", _I, [_P] * 7 + [_I] * 2 + [_L, _F] + [_I] * 2 + [_P, _SZ, _P]),
    ("gdn_conv_fwd", _I, [_P] * 7 + [_I] * 5 + [_L] + [_I] * 2 + [_P]),
    ("gdn_conv_bwd_workspace_bytes", _SZ, [_I] * 4),
    ("gdn_conv_bwd", _I, [_P] * 11 + [_I] * 5 + [_L] * 2 + [_I] * 2 + [_P, _SZ, _P]),
    ("gdn_conv_update", _I, [_P] * 8 + [_I] * 5 + [_L] + [_I] * 2 + [_P]),
    ("gdn_scan_carry_rows", _L, [_I] * 4),
    ("gdn_scan_workspace_bytes", _SZ, [_I] * 5),
    ("gdn_scan_fwd", _I, [_P] * 7 + [_I] * 4 + [_L] + [_I] * 3 + [_P, _SZ, _P]),
    ("gdn_scan_bwd", _I, [_P] * 9 + [_I] * 4 + [_L] + [_I] * 3 + [_P, _SZ, _P]),
    ("gdn_scan_update", _I, [_P] * 7 + [_I] * 4 + [_L] + [_I] * 3 + [_P]),
]

_lib = None


class GDNError(RuntimeError):
    """A call into libgdn.so returned a negative gdn_status."""


def lib():
    """Load libgdn.so (built in-tree by gated_delta_rule_42_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gated_delta_rule_42_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGNATURES:
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def gdn_version() -> int:
    return lib().gdn_version()


def gdn_status_string(status: int) -> str:
    return lib().gdn_status_string(status).decode()


def _check(status: int, what: str):
    if status != 0:
        raise GDNError(f"{what}: {gdn_status_string(status)} (status {status})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need_gpu(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("gdn: every tensor must be a contiguous tensor on a GPU")


def _expect(t, name, shape, dtypes):
    """Raise ValueError unless tensor t (if given) has this shape and one of these dtypes: the C
    ABI sees raw pointers only, so a wrong shape or dtype would otherwise be read or written out
    of bounds on the device."""
    if t is None:
        return
    if t.shape != tuple(shape):
        raise ValueError(f"gdn: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"gdn: {name} has dtype {str(t.dtype).replace('torch.', '')}, expected {names}")


_IN = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)


def _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, o=None, hT=None, g_channels=False):
    """Shapes and dtypes of the chunked forward (and backward) arguments; returns the sizes."""
    if q.dim() != 4:
        raise ValueError(f"gdn: q must be [B, T, H, d_k], got shape {tuple(q.shape)}")
    if q.dtype not in _IN:
        raise ValueError(f"gdn: q has dtype {q.dtype}, expected float32 or bfloat16")
    B, T, H, dk = q.shape
    if v.dim() != 4:
        raise ValueError(f"gdn: v must be [B, T, H, d_v], got shape {tuple(v.shape)}")
    dv = v.shape[-1]
    _expect(k, "k", q.shape, (q.dtype,))
    _expect(v, "v", (B, T, H, dv), (q.dtype,))
    _expect(g, "g", (B, T, H, dk) if g_channels else (B, T, H), _F32)
    _expect(beta, "beta", (B, T, H), _F32)
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.dtype != torch.int32:
            raise ValueError("gdn: cu_seqlens must be a 1-D int32 tensor of N + 1 >= 2 offsets")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _expect(h0, "h0", (N, H, dv, dk), _F32)
    _expect(hT, "hT", (N, H, dv, dk), _F32)
    _expect(o, "o", (B, T, H, dv), _IN)
    return B, T, H, dk, dv, N


def _check_decode_args(q, k, v, g, beta, state, o, g_channels=False):
    if q.dim() != 3 or q.dtype not in _IN:
        raise ValueError(f"gdn: q must be [N, H, d_k] float32 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    N, H, dk = q.shape
    if v.dim() != 3:
        raise ValueError(f"gdn: v must be [N, H, d_v], got shape {tuple(v.shape)}")
    dv = v.shape[-1]
    _expect(k, "k", q.shape, (q.dtype,))
    _expect(v, "v", (N, H, dv), (q.dtype,))
    _expect(g, "g", (N, H, dk) if g_channels else (N, H), _F32)
    _expect(beta, "beta", (N, H), _F32)
    _expect(state, "state", (N, H, dv, dk), _F32)
    _expect(o, "o", (N, H, dv), _IN)
    return N, H, dk, dv


def gdn_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, varlen, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return lib().gdn_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, int(bool(varlen)), chunk,
                                               _DTYPE[dtype])


def _workspace(B, T, H, dk, dv, N, cu_seqlens, dtype, device, workspace):
    need = gdn_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, cu_seqlens is not None, CHUNK, dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, need


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, chunk=CHUNK, *, o=None, hT=None,
                  o_dtype=None, output_final_state=True, workspace=None, stream=None):
    """Chunkwise forward pass. q, k [B,T,H,dk], v [B,T,H,dv] (fp32 or bf16); g, beta
    [B,T,H] fp32; h0 [N,H,dv,dk] fp32 or None; cu_seqlens int32 [N+1] or None.
    o is written in o_dtype (default: the dtype of q; fp32 is allowed for bf16 inputs).
    Returns (o [B,T,H,dv], hT [N,H,dv,dk] fp32 or None)."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, o, hT)
    _need_gpu(q, k, v, g, beta, h0, cu_seqlens, o, hT, workspace)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    workspace, need = _workspace(B, T, H, dk, dv, N, cu_seqlens, q.dtype, q.device, workspace)
    st = lib().gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                             _ptr(hT), _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N,
                             _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1), _ptr(workspace),
                             workspace.numel() if workspace is not None else 0,
                             _stream(q.device, stream))
    _check(st, "gdn_chunk_fwd")
    return o, hT


def gdn_chunk_fwd_noalloc(q, k, v, g, beta, h0=None, cu_seqlens=None, chunk=CHUNK, *, o=None, hT=None,
                          o_dtype=None, output_final_state=True, stream=None):
    """gdn_chunk_fwd on the library's own device scratch array (no workspace argument, no
    allocation inside the call; outputs are allocated here unless given)."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, o, hT)
    _need_gpu(q, k, v, g, beta, h0, cu_seqlens, o, hT)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    st = lib().gdn_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                     _ptr(hT), _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N,
                                     _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1),
                                     _stream(q.device, stream))
    _check(st, "gdn_chunk_fwd_noalloc")
    return o, hT


def gdn_chunk_prepare(q, k, g, beta, workspace, cu_seqlens=None, chunk=CHUNK, *, dv=None, stream=None):
    """Stage 1 (per-chunk gate scan, gated Gram, UT transform, chunk operators) into
    `workspace` (uint8 tensor of gdn_chunk_fwd_workspace_bytes bytes)."""
    if q.dim() != 4 or q.dtype not in _IN:
        raise ValueError(f"gdn: q must be [B, T, H, d_k] float32 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    B, T, H, dk = q.shape
    dv = dk if dv is None else dv
    _check_chunk_args(q, k, q.new_empty((B, T, H, dv), device="meta"), g, beta, None, cu_seqlens)
    _need_gpu(q, k, g, beta, cu_seqlens, workspace)
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    st = lib().gdn_chunk_prepare(_ptr(q), _ptr(k), _ptr(g), _ptr(beta), _ptr(cu_seqlens), chunk, B, T,
                                 H, dk, dv, N, _DTYPE.get(q.dtype, -1), _ptr(workspace),
                                 workspace.numel() if workspace is not None else 0,
                                 _stream(q.device, stream))
    _check(st, "gdn_chunk_prepare")


def gdn_chunk_propagate(q, k, v, workspace, h0=None, cu_seqlens=None, chunk=CHUNK, *, o=None,
                        hT=None, o_dtype=None, output_final_state=True, stream=None):
    """Stage 2 (state carried across chunks, chunk outputs) from a prepared workspace."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, None, None, h0, cu_seqlens, o, hT)
    _need_gpu(q, k, v, h0, cu_seqlens, o, hT, workspace)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    st = lib().gdn_chunk_propagate(_ptr(q), _ptr(k), _ptr(v), _ptr(h0), _ptr(o), _ptr(hT),
                                   _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N,
                                   _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1), _ptr(workspace),
                                   workspace.numel() if workspace is not None else 0,
                                   _stream(q.device, stream))
    _check(st, "gdn_chunk_propagate")
    return o, hT


def gdn_decode_step(q, k, v, g, beta, state, o=None, *, o_dtype=torch.float32, stream=None):
    """One decode step: q, k [N,H,dk], v [N,H,dv] (fp32 or bf16), g, beta [N,H] fp32,
    state [N,H,dv,dk] fp32 updated in place. Returns o [N,H,dv] in o_dtype (fp32 by
    default; bf16 gives the fp32 result rounded to nearest even)."""
    N, H, dk, dv = _check_decode_args(q, k, v, g, beta, state, o)
    _need_gpu(q, k, v, g, beta, state, o)
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype, device=q.device)
    st = lib().gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(o),
                               N, H, dk, dv, _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1),
                               _stream(q.device, stream))
    _check(st, "gdn_decode_step")
    return o


def gdn_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, varlen, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return lib().gdn_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, int(bool(varlen)), chunk,
                                               _DTYPE[dtype])


def gdn_chunk_bwd(q, k, v, g, beta, do, h0=None, dhT=None, cu_seqlens=None, chunk=CHUNK, *,
                  grad_dtype=None, need_dh0=True, workspace=None, stream=None):
    """Backward pass of gdn_chunk_fwd for output gradients do [B,T,H,dv] (dtype of q) and
    final-state gradients dhT [N,H,dv,dk] fp32 (or None). Returns dq, dk, dv (grad_dtype,
    default the dtype of q; fp32 is allowed for bf16 inputs), dg, dbeta [B,T,H] fp32 and
    dh0 [N,H,dv,dk] fp32 (None unless need_dh0)."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, hT=dhT)
    _expect(do, "do", (B, T, H, dv), (q.dtype,))
    _need_gpu(q, k, v, g, beta, do, h0, dhT, cu_seqlens, workspace)
    dev = q.device
    gd = grad_dtype or q.dtype
    dq = torch.empty(q.shape, dtype=gd, device=dev)
    dk_ = torch.empty(k.shape, dtype=gd, device=dev)
    dv_ = torch.empty(v.shape, dtype=gd, device=dev)
    dg = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    db = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    dh0 = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev) if need_dh0 else None
    need = gdn_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, cu_seqlens is not None, chunk, q.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib().gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(do), _ptr(dhT),
                             _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db), _ptr(dh0),
                             _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N, _DTYPE.get(q.dtype, -1),
                             _DTYPE.get(gd, -1), _ptr(workspace),
                             workspace.numel() if workspace is not None else 0,
                             _stream(dev, stream))
    _check(st, "gdn_chunk_bwd")
    return dq, dk_, dv_, dg, db, dh0


def gdn_kda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, varlen, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return lib().gdn_kda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, int(bool(varlen)), chunk,
                                                   _DTYPE[dtype])


def gdn_kda_chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, chunk=CHUNK, *, o=None, hT=None,
                      o_dtype=None, output_final_state=True, workspace=None, stream=None):
    """Chunkwise forward pass with a channel-wise decay: as gdn_chunk_fwd, with g
    [B,T,H,dk] fp32 (log of one decay per key channel)."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, o, hT, g_channels=True)
    _need_gpu(q, k, v, g, beta, h0, cu_seqlens, o, hT, workspace)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    need = gdn_kda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, cu_seqlens is not None, chunk, q.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = lib().gdn_kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                 _ptr(hT), _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N,
                                 _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1), _ptr(workspace),
                                 workspace.numel() if workspace is not None else 0,
                                 _stream(q.device, stream))
    _check(st, "gdn_kda_chunk_fwd")
    return o, hT


def gdn_kda_decode_step(q, k, v, g, beta, state, o=None, *, o_dtype=torch.float32, stream=None):
    """One decode step with a channel-wise decay: g [N,H,dk] fp32; otherwise as
    gdn_decode_step (state updated in place)."""
    N, H, dk, dv = _check_decode_args(q, k, v, g, beta, state, o, g_channels=True)
    _need_gpu(q, k, v, g, beta, state, o)
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype, device=q.device)
    st = lib().gdn_kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(o),
                                   N, H, dk, dv, _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1),
                                   _stream(q.device, stream))
    _check(st, "gdn_kda_decode_step")
    return o


def gdn_decoupled_chunk_fwd(q, k, v, g, erase, write, h0=None, cu_seqlens=None, chunk=CHUNK, *, o=None,
                            hT=None, o_dtype=None, output_final_state=True, workspace=None, stream=None):
    """Chunkwise forward pass with a channel-wise decay g [B,T,H,dk] and decoupled erase
    [B,T,H,dk] and write [B,T,H,dv] gates (fp32) in place of beta."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, None, h0, cu_seqlens, o, hT, g_channels=True)
    _expect(erase, "erase", (B, T, H, dk), _F32)
    _expect(write, "write", (B, T, H, dv), _F32)
    _need_gpu(q, k, v, g, erase, write, h0, cu_seqlens, o, hT, workspace)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    need = gdn_kda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, cu_seqlens is not None, chunk, q.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = lib().gdn_decoupled_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(erase), _ptr(write), _ptr(h0),
                                       _ptr(o), _ptr(hT), _ptr(cu_seqlens), chunk, B, T, H, dk, dv, N,
                                       _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1), _ptr(workspace),
                                       workspace.numel() if workspace is not None else 0,
                                       _stream(q.device, stream))
    _check(st, "gdn_decoupled_chunk_fwd")
    return o, hT


def gdn_decoupled_decode_step(q, k, v, g, erase, write, state, o=None, *, o_dtype=torch.float32, stream=None):
    """One decode step with a channel-wise decay g [N,H,dk] and decoupled erase [N,H,dk] and
    write [N,H,dv] gates; the state is updated in place."""
    N, H, dk, dv = _check_decode_args(q, k, v, g, None, state, o, g_channels=True)
    _expect(erase, "erase", (N, H, dk), _F32)
    _expect(write, "write", (N, H, dv), _F32)
    _need_gpu(q, k, v, g, erase, write, state, o)
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype, device=q.device)
    st = lib().gdn_decoupled_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(erase), _ptr(write),
                                         _ptr(state), _ptr(o), N, H, dk, dv, _DTYPE.get(q.dtype, -1),
                                         _DTYPE.get(o.dtype, -1), _stream(q.device, stream))
    _check(st, "gdn_decoupled_decode_step")
    return o


def _same_gpu(device, **ts):
    """Raise ValueError unless every given tensor is on this GPU (any strides)."""
    if device.type != "cuda":
        raise ValueError("gdn: every tensor must be on a GPU")
    index = device.index
    for name, t in ts.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"gdn: {name} is on {t.device}, expected {device}")


def _adr(t):
    return None if t is None else t.data_ptr()


def _dense_on(device, **ts):
    """_same_gpu, and every given tensor contiguous."""
    if device.type != "cuda":
        raise ValueError("gdn: every tensor must be on a GPU")
    index = device.index
    for name, t in ts.items():
        if t is not None:
            if t.get_device() != index:
                raise ValueError(f"gdn: {name} is on {t.device}, expected {device}")
            if not t.is_contiguous():
                raise ValueError(f"gdn: {name} must be contiguous")


# the current stream's handle without the Stream object around it, where this torch has it: a call's checks and marshalling
# are a third of a small call's time
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _new(shape, dtype, device, stream):
    """An output or workspace of a call on `stream`, from that stream's share of the allocator: memory that is still in
    use on another stream is never handed out for it."""
    if stream is None:   # the sizes one by one: 1.3 us where a shape object takes 2.1
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _call(name, device, stream, *args):
    """Run an entry point on `stream` (default: the current one of `device`) with `device` current."""
    fn = getattr(_lib or lib(), name)
    if stream is not None:
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != 0:
        _check(st, name)


def _token_stride(t, name, tail):
    """The stride between tokens of t [..., *tail dims]: its leading dimensions must collapse to one."""
    lead, strides = t.shape[:-tail], t.stride()[:-tail]
    stride = None
    for n, s in zip(reversed(lead), reversed(strides)):
        if n == 1:
            continue
        if stride is None:
            stride, span = s, s * n
        elif s != span:
            raise ValueError(f"gdn: the leading dimensions of {name} (shape {tuple(t.shape)}, strides {t.stride()}) "
                             "do not form one token dimension of a single stride")
        else:
            span = s * n
    return 0 if stride is None else stride


def _row_strides(t, name):
    """Token and head strides of t [..., heads, d] with contiguous channels."""
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"gdn: the last dimension of {name} must be contiguous")
    head = strides[-2] if shape[-2] > 1 else 0
    if len(shape) == 3:
        return (strides[0] if shape[0] > 1 else 0), head
    return (_token_stride(t, name, 2) if t.numel() else 0), head


def gdn_recurrent_fwd(q, k, v, g, beta, states, slots, cu_seqlens=None, out_slots=None, o=None, *,
                      o_dtype=torch.float32, stream=None):
    """Runs of tokens on a pool of states. q, k [T,H,dk], v [T,HV,dv] (fp32 or bf16; token strides are free, HV a
    multiple of H); g [T,HV] or, channel-wise, [T,HV,dk], beta [T,HV] fp32; states [n_slots,HV,dv,dk] fp32, updated
    in place; slots int32 [N], the slot of each sequence (outside the pool: a padded entry, o = 0); cu_seqlens
    int32 [N+1], or None: one token per sequence; out_slots int32 [T], or None: with it the state after token t goes
    to slot out_slots[t] (outside the pool: not kept) instead of the last one to the sequence's own slot.
    Slots written must be distinct. Returns o [T,HV,dv] in o_dtype; rows that no sequence covers are not written."""
    if q.dim() != 3 or q.dtype not in _IN:
        raise ValueError(f"gdn: q must be [T, H, d_k] float32 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    T, H, dk = q.shape
    if v.dim() != 3:
        raise ValueError(f"gdn: v must be [T, HV, d_v], got shape {tuple(v.shape)}")
    HV, dv = v.shape[1:]
    if H < 1 or HV < H or HV % H:
        raise ValueError(f"gdn: the {HV} value heads must be a multiple of the {H} query heads")
    _expect(k, "k", q.shape, (q.dtype,))
    _expect(v, "v", (T, HV, dv), (q.dtype,))
    channels = g.dim() == 3
    _expect(g, "g", (T, HV, dk) if channels else (T, HV), _F32)
    _expect(beta, "beta", (T, HV), _F32)
    if states.dim() != 4:
        raise ValueError(f"gdn: states must be [n_slots, HV, d_v, d_k], got shape {tuple(states.shape)}")
    _expect(states, "states", (states.shape[0], HV, dv, dk), _F32)
    if slots.dim() != 1 or slots.dtype != torch.int32:
        raise ValueError("gdn: slots must be a 1-D int32 tensor")
    N = slots.numel()
    if cu_seqlens is None and T != N:
        raise ValueError(f"gdn: {T} tokens for {N} sequences without cu_seqlens")
    _expect(cu_seqlens, "cu_seqlens", (N + 1,), (torch.int32,))
    _expect(out_slots, "out_slots", (T,), (torch.int32,))
    _expect(o, "o", (T, HV, dv), _IN)
    dev = q.device
    _same_gpu(dev, k=k, v=v)
    _dense_on(dev, g=g, beta=beta, states=states, slots=slots, cu_seqlens=cu_seqlens, out_slots=out_slots, o=o)
    strides = []
    for name, t, heads, d in (("q", q, H, dk), ("k", k, H, dk), ("v", v, HV, dv)):
        step = t.stride()
        if T and (step[2] != 1 or (heads > 1 and step[1] != d)):
            raise ValueError(f"gdn: the heads of {name} must follow each other densely within a token")
        strides.append(step[0] if T > 1 else 0)
    if o is None:
        o = _new((T, HV, dv), o_dtype, dev, stream)
    _call("gdn_recurrent_fwd", dev, stream, _adr(q), _adr(k), _adr(v), _adr(g), _adr(beta), _adr(states),
          _adr(slots), _adr(cu_seqlens), _adr(out_slots), _adr(o), T, N, H, HV, dk, dv, states.shape[0], *strides,
          int(channels), _DTYPE.get(q.dtype, -1), _DTYPE.get(o.dtype, -1))
    return o


_NORM = {"l2": 0, "rms": 1}
_ROPE = {"half": 0, "interleaved": 1}


def _check_norm_args(q, k, q_weight, k_weight, positions, inv_freq, norm, layout):
    qs, ks, dtype = q.shape, k.shape, q.dtype
    if len(qs) < 3 or dtype not in _IN:
        raise ValueError(f"gdn: q must be [..., heads, d] float32 or bfloat16, got {tuple(qs)} {dtype}")
    lead, hq, d = qs[:-2], qs[-2], qs[-1]
    if len(ks) != len(qs):
        raise ValueError(f"gdn: k has shape {tuple(ks)}, expected {tuple(lead)} + (heads, {d})")
    hk = ks[-2]
    _expect(k, "k", (*lead, hk, d), (dtype,))
    if norm not in _NORM:
        raise ValueError(f"gdn: norm must be one of {sorted(_NORM)}, got {norm!r}")
    if layout not in _ROPE:
        raise ValueError(f"gdn: layout must be one of {sorted(_ROPE)}, got {layout!r}")
    _expect(q_weight, "q_weight", (d,), _F32)
    _expect(k_weight, "k_weight", (d,), _F32)
    if (positions is None) != (inv_freq is None):
        raise ValueError("gdn: positions and inv_freq go together")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1 or inv_freq.dtype != torch.float32:
            raise ValueError("gdn: inv_freq must be a 1-D float32 tensor of rot / 2 frequencies")
        rot = 2 * inv_freq.numel()
        _expect(positions, "positions", lead, (torch.int32,))
    dev = q.device
    _same_gpu(dev, k=k)
    _dense_on(dev, q_weight=q_weight, k_weight=k_weight, positions=positions, inv_freq=inv_freq)
    tokens = 1
    for n in lead:
        tokens *= n
    return tokens, hq, hk, d, rot


def gdn_qk_norm_fwd(q, k, q_weight=None, k_weight=None, *, positions=None, inv_freq=None, norm="l2", eps=1e-6,
                    q_scale=1.0, layout="half", rope_scale=1.0, out_dtype=None, q_out=None, k_out=None, stream=None):
    """Norm of every head of q [..., Hq, d] and k [..., Hk, d] (fp32 or bf16, views of a fused projection allowed),
    with the rotary rotation in the same pass: norm "l2" (unit vectors) or "rms", times the weights [d] fp32 (None:
    ones), rotated over the first 2 * len(inv_freq) channels by positions [...] int32 times inv_freq, in
    layout "half" or "interleaved", those channels times rope_scale; q times q_scale. Returns q and k, dense, in out_dtype
    (default the dtype of q; fp32 is allowed for bf16 inputs)."""
    tokens, hq, hk, d, rot = _check_norm_args(q, k, q_weight, k_weight, positions, inv_freq, norm, layout)
    qs, ks = _row_strides(q, "q"), _row_strides(k, "k")
    dev, od = q.device, out_dtype or q.dtype
    if q_out is not None or k_out is not None:
        _expect(q_out, "q_out", q.shape, _IN)
        _expect(k_out, "k_out", k.shape, _IN)
        if q_out is not None and k_out is not None and q_out.dtype != k_out.dtype:
            raise ValueError("gdn: q_out and k_out must have one dtype")
        _dense_on(dev, q_out=q_out, k_out=k_out)
        od = (k_out if q_out is None else q_out).dtype
    if q_out is None:
        q_out = _new(q.shape, od, dev, stream)
    if k_out is None:
        k_out = _new(k.shape, od, dev, stream)
    _call("gdn_qk_norm_fwd", dev, stream, _adr(q), _adr(k), _adr(q_weight), _adr(k_weight), _adr(positions),
          _adr(inv_freq), _adr(q_out), _adr(k_out), tokens, hq, hk, d, *qs, *ks, _NORM[norm], eps, rot, _ROPE[layout],
          q_scale, rope_scale, _DTYPE.get(q.dtype, -1), _DTYPE.get(od, -1))
    return q_out, k_out


def gdn_qk_norm_bwd_workspace_bytes(tokens, hq, hk, d) -> int:
    return lib().gdn_qk_norm_bwd_workspace_bytes(tokens, hq, hk, d)


def gdn_qk_norm_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, *, positions=None, inv_freq=None, norm="l2",
                    eps=1e-6, q_scale=1.0, layout="half", rope_scale=1.0, dq=None, dk=None, need_dw=None,
                    workspace=None, stream=None):
    """Backward pass of gdn_qk_norm_fwd with the same arguments: from the gradients dq_out, dk_out of its outputs
    (dense, the dtype of q, or fp32) returns dq, dk (the dtype of q; given ones may be views with strides, as of a fused
    gradient) and dq_weight, dk_weight (fp32 [d], None unless need_dw; default: for the weights that are given)."""
    tokens, hq, hk, d, rot = _check_norm_args(q, k, q_weight, k_weight, positions, inv_freq, norm, layout)
    gt = (q.dtype, torch.float32)
    _expect(dq_out, "dq_out", q.shape, gt)
    _expect(dk_out, "dk_out", k.shape, (dq_out.dtype,))
    _expect(dq, "dq", q.shape, (q.dtype,))
    _expect(dk, "dk", k.shape, (q.dtype,))
    dev = q.device
    _same_gpu(dev, dq=dq, dk=dk)
    _dense_on(dev, dq_out=dq_out, dk_out=dk_out, workspace=workspace)
    if dq is None:
        dq = _new(q.shape, q.dtype, dev, stream)
    if dk is None:
        dk = _new(k.shape, q.dtype, dev, stream)
    dqw = dkw = None
    if need_dw or (need_dw is None and q_weight is not None):
        dqw = _new((d,), torch.float32, dev, stream)
    if need_dw or (need_dw is None and k_weight is not None):
        dkw = _new((d,), torch.float32, dev, stream)
    if dqw is not None or dkw is not None:
        need = gdn_qk_norm_bwd_workspace_bytes(tokens, hq, hk, d)
        if workspace is None and need:
            workspace = _new((need,), torch.uint8, dev, stream)
    strides = [s for t, name in ((q, "q"), (k, "k"), (dq, "dq"), (dk, "dk")) for s in _row_strides(t, name)]
    _call("gdn_qk_norm_bwd", dev, stream, _adr(q), _adr(k), _adr(dq_out), _adr(dk_out), _adr(q_weight),
          _adr(k_weight), _adr(positions), _adr(inv_freq), _adr(dq), _adr(dk), _adr(dqw), _adr(dkw), tokens, hq, hk, d,
          *strides, _NORM[norm], eps, rot, _ROPE[layout], q_scale, rope_scale, _DTYPE.get(q.dtype, -1),
          _DTYPE.get(dq_out.dtype, -1), _adr(workspace),
          workspace.numel() * workspace.element_size() if workspace is not None else 0)
    return dq, dk, dqw, dkw


def gdn_kda_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, varlen, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return lib().gdn_kda_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, int(bool(varlen)), chunk, _DTYPE[dtype])


def gdn_kda_chunk_bwd(q, k, v, g, beta, do, h0=None, dhT=None, cu_seqlens=None, chunk=CHUNK, *, grad_dtype=None,
                      need_dh0=True, workspace=None, stream=None):
    """Backward pass of gdn_kda_chunk_fwd: as gdn_chunk_bwd, with g [B,T,H,dk] fp32. Returns dq, dk, dv (grad_dtype,
    default the dtype of q; fp32 is allowed for bf16 inputs), dg [B,T,H,dk] and dbeta [B,T,H] fp32 and dh0 [N,H,dv,dk]
    fp32 (None unless need_dh0)."""
    B, T, H, dk, dv, N = _check_chunk_args(q, k, v, g, beta, h0, cu_seqlens, hT=dhT, g_channels=True)
    _expect(do, "do", (B, T, H, dv), (q.dtype,))
    dev = q.device
    _dense_on(dev, q=q, k=k, v=v, g=g, beta=beta, do=do, h0=h0, dhT=dhT, cu_seqlens=cu_seqlens, workspace=workspace)
    gd = grad_dtype or q.dtype
    dq = _new(q.shape, gd, dev, stream)
    dk_ = _new(k.shape, gd, dev, stream)
    dv_ = _new(v.shape, gd, dev, stream)
    dg = _new(g.shape, torch.float32, dev, stream)
    db = _new((B, T, H), torch.float32, dev, stream)
    dh0 = _new((N, H, dv, dk), torch.float32, dev, stream) if need_dh0 else None
    need = gdn_kda_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N, cu_seqlens is not None, chunk, q.dtype)
    if workspace is None and need:
        workspace = _new((need,), torch.uint8, dev, stream)
    _call("gdn_kda_chunk_bwd", dev, stream, _adr(q), _adr(k), _adr(v), _adr(g), _adr(beta), _adr(h0), _adr(do),
          _adr(dhT), _adr(dq), _adr(dk_), _adr(dv_), _adr(dg), _adr(db), _adr(dh0), _adr(cu_seqlens), chunk, B, T, H, dk,
          dv, N, _DTYPE.get(q.dtype, -1), _DTYPE.get(gd, -1), _adr(workspace),
          workspace.numel() * workspace.element_size() if workspace is not None else 0)
    return dq, dk_, dv_, dg, db, dh0


def _rows_of(t, name):
    """Stride between the rows of t [..., d] with contiguous channels."""
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"gdn: the last dimension of {name} must be contiguous")
    if len(shape) == 2:
        return strides[0] if shape[0] > 1 else 0
    return _token_stride(t, name, 1) if t.numel() else 0


def _check_sizes(*sizes):
    """Sizes reach the C ABI as 32-bit integers."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"gdn: a size of {sizes} exceeds 2^31 - 1")


def _bytes(workspace):
    return workspace.numel() * workspace.element_size() if workspace is not None else 0


def gdn_layer_norm_fwd(x, weight=None, bias=None, *, residual=None, eps=1e-5, out_dtype=None, y=None, sum_out=None, stream=None):
    """Layer norm of the rows of x [..., d] (fp32 or bf16; rows may be strided), after adding residual [...,d] (the dtype of x, or fp32)
    where given. weight, bias [d] fp32 or None (ones, zeros). Returns y (dense, out_dtype, default the dtype of x) and
    the sum as it was normalised (dense, the residual's dtype; None without a residual)."""
    shape, dtype = x.shape, x.dtype
    if len(shape) < 1 or dtype not in _IN:
        raise ValueError(f"gdn: x must be [..., d] float32 or bfloat16, got {tuple(shape)} {dtype}")
    d = shape[-1]
    rows = x.numel() // d if d else 0
    _check_sizes(rows, d)
    _expect(weight, "weight", (d,), _F32)
    _expect(bias, "bias", (d,), _F32)
    _expect(residual, "residual", shape, (dtype, torch.float32))
    _expect(y, "y", shape, _IN)
    if residual is None and sum_out is not None:
        raise ValueError("gdn: sum_out needs a residual")
    dev = x.device
    if residual is not None:
        _expect(sum_out, "sum_out", shape, (residual.dtype,))
        _same_gpu(dev, residual=residual)
    _dense_on(dev, weight=weight, bias=bias, y=y, sum_out=sum_out)
    xs = _rows_of(x, "x")
    rs = _rows_of(residual, "residual") if residual is not None else 0
    if y is None:
        y = _new(shape, out_dtype or dtype, dev, stream)
    if residual is not None and sum_out is None:
        sum_out = _new(shape, residual.dtype, dev, stream)
    _call("gdn_layer_norm_fwd", dev, stream, _adr(x), _adr(residual), _adr(weight), _adr(bias), _adr(y), _adr(sum_out), rows, d,
          xs, rs, eps, _DTYPE[dtype], -1 if residual is None else _DTYPE[residual.dtype], _DTYPE.get(y.dtype, -1))
    return y, sum_out


def gdn_layer_norm_bwd_workspace_bytes(rows, d) -> int:
    return lib().gdn_layer_norm_bwd_workspace_bytes(rows, d)


def gdn_layer_norm_bwd(s, dy, weight=None, *, ds=None, eps=1e-5, need_dw=None, dx=None, workspace=None, stream=None):
    """Backward pass of gdn_layer_norm_fwd: s [..., d] is what was normalised (its sum, or its x without a residual), dy the gradient of y
    (dense, fp32 or bf16), ds the gradient that reaches the sum elsewhere (dense, the dtype of s) or None. Returns dx (dense, the
    dtype of s), the gradient of x and residual alike, and the gradients of weight and bias (fp32 [d], None unless need_dw;
    default: where a weight is given)."""
    shape, dtype = s.shape, s.dtype
    if len(shape) < 1 or dtype not in _IN:
        raise ValueError(f"gdn: s must be [..., d] float32 or bfloat16, got {tuple(shape)} {dtype}")
    d = shape[-1]
    rows = s.numel() // d if d else 0
    _check_sizes(rows, d)
    _expect(dy, "dy", shape, _IN)
    _expect(weight, "weight", (d,), _F32)
    _expect(ds, "ds", shape, (dtype,))
    _expect(dx, "dx", shape, (dtype,))
    dev = s.device
    _dense_on(dev, dy=dy, weight=weight, ds=ds, dx=dx, workspace=workspace)
    xs = _rows_of(s, "s")
    if dx is None:
        dx = _new(shape, dtype, dev, stream)
    dw = db = None
    if need_dw or (need_dw is None and weight is not None):
        dw, db = _new((d,), torch.float32, dev, stream), _new((d,), torch.float32, dev, stream)
        need = gdn_layer_norm_bwd_workspace_bytes(rows, d)
        if workspace is None and need:
            workspace = _new((need,), torch.uint8, dev, stream)
    _call("gdn_layer_norm_bwd", dev, stream, _adr(s), _adr(dy), _adr(ds), _adr(weight), _adr(dx), _adr(dw), _adr(db), rows, d, xs, eps,
          _DTYPE[dtype], _DTYPE[dy.dtype], _adr(workspace), _bytes(workspace))
    return dx, dw, db


_ACT = {None: 0, "silu": 1}


def _check_sequences(x, cu_seqlens):
    """Sizes of x [B, T, D] and its sequences."""
    if x.dim() != 3 or x.dtype not in _IN:
        raise ValueError(f"gdn: x must be [B, T, D] float32 or bfloat16, got {tuple(x.shape)} {x.dtype}")
    B, T, D = x.shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _check_sizes(B, T, D, N)
    if cu_seqlens is None:
        return B, T, D, N
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.dtype != torch.int32:
        raise ValueError("gdn: cu_seqlens must be a 1-D int32 tensor of N + 1 >= 2 offsets")
    return B, T, D, N


def _check_conv(x, weight, bias, activation):
    if activation not in _ACT:
        raise ValueError(f"gdn: activation must be None or 'silu', got {activation!r}")
    if weight.dim() != 2:
        raise ValueError(f"gdn: weight must be [D, width], got shape {tuple(weight.shape)}")
    D, W = x.shape[-1], weight.shape[1]
    _expect(weight, "weight", (D, W), _F32)
    _expect(bias, "bias", (D,), _F32)
    return W


def gdn_conv_fwd(x, weight, bias=None, window0=None, cu_seqlens=None, *, activation=None, y=None, windowT=None,
                 output_final_window=True, stream=None):
    """Causal convolution per channel over x [B, T, D] (fp32 or bf16; tokens may be strided) with weight [D, W] fp32, W in 2 .. 4
    (weight[:, -1] meets the token itself), bias [D] fp32 or None, then activation None or "silu". window0 [N, W-1, D] (the dtype
    of x): the inputs before each sequence, or None (zeros). cu_seqlens int32 [N+1]: packed sequences (B = 1).
    Returns y [B, T, D] (dense; rows that no sequence covers are not written) and the windows behind the sequences [N, W-1, D] (None
    unless output_final_window)."""
    B, T, D, N = _check_sequences(x, cu_seqlens)
    W = _check_conv(x, weight, bias, activation)
    dtype, dev = x.dtype, x.device
    _expect(window0, "window0", (N, W - 1, D), (dtype,))
    _expect(y, "y", x.shape, (dtype,))
    _expect(windowT, "windowT", (N, W - 1, D), (dtype,))
    _dense_on(dev, weight=weight, bias=bias, window0=window0, cu_seqlens=cu_seqlens, y=y, windowT=windowT)
    xs = _rows_of(x, "x")
    if y is None:
        y = _new((B, T, D), dtype, dev, stream)
    if windowT is None and output_final_window:
        windowT = _new((N, W - 1, D), dtype, dev, stream)
    _call("gdn_conv_fwd", dev, stream, _adr(x), _adr(weight), _adr(bias), _adr(window0), _adr(cu_seqlens), _adr(y), _adr(windowT),
          B, T, N, D, W, xs, _ACT[activation], _DTYPE[dtype])
    return y, windowT


def gdn_conv_bwd_workspace_bytes(B, T, D, width) -> int:
    return lib().gdn_conv_bwd_workspace_bytes(B, T, D, width)


def gdn_conv_bwd(x, weight, dy, bias=None, window0=None, dwindowT=None, cu_seqlens=None, *, activation=None, need_dw=True,
                 need_dwindow0=True, dx=None, workspace=None, stream=None):
    """Backward pass of gdn_conv_fwd: from dy [B, T, D] (dense) and dwindowT [N, W-1, D] or None, both of the dtype of x, returns dx (that
    dtype; a given one may have strided tokens, as of a fused gradient), dweight [D, W] fp32 (None unless need_dw), dbias [D] fp32 (None
    without a bias too) and dwindow0 [N, W-1, D] (None unless need_dwindow0)."""
    B, T, D, N = _check_sequences(x, cu_seqlens)
    W = _check_conv(x, weight, bias, activation)
    dtype, dev = x.dtype, x.device
    _expect(dy, "dy", x.shape, (dtype,))
    _expect(window0, "window0", (N, W - 1, D), (dtype,))
    _expect(dwindowT, "dwindowT", (N, W - 1, D), (dtype,))
    _expect(dx, "dx", x.shape, (dtype,))
    _same_gpu(dev, dx=dx)
    _dense_on(dev, weight=weight, dy=dy, bias=bias, window0=window0, dwindowT=dwindowT, cu_seqlens=cu_seqlens, workspace=workspace)
    xs = _rows_of(x, "x")
    if dx is None:
        dx = _new((B, T, D), dtype, dev, stream)
    dxs = _rows_of(dx, "dx")
    dw = db = None
    if need_dw:
        dw = _new((D, W), torch.float32, dev, stream)
        if bias is not None:
            db = _new((D,), torch.float32, dev, stream)
        need = gdn_conv_bwd_workspace_bytes(B, T, D, W)
        if workspace is None and need:
            workspace = _new((need,), torch.uint8, dev, stream)
    dwin = _new((N, W - 1, D), dtype, dev, stream) if need_dwindow0 else None
    _call("gdn_conv_bwd", dev, stream, _adr(x), _adr(weight), _adr(bias), _adr(window0), _adr(dy), _adr(dwindowT), _adr(cu_seqlens),
          _adr(dx), _adr(dw), _adr(db), _adr(dwin), B, T, N, D, W, xs, dxs, _ACT[activation], _DTYPE[dtype], _adr(workspace),
          _bytes(workspace))
    return dx, dw, db, dwin


def _check_runs(x, slots, cu_seqlens, out_slots):
    if x.dim() != 2 or x.dtype not in _IN:
        raise ValueError(f"gdn: x must be [T, D] float32 or bfloat16, got {tuple(x.shape)} {x.dtype}")
    T, D = x.shape
    _check_sizes(T, D, slots.numel())
    if slots.dim() != 1 or slots.dtype != torch.int32:
        raise ValueError("gdn: slots must be a 1-D int32 tensor")
    N = slots.numel()
    if cu_seqlens is None and T != N:
        raise ValueError(f"gdn: {T} tokens for {N} sequences without cu_seqlens")
    _expect(cu_seqlens, "cu_seqlens", (N + 1,), (torch.int32,))
    _expect(out_slots, "out_slots", (T,), (torch.int32,))
    return T, D, N


def gdn_conv_update(x, weight, bias, windows, slots, cu_seqlens=None, out_slots=None, y=None, *, activation=None, stream=None):
    """gdn_conv_fwd for runs of tokens on a pool of windows: x [T, D] (tokens may be strided), windows [n_slots, W-1, D] of the dtype of x,
    updated in place; slots, cu_seqlens and out_slots as in gdn_recurrent_fwd. Returns y [T, D]; rows that no sequence covers
    are not written."""
    T, D, N = _check_runs(x, slots, cu_seqlens, out_slots)
    W = _check_conv(x, weight, bias, activation)
    dtype, dev = x.dtype, x.device
    if windows.dim() != 3:
        raise ValueError(f"gdn: windows must be [n_slots, width - 1, D], got shape {tuple(windows.shape)}")
    _check_sizes(windows.shape[0])
    _expect(windows, "windows", (windows.shape[0], W - 1, D), (dtype,))
    _expect(y, "y", (T, D), (dtype,))
    _dense_on(dev, weight=weight, bias=bias, windows=windows, slots=slots, cu_seqlens=cu_seqlens, out_slots=out_slots, y=y)
    xs = _rows_of(x, "x")
    if y is None:
        y = _new((T, D), dtype, dev, stream)
    _call("gdn_conv_update", dev, stream, _adr(x), _adr(weight), _adr(bias), _adr(windows), _adr(slots), _adr(cu_seqlens),
          _adr(out_slots), _adr(y), T, N, D, W, windows.shape[0], xs, _ACT[activation], _DTYPE[dtype])
    return y


def gdn_scan_workspace_bytes(B, T, N, D, varlen) -> int:
    return lib().gdn_scan_workspace_bytes(B, T, N, D, int(bool(varlen)))


def gdn_scan_carry_rows(B, T, N, varlen) -> int:
    return lib().gdn_scan_carry_rows(B, T, N, int(bool(varlen)))


def gdn_scan_fwd(x, g, h0=None, cu_seqlens=None, *, blend=False, h=None, hT=None, out_dtype=None, output_final_state=True,
                 keep_carries=False, workspace=None, stream=None):
    """Gated linear recurrence per channel over x [B, T, D] (fp32 or bf16; tokens may be strided): h_t = a_t h_{t-1} + x_t, or with blend
    a_t h_{t-1} + (1 - a_t) x_t, a = exp(g), g [B, T, D] fp32 <= 0. h0 [N, D] fp32 or None (zeros); cu_seqlens int32 [N+1]: packed
    sequences (B = 1). Returns h [B, T, D] (out_dtype, default the dtype of x; rows that no sequence covers are not written), the
    final states [N, D] fp32 (None unless output_final_state) and, with keep_carries, what gdn_scan_bwd takes of this
    pass (fp32, a row per tile of 256 tokens, or of 32 where the sequences, empty ones among them, are short on average), else None."""
    B, T, D, N = _check_sequences(x, cu_seqlens)
    dtype, dev = x.dtype, x.device
    _expect(g, "g", (B, T, D), _F32)
    _expect(h0, "h0", (N, D), _F32)
    _expect(h, "h", (B, T, D), _IN)
    _expect(hT, "hT", (N, D), _F32)
    _dense_on(dev, g=g, h0=h0, cu_seqlens=cu_seqlens, h=h, hT=hT, workspace=workspace)
    xs = _rows_of(x, "x")
    if h is None:
        h = _new((B, T, D), out_dtype or dtype, dev, stream)
    if hT is None and output_final_state:
        hT = _new((N, D), torch.float32, dev, stream)
    carries = None
    if keep_carries:
        carries = _new((gdn_scan_carry_rows(B, T, N, cu_seqlens is not None), D), torch.float32, dev, stream)
    if workspace is None:
        need = gdn_scan_workspace_bytes(B, T, N, D, cu_seqlens is not None)
        if need:
            workspace = _new((need,), torch.uint8, dev, stream)
    _call("gdn_scan_fwd", dev, stream, _adr(x), _adr(g), _adr(h0), _adr(cu_seqlens), _adr(h), _adr(hT), _adr(carries), B, T, N, D, xs,
          int(blend), _DTYPE[dtype], _DTYPE.get(h.dtype, -1), _adr(workspace), _bytes(workspace))
    return h, hT, carries


def gdn_scan_bwd(x, g, dh, carries, dhT=None, cu_seqlens=None, *, blend=False, need_dh0=True, workspace=None, stream=None):
    """Backward pass of gdn_scan_fwd on the same x, g and cu_seqlens and the carries that it returned: from dh [B, T, D] (dense, the dtype
    of h) and dhT [N, D] fp32 or None returns dx [B, T, D] (the dtype of x), dg [B, T, D] fp32 and dh0 [N, D] fp32 (None unless
    need_dh0)."""
    B, T, D, N = _check_sequences(x, cu_seqlens)
    dtype, dev = x.dtype, x.device
    _expect(g, "g", (B, T, D), _F32)
    _expect(dh, "dh", (B, T, D), (dtype, torch.float32))
    _expect(dhT, "dhT", (N, D), _F32)
    _expect(carries, "carries", (gdn_scan_carry_rows(B, T, N, cu_seqlens is not None), D), _F32)
    _dense_on(dev, g=g, dh=dh, carries=carries, dhT=dhT, cu_seqlens=cu_seqlens, workspace=workspace)
    xs = _rows_of(x, "x")
    dx = _new((B, T, D), dtype, dev, stream)
    dg = _new((B, T, D), torch.float32, dev, stream)
    dh0 = _new((N, D), torch.float32, dev, stream) if need_dh0 else None
    if workspace is None:
        need = gdn_scan_workspace_bytes(B, T, N, D, cu_seqlens is not None)
        if need:
            workspace = _new((need,), torch.uint8, dev, stream)
    _call("gdn_scan_bwd", dev, stream, _adr(x), _adr(g), _adr(carries), _adr(dh), _adr(dhT), _adr(cu_seqlens), _adr(dx), _adr(dg),
          _adr(dh0), B, T, N, D, xs, int(blend), _DTYPE[dtype], _DTYPE[dh.dtype], _adr(workspace), _bytes(workspace))
    return dx, dg, dh0


def gdn_scan_update(x, g, states, slots, cu_seqlens=None, out_slots=None, h=None, *, blend=False, out_dtype=None, stream=None):
    """gdn_scan_fwd for runs of tokens on a pool of states: x [T, D] (tokens may be strided), g [T, D] fp32, states [n_slots, D] fp32, updated
    in place; slots, cu_seqlens and out_slots as in gdn_recurrent_fwd. Returns h [T, D] (out_dtype, default the dtype of x); rows
    that no sequence covers are not written."""
    T, D, N = _check_runs(x, slots, cu_seqlens, out_slots)
    dtype, dev = x.dtype, x.device
    _expect(g, "g", (T, D), _F32)
    if states.dim() != 2:
        raise ValueError(f"gdn: states must be [n_slots, D], got shape {tuple(states.shape)}")
    _check_sizes(states.shape[0])
    _expect(states, "states", (states.shape[0], D), _F32)
    _expect(h, "h", (T, D), _IN)
    _dense_on(dev, g=g, states=states, slots=slots, cu_seqlens=cu_seqlens, out_slots=out_slots, h=h)
    xs = _rows_of(x, "x")
    if h is None:
        h = _new((T, D), out_dtype or dtype, dev, stream)
    _call("gdn_scan_update", dev, stream, _adr(x), _adr(g), _adr(states), _adr(slots), _adr(cu_seqlens), _adr(out_slots), _adr(h), T, N,
          D, states.shape[0], xs, int(blend), _DTYPE[dtype], _DTYPE.get(h.dtype, -1))
    return h
