"""Thin Python binding of libsdm.so (include/sdm.h), same names as the C ABI.

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity), outputs are allocated with torch on the tensors' device, and the
raw device pointers plus the current torch stream are handed to the C ABI.
Every step of the hot path runs in the library's HIP kernels; there is no
fallback. If the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsdm.so")

SDM_F32, SDM_BF16, SDM_E4M3 = 0, 1, 2
SDM_DELTA_EQ4, SDM_DELTA_FIG2 = 0, 1
FORMS = {"eq4": SDM_DELTA_EQ4, "fig2": SDM_DELTA_FIG2}

# int sdm_*(...) signatures, in the order of include/sdm.h
_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGS = {
    "sdm_abi_version": (_I, []),
    "sdm_status_string": (ctypes.c_char_p, [_I]),
    "sdm_last_error": (ctypes.c_char_p, []),
    "sdm_address": (_I, [_P, _P, _I, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                         _P, _P, _P, _P, _P, _P, _P]),
    "sdm_debug_half_scores": (_I, [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "sdm_address_idw": (_I, [_P, _P, _I, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                             _P, _P, _P, _P, _P, _P, _P]),
    "sdm_debug_half_scores_idw": (_I, [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "sdm_state_init": (_I, [_P, _P, _I, _I64, _I64, _I64, _I64, _P]),
    "sdm_scan_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "sdm_scan_forward": (_I, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I, _P, _I, _P,
                              _I64, _I64, _I64, _I64, _I64, _I, _P, _I64, _P]),
    "sdm_scan_gated_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "sdm_scan_forward_gated": (_I, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I, _P, _I, _P,
                                    _P, _P, _I, ctypes.c_float, _P,
                                    _I64, _I64, _I64, _I64, _I64, _I, _P, _I64, _P]),
    "sdm_scan_forward_noalloc": (_I, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I, _P, _I, _P,
                                      _I64, _I64, _I64, _I64, _I64, _I, _P]),
    "sdm_scan_snapshot_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64]),
    "sdm_scan_forward_save": (_I, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I, _P, _P, _P,
                                   _I64, _I64, _I64, _I64, _I64, _I, _P, _I64, _P]),
    "sdm_scan_backward_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "sdm_scan_backward": (_I, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I, _P, _P, _P, _P,
                               _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I, _P, _I64, _P]),
    "sdm_state_init_backward": (_I, [_P, _P, _I64, _I64, _I64, _I64, _P]),
    "sdm_gates": (_I, [_P, _I, _P, _P, _I, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P]),
    "sdm_output_gate": (_I, [_P, _P, _P, _I, ctypes.c_float, _I64, _I64, _I64, _I64, _P, _P]),
    "sdm_dense_scan_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64]),
    "sdm_dense_scan_forward": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                                    _P, _I64, _P]),
    "sdm_dense_scan_backward_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64]),
    "sdm_dense_scan_backward": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _I64, _I64, _I64, _I64, _I64, _P, _I64, _P]),
    "sdm_residual_norm": (_I, [_P, _I, _P, _P, _I, _P, ctypes.c_float, _I64, _I64, _P, _I, _P, _I64, _P]),
    "sdm_residual_norm_backward_workspace_bytes": (_I64, [_I64, _I64]),
    "sdm_residual_norm_backward": (_I, [_P, _P, _I, _P, _I, _P, ctypes.c_float, _I64, _I64, _P, _P,
                                        _P, _I64, _P]),
    "sdm_balance_workspace_bytes": (_I64, [_I64, _I64, _I64, _I64, _I64]),
    "sdm_balance_forward": (_I, [_P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P]),
    "sdm_balance_backward": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "sdm_causal_conv_forward": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P] + [_I64] * 5 + [_P]),
    "sdm_causal_conv_backward_workspace_bytes": (_I64, [_I64] * 5),
    "sdm_causal_conv_backward": (_I, [_P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P] + [_I64] * 5
                                 + [_P, _I64, _P]),
    "sdm_selective_scan_workspace_bytes": (_I64, [_I64] * 5),
    "sdm_selective_scan_forward": (_I, [_P] * 5 + [_I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P] + [_I64] * 5 + [_P, _I64, _P]),
    "sdm_selective_scan_backward_workspace_bytes": (_I64, [_I64] * 5),
    "sdm_selective_scan_backward": (_I, [_P] * 6 + [_I, _P, _P, _P, _P, _I] + [_P] * 13 + [_I64] * 5 + [_P, _I64, _P]),
    "sdm_residual_layer_norm": (_I, [_P, _I, _P, _P, _I, _P, _P, ctypes.c_float, _I64, _I64, _P, _I, _P, _I64, _P]),
    "sdm_residual_layer_norm_backward_workspace_bytes": (_I64, [_I64, _I64]),
    "sdm_residual_layer_norm_backward": (_I, [_P, _P, _I, _P, _I, _P, ctypes.c_float, _I64, _I64, _P, _P, _P,
                                              _P, _I64, _P]),
}

_lib = None


class SdmError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str):
        super().__init__(f"{fn} failed with status {code}: {detail}")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded libsdm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(fn: str, rc: int):
    if rc != 0:
        raise SdmError(fn, rc, lib().sdm_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dev(*ts: torch.Tensor) -> torch.device:
    d = ts[0].device
    for t in ts:
        if t.device.type != "cuda" or t.device != d:
            raise ValueError("all tensors must be on the same GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return d


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SDM_F32
    if t.dtype == torch.bfloat16:
        return SDM_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def sdm_abi_version() -> int:
    return lib().sdm_abi_version()


def sdm_status_string(code: int) -> str:
    return lib().sdm_status_string(code).decode()


def sdm_last_error() -> str:
    return lib().sdm_last_error().decode()


SCORINGS = ("dot", "idw")


def sdm_address(q_w: torch.Tensor, q_r: torch.Tensor, subkeys_w: torch.Tensor,
                subkeys_r: torch.Tensor, W: int, R: int, return_scores: bool = False,
                out: Optional[Tuple[torch.Tensor, ...]] = None, scoring: str = "dot"):
    """Product-key addressing of both branches.

    q_w, q_r [B,H,T,2,dh]; subkeys [H,2,n_sub,dh] (same dtype, fp32 or bf16).
    Returns (idx_w, wt_w, idx_r, wt_r) and, with return_scores, (score_w, score_r).
    ``out`` may pass preallocated (idx_w, wt_w, idx_r, wt_r) tensors. ``scoring``
    "dot" calls sdm_address, "idw" sdm_address_idw (inverse-distance half-scores).
    """
    if scoring not in SCORINGS:
        raise ValueError(f"unknown scoring {scoring!r}")
    fn = "sdm_address" if scoring == "dot" else "sdm_address_idw"
    d = _dev(q_w, q_r, subkeys_w, subkeys_r)
    B, H, T, two, dh = q_w.shape
    n = subkeys_w.shape[2]
    if two != 2 or q_r.shape != q_w.shape or subkeys_w.shape != (H, 2, n, dh) \
            or subkeys_r.shape != subkeys_w.shape:
        raise ValueError("shape mismatch in sdm_address")
    kw = dict(device=d)
    if out is not None:
        idx_w, wt_w, idx_r, wt_r = out
        for t, shp, dt in ((idx_w, (B, H, T, W), torch.int32), (wt_w, (B, H, T, W), torch.float32),
                           (idx_r, (B, H, T, R), torch.int32), (wt_r, (B, H, T, R), torch.float32)):
            if tuple(t.shape) != shp or t.dtype != dt:
                raise ValueError("preallocated address output has the wrong shape or dtype")
        _dev(q_w, idx_w, wt_w, idx_r, wt_r)
    else:
        idx_w = torch.empty((B, H, T, W), dtype=torch.int32, **kw)
        wt_w = torch.empty((B, H, T, W), dtype=torch.float32, **kw)
        idx_r = torch.empty((B, H, T, R), dtype=torch.int32, **kw)
        wt_r = torch.empty((B, H, T, R), dtype=torch.float32, **kw)
    sc_w = torch.empty((B, H, T, W), dtype=torch.float32, **kw) if return_scores else None
    sc_r = torch.empty((B, H, T, R), dtype=torch.float32, **kw) if return_scores else None
    _check(fn, getattr(lib(), fn)(
        _ptr(q_w), _ptr(q_r), _dtype_code(q_w), _ptr(subkeys_w), _ptr(subkeys_r),
        _dtype_code(subkeys_w), B, H, T, n, dh, W, R, _ptr(idx_w), _ptr(wt_w), _ptr(idx_r),
        _ptr(wt_r), _ptr(sc_w), _ptr(sc_r), _stream(d)))
    out = (idx_w, wt_w, idx_r, wt_r)
    return out + (sc_w, sc_r) if return_scores else out


def sdm_debug_half_scores(q: torch.Tensor, subkeys: torch.Tensor, scoring: str = "dot") -> torch.Tensor:
    """Half-scores [B,H,T,2,n_sub] fp32 of one branch (the contraction of sdm_address,
    or with scoring "idw" the inverse-distance scores of sdm_address_idw)."""
    if scoring not in SCORINGS:
        raise ValueError(f"unknown scoring {scoring!r}")
    fn = "sdm_debug_half_scores" if scoring == "dot" else "sdm_debug_half_scores_idw"
    d = _dev(q, subkeys)
    B, H, T, _, dh = q.shape
    n = subkeys.shape[2]
    half = torch.empty((B, H, T, 2, n), dtype=torch.float32, device=d)
    _check(fn, getattr(lib(), fn)(
        _ptr(q), _dtype_code(q), _ptr(subkeys), _dtype_code(subkeys), B, H, T, n, dh,
        _ptr(half), _stream(d)))
    return half


def sdm_state_init(M0: torch.Tensor, B: int, out: Optional[torch.Tensor] = None,
                   dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Per-sequence table [B,H,N,dv] initialised from M0 [H,N,dv] fp32, stored in
    ``dtype`` (float32, or bfloat16: rounded to nearest even)."""
    d = _dev(M0)
    H, N, dv = M0.shape
    if M0.dtype != torch.float32:
        raise ValueError("M0 must be fp32")
    M = out if out is not None else torch.empty((B, H, N, dv), dtype=dtype, device=d)
    if M.shape != (B, H, N, dv) or M.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("state tensor has the wrong shape or dtype")
    _dev(M0, M)
    _check("sdm_state_init", lib().sdm_state_init(_ptr(M0), _ptr(M), _dtype_code(M), B, H, N, dv,
                                                  _stream(d)))
    return M


def sdm_scan_workspace_bytes(B: int, H: int, T: int, W: int, R: int, dv: int) -> int:
    n = lib().sdm_scan_workspace_bytes(B, H, T, W, R, dv)
    if n < 0:
        raise ValueError("invalid sizes for the scan workspace")
    return n


def _scan_inputs(fn, idx_w, wt_w, idx_r, wt_r, alpha, beta, v, M, table_dtypes=(torch.float32,)):
    d = _dev(idx_w, wt_w, idx_r, wt_r, alpha, beta, v, M)
    B, H, T, W = idx_w.shape
    R = idx_r.shape[3]
    N, dv = M.shape[2], M.shape[3]
    shapes = {"wt_w": (wt_w, (B, H, T, W)), "idx_r": (idx_r, (B, H, T, R)),
              "wt_r": (wt_r, (B, H, T, R)), "alpha": (alpha, (B, H, T)),
              "beta": (beta, (B, H, T)), "v": (v, (B, H, T, dv)), "M": (M, (B, H, N, dv))}
    for name, (t, shp) in shapes.items():
        if tuple(t.shape) != shp:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shp}")
    if idx_w.dtype != torch.int32 or idx_r.dtype != torch.int32 or wt_w.dtype != torch.float32 \
            or wt_r.dtype != torch.float32 or alpha.dtype != torch.float32 \
            or beta.dtype != torch.float32 or M.dtype not in table_dtypes:
        raise ValueError(f"dtype mismatch in {fn}")
    return d, (B, H, T, W, R, N, dv)


def _f32_out(t: Optional[torch.Tensor], shape, d, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=d)
    if tuple(t.shape) != tuple(shape) or t.dtype != torch.float32:
        raise ValueError(f"{name} has the wrong shape or dtype")
    _dev(t)
    if t.device != d:
        raise ValueError("all tensors must be on the same GPU")
    return t


def _workspace(ws: Optional[torch.Tensor], nbytes: int, d) -> torch.Tensor:
    if ws is None:
        return torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=d)
    if ws.dtype != torch.uint8 or ws.dim() != 1:
        raise ValueError("workspace must be a 1-D uint8 tensor")
    _dev(ws)
    return ws


def sdm_scan_forward(idx_w: torch.Tensor, wt_w: torch.Tensor, idx_r: torch.Tensor,
                     wt_r: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                     v: torch.Tensor, M: torch.Tensor, form: str = "eq4",
                     y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sparse gated delta scan over all T tokens; M [B,H,N,dv] (float32 or
    bfloat16 storage) is updated in place.

    Returns y [B,H,T,dv] fp32.
    """
    d, (B, H, T, W, R, N, dv) = _scan_inputs("sdm_scan_forward", idx_w, wt_w, idx_r, wt_r,
                                             alpha, beta, v, M, (torch.float32, torch.bfloat16))
    y = _f32_out(y, (B, H, T, dv), d, "y")
    workspace = _workspace(workspace, sdm_scan_workspace_bytes(B, H, T, W, R, dv), d)
    _check("sdm_scan_forward", lib().sdm_scan_forward(
        _ptr(idx_w), _ptr(wt_w), W, _ptr(idx_r), _ptr(wt_r), R, _ptr(alpha), _ptr(beta),
        _ptr(v), _dtype_code(v), _ptr(M), _dtype_code(M), _ptr(y), B, H, T, N, dv, FORMS[form],
        _ptr(workspace), workspace.numel(), _stream(d)))
    return y


def sdm_scan_gated_workspace_bytes(B: int, H: int, T: int, W: int, R: int, dv: int) -> int:
    n = lib().sdm_scan_gated_workspace_bytes(B, H, T, W, R, dv)
    if n < 0:
        raise ValueError("invalid sizes for the gated scan workspace")
    return n


def sdm_scan_forward_gated(idx_w: torch.Tensor, wt_w: torch.Tensor, idx_r: torch.Tensor,
                           wt_r: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                           v: torch.Tensor, M: torch.Tensor, gamma: torch.Tensor, g: torch.Tensor,
                           eps: float = 1e-6, form: str = "eq4", y: Optional[torch.Tensor] = None,
                           keep_y: bool = False, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """The scan followed by the output step (RMS-Norm, gamma, sigmoid gate).
    M is updated in place. Returns o [B,H,T,dv] fp32, or (o, y) when y is given
    or keep_y is set (otherwise y is not stored where the scan need not)."""
    d, (B, H, T, W, R, N, dv) = _scan_inputs("sdm_scan_forward_gated", idx_w, wt_w, idx_r, wt_r,
                                             alpha, beta, v, M, (torch.float32, torch.bfloat16))
    if gamma.shape != (H, dv) or gamma.dtype != torch.float32 or g.shape != (B, H, T, dv):
        raise ValueError("shape or dtype mismatch of gamma or g in sdm_scan_forward_gated")
    _dev(idx_w, gamma, g)
    if y is not None or keep_y:
        y = _f32_out(y, (B, H, T, dv), d, "y")
    o = _f32_out(out, (B, H, T, dv), d, "o")
    workspace = _workspace(workspace, sdm_scan_gated_workspace_bytes(B, H, T, W, R, dv), d)
    _check("sdm_scan_forward_gated", lib().sdm_scan_forward_gated(
        _ptr(idx_w), _ptr(wt_w), W, _ptr(idx_r), _ptr(wt_r), R, _ptr(alpha), _ptr(beta),
        _ptr(v), _dtype_code(v), _ptr(M), _dtype_code(M), _ptr(y),
        _ptr(gamma), _ptr(g), _dtype_code(g), float(eps), _ptr(o), B, H, T, N, dv, FORMS[form],
        _ptr(workspace), workspace.numel(), _stream(d)))
    return (o, y) if y is not None else o


def sdm_scan_forward_noalloc(idx_w: torch.Tensor, wt_w: torch.Tensor, idx_r: torch.Tensor,
                             wt_r: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                             v: torch.Tensor, M: torch.Tensor, form: str = "eq4",
                             y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sdm_scan_forward with the library's own per-GPU scratch instead of a
    workspace (the C call allocates nothing; pass y to keep this binding from
    allocating it). M is updated in place. Returns y [B,H,T,dv] fp32."""
    d, (B, H, T, W, R, N, dv) = _scan_inputs("sdm_scan_forward_noalloc", idx_w, wt_w, idx_r, wt_r,
                                             alpha, beta, v, M, (torch.float32, torch.bfloat16))
    y = _f32_out(y, (B, H, T, dv), d, "y")
    _check("sdm_scan_forward_noalloc", lib().sdm_scan_forward_noalloc(
        _ptr(idx_w), _ptr(wt_w), W, _ptr(idx_r), _ptr(wt_r), R, _ptr(alpha), _ptr(beta),
        _ptr(v), _dtype_code(v), _ptr(M), _dtype_code(M), _ptr(y), B, H, T, N, dv, FORMS[form],
        _stream(d)))
    return y


def sdm_scan_snapshot_bytes(B: int, H: int, T: int, W: int, dv: int) -> int:
    n = lib().sdm_scan_snapshot_bytes(B, H, T, W, dv)
    if n < 0:
        raise ValueError("invalid sizes for the pre-image buffer")
    return n


def sdm_scan_forward_save(idx_w: torch.Tensor, wt_w: torch.Tensor, idx_r: torch.Tensor,
                          wt_r: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                          v: torch.Tensor, M: torch.Tensor, form: str = "eq4",
                          y: Optional[torch.Tensor] = None, snap: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The training forward: sdm_scan_forward that also stores the pre-image of
    every write. M is updated in place. Returns (y [B,H,T,dv], snap [B,H,T,W,dv])."""
    d, (B, H, T, W, R, N, dv) = _scan_inputs("sdm_scan_forward_save", idx_w, wt_w, idx_r, wt_r,
                                             alpha, beta, v, M)
    y = _f32_out(y, (B, H, T, dv), d, "y")
    snap = _f32_out(snap, (B, H, T, W, dv), d, "snap")
    workspace = _workspace(workspace, sdm_scan_workspace_bytes(B, H, T, W, R, dv), d)
    _check("sdm_scan_forward_save", lib().sdm_scan_forward_save(
        _ptr(idx_w), _ptr(wt_w), W, _ptr(idx_r), _ptr(wt_r), R, _ptr(alpha), _ptr(beta),
        _ptr(v), _dtype_code(v), _ptr(M), _ptr(y), _ptr(snap), B, H, T, N, dv, FORMS[form],
        _ptr(workspace), workspace.numel(), _stream(d)))
    return y, snap


def sdm_scan_backward_workspace_bytes(B: int, H: int, T: int, W: int, R: int, dv: int) -> int:
    n = lib().sdm_scan_backward_workspace_bytes(B, H, T, W, R, dv)
    if n < 0:
        raise ValueError("invalid sizes for the backward workspace")
    return n


def sdm_scan_backward(idx_w: torch.Tensor, wt_w: torch.Tensor, idx_r: torch.Tensor,
                      wt_r: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                      v: torch.Tensor, snap: torch.Tensor, dy: torch.Tensor, M: torch.Tensor,
                      dM: torch.Tensor, form: str = "eq4", out: Optional[dict] = None,
                      workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward of one sdm_scan_forward_save call, undoing its writes in place.

    M [B,H,N,dv] (in: after the forward call, out: before it) and dM (in: dL/dM
    after the call, out: before it) are updated in place. Returns a dict with dv
    [B,H,T,dv], dalpha, dbeta [B,H,T], dwt_w [B,H,T,W], dwt_r [B,H,T,R]; ``out``
    may pass those tensors preallocated.
    """
    d, (B, H, T, W, R, N, dv) = _scan_inputs("sdm_scan_backward", idx_w, wt_w, idx_r, wt_r,
                                             alpha, beta, v, M)
    for name, t, shp in (("snap", snap, (B, H, T, W, dv)), ("dy", dy, (B, H, T, dv)),
                         ("dM", dM, (B, H, N, dv))):
        if tuple(t.shape) != shp or t.dtype != torch.float32:
            raise ValueError(f"{name} has the wrong shape or dtype")
        _dev(M, t)
    out = dict(out or {})
    shapes = {"dv": (B, H, T, dv), "dalpha": (B, H, T), "dbeta": (B, H, T),
              "dwt_w": (B, H, T, W), "dwt_r": (B, H, T, R)}
    for k, shp in shapes.items():
        out[k] = _f32_out(out.get(k), shp, d, k)
    workspace = _workspace(workspace, sdm_scan_backward_workspace_bytes(B, H, T, W, R, dv), d)
    _check("sdm_scan_backward", lib().sdm_scan_backward(
        _ptr(idx_w), _ptr(wt_w), W, _ptr(idx_r), _ptr(wt_r), R, _ptr(alpha), _ptr(beta),
        _ptr(v), _dtype_code(v), _ptr(snap), _ptr(dy), _ptr(M), _ptr(dM), _ptr(out["dv"]),
        _ptr(out["dalpha"]), _ptr(out["dbeta"]), _ptr(out["dwt_w"]), _ptr(out["dwt_r"]),
        B, H, T, N, dv, FORMS[form], _ptr(workspace), workspace.numel(), _stream(d)))
    return out


def sdm_gates(x: torch.Tensor, W_a: torch.Tensor, W_b: torch.Tensor, b_dt: torch.Tensor,
              A: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Scan gates from the layer input: alpha = exp(-A softplus(W_a x + b_dt)),
    beta = sigmoid(W_b x). x [B,T,d], W_a/W_b [H,d] (same dtype, fp32 or bf16),
    b_dt/A [H] fp32. Returns (alpha, beta) [B,H,T] fp32."""
    d_ = _dev(x, W_a, W_b, b_dt, A)
    B, T, d = x.shape
    H = W_a.shape[0]
    if W_a.shape != (H, d) or W_b.shape != (H, d) or b_dt.shape != (H,) or A.shape != (H,):
        raise ValueError("shape mismatch in sdm_gates")
    if b_dt.dtype != torch.float32 or A.dtype != torch.float32:
        raise ValueError("b_dt and A must be fp32")
    al, be = out if out is not None else (None, None)
    al = _f32_out(al, (B, H, T), d_, "alpha")
    be = _f32_out(be, (B, H, T), d_, "beta")
    _check("sdm_gates", lib().sdm_gates(
        _ptr(x), _dtype_code(x), _ptr(W_a), _ptr(W_b), _dtype_code(W_a), _ptr(b_dt), _ptr(A),
        B, T, d, H, _ptr(al), _ptr(be), _stream(d_)))
    return al, be


def sdm_output_gate(y: torch.Tensor, gamma: torch.Tensor, g: torch.Tensor, eps: float = 1e-6,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-head RMS-Norm of y [B,H,T,dv] times gamma [H,dv] and sigmoid(g) (g
    [B,H,T,dv], fp32 or bf16). Returns o [B,H,T,dv] fp32."""
    d_ = _dev(y, gamma, g)
    B, H, T, dv = y.shape
    if gamma.shape != (H, dv) or g.shape != y.shape or y.dtype != torch.float32 \
            or gamma.dtype != torch.float32:
        raise ValueError("shape or dtype mismatch in sdm_output_gate")
    o = _f32_out(out, (B, H, T, dv), d_, "o")
    if o.data_ptr() == y.data_ptr() and o.numel() > 0:
        raise ValueError("o may not alias y")
    _check("sdm_output_gate", lib().sdm_output_gate(
        _ptr(y), _ptr(gamma), _ptr(g), _dtype_code(g), float(eps), B, H, T, dv, _ptr(o), _stream(d_)))
    return o


def sdm_state_init_backward(dM: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the shared initial state: dM0 [H,N,dv] = sum over b of dM [B,H,N,dv]."""
    d = _dev(dM)
    B, H, N, dv = dM.shape
    if dM.dtype != torch.float32:
        raise ValueError("dM must be fp32")
    dM0 = _f32_out(out, (H, N, dv), d, "dM0")
    _check("sdm_state_init_backward", lib().sdm_state_init_backward(
        _ptr(dM), _ptr(dM0), B, H, N, dv, _stream(d)))
    return dM0


# The calls below are short enough to be bound by their host side: addresses are
# passed as plain integers, devices compared by index.

def _gpu(t0: torch.Tensor, *ts: Optional[torch.Tensor]) -> torch.device:
    """The tensors' device: all contiguous, on one GPU (None: not given)."""
    i = t0.get_device()
    if i < 0 or not t0.is_contiguous():
        raise ValueError("tensors must be contiguous and on a GPU")
    for t in ts:
        if t is not None and (t.get_device() != i or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous and on the same GPU")
    return t0.device


def _call(fn: str, d: torch.device, *args):
    """Library call ``fn`` on the device's current stream, whatever device is current."""
    i = d.index
    if torch.cuda.current_device() != i:
        with torch.cuda.device(i):
            return _call(fn, d, *args)
    rc = getattr(_lib or lib(), fn)(*args, _stream_of(i))
    if rc:
        _check(fn, rc)


def _stream_of(i: int) -> int:
    return torch.cuda.current_stream(i).cuda_stream


# the handle itself, without a Stream object around it (2 of 11 us of a short call)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _out(t: Optional[torch.Tensor], like: torch.Tensor, shape, dtype: torch.dtype, name: str) -> torch.Tensor:
    """A new tensor on ``like``'s device, or the given one after its checks."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} has the wrong shape or dtype")
    _gpu(like, t)
    return t


def _known(out: dict, names):
    """Refuses preallocated tensors under names that the call does not write."""
    if not out.keys() <= set(names):
        raise ValueError(f"no such output: {sorted(out.keys() - set(names))}")


def sdm_dense_scan_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int) -> int:
    n = lib().sdm_dense_scan_workspace_bytes(B, H, T, dk, dv)
    if n < 0:
        raise ValueError("invalid sizes for the dense scan workspace")
    return n


def _dense_inputs(fn, q, k, v, alpha, beta, states):
    d = _gpu(q, k, v, alpha, beta)
    B, H, T, dk = q.shape
    dv = v.shape[-1] if v.dim() else 0
    for name, t, shp in (("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)), ("alpha", alpha, (B, H, T)),
                         ("beta", beta, (B, H, T))):
        if tuple(t.shape) != shp:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shp}")
    if k.dtype != q.dtype or v.dtype != q.dtype or alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError(f"dtype mismatch in {fn}")
    for name, t in states:
        if t is not None:
            _out(t, q, (B, H, dk, dv), torch.float32, name)
    return d, (B, H, T, dk, dv)


def sdm_dense_scan_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                           beta: torch.Tensor, S0: Optional[torch.Tensor] = None,
                           S: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense gated recurrence S_t = alpha_t S_{t-1} + beta_t k_t (x) v_t, y_t = q_t S_t (no delta rule).

    q, k [B,H,T,dk], v [B,H,T,dv] (one dtype, fp32 or bf16), alpha, beta [B,H,T] fp32,
    S0 [B,H,dk,dv] fp32 or None (zeros). Returns (y [B,H,T,dv] fp32, S the last state);
    ``S`` and ``y`` may pass them preallocated, and S may be S0 (updated in place).
    """
    d, (B, H, T, dk, dv) = _dense_inputs("sdm_dense_scan_forward", q, k, v, alpha, beta, (("S0", S0), ("S", S)))
    S = _out(S, q, (B, H, dk, dv), torch.float32, "S")
    y = _out(y, q, (B, H, T, dv), torch.float32, "y")
    n = sdm_dense_scan_workspace_bytes(B, H, T, dk, dv)
    ws = _workspace(workspace, n, d) if n or workspace is not None else None
    _call("sdm_dense_scan_forward", d,
        _at(q), _at(k), _at(v), _dtype_code(q), _at(alpha), _at(beta), _at(S0), _at(S), _at(y),
        B, H, T, dk, dv, _at(ws), ws.numel() if ws is not None else 0)
    return y, S


def sdm_dense_scan_backward_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int) -> int:
    n = lib().sdm_dense_scan_backward_workspace_bytes(B, H, T, dk, dv)
    if n < 0:
        raise ValueError("invalid sizes for the dense backward workspace")
    return n


def sdm_dense_scan_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                            beta: torch.Tensor, dy: torch.Tensor, S0: Optional[torch.Tensor] = None,
                            dS: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                            workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of one sdm_dense_scan_forward call (nothing is kept from it).

    dy [B,H,T,dv] fp32; dS [B,H,dk,dv] fp32 or None: the gradient of the last state. Returns
    a dict with dq, dk [B,H,T,dk], dv [B,H,T,dv], dlog_alpha (to ln alpha), dbeta [B,H,T] and
    dS0 [B,H,dk,dv], all fp32; ``out`` may pass those tensors preallocated.
    """
    d, (B, H, T, dk, dv) = _dense_inputs("sdm_dense_scan_backward", q, k, v, alpha, beta, (("S0", S0), ("dS", dS)))
    _out(dy, q, (B, H, T, dv), torch.float32, "dy")
    out = dict(out or {})
    shapes = {"dq": (B, H, T, dk), "dk": (B, H, T, dk), "dv": (B, H, T, dv), "dlog_alpha": (B, H, T),
              "dbeta": (B, H, T), "dS0": (B, H, dk, dv)}
    _known(out, shapes)
    for name, shp in shapes.items():
        out[name] = _out(out.get(name), q, shp, torch.float32, name)
    workspace = _workspace(workspace, sdm_dense_scan_backward_workspace_bytes(B, H, T, dk, dv), d)
    _call("sdm_dense_scan_backward", d,
        _at(q), _at(k), _at(v), _dtype_code(q), _at(alpha), _at(beta), _at(dy), _at(S0), _at(dS),
        _at(out["dq"]), _at(out["dk"]), _at(out["dv"]), _at(out["dlog_alpha"]), _at(out["dbeta"]),
        _at(out["dS0"]), B, H, T, dk, dv, _at(workspace), workspace.numel())
    return out


NORM_OUT = {"f32": (SDM_F32, torch.float32), "bf16": (SDM_BF16, torch.bfloat16),
            "e4m3": (SDM_E4M3, torch.float8_e4m3fn)}


def sdm_residual_norm(x: torch.Tensor, gamma: torch.Tensor, res: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, dtype: str = "bf16", group: int = 0,
                      out: Optional[dict] = None) -> dict:
    """h = x + res and its RMS-Norm y = h / sqrt(mean h^2 + eps) * gamma, per row.

    x [..., d], res the same shape or None, gamma [d] fp32. ``dtype`` is y's: "f32",
    "bf16" or "e4m3", the last with fp32 scales per row (group 0: [..., 1]) or per ``group``
    columns ([..., d / group]); a row or group with a NaN or infinity has such a scale. Returns
    a dict with y, h (with res; in res's dtype) and scale (for e4m3); ``out`` may pass those
    tensors preallocated, h may be res or x.
    """
    return _norm("sdm_residual_norm", x, gamma, (), res, eps, dtype, group, out)


def _norm(fn, x, gamma, more, res, eps, dtype, group, out):
    """``more``: the parameters that the call takes behind gamma, [d] fp32 or None."""
    d_ = _gpu(x, gamma, res, *more)
    if dtype not in NORM_OUT:
        raise ValueError(f"unknown output dtype {dtype!r}")
    if x.dim() < 1 or gamma.shape != x.shape[-1:] or gamma.dtype != torch.float32 \
            or (res is not None and res.shape != x.shape) \
            or any(p is not None and (p.shape != gamma.shape or p.dtype != torch.float32) for p in more):
        raise ValueError(f"shape or dtype mismatch in {fn}")
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    code, yt = NORM_OUT[dtype]
    out = dict(out) if out else {}
    shape = x.shape
    want = {"y": (shape, yt)}
    if res is not None:
        want["h"] = (shape, res.dtype)
    if dtype == "e4m3":
        if group < 0 or (group and d % group):
            raise ValueError("group must be 0 or divide d")
        want["scale"] = ((*shape[:-1], d // group if group else 1), torch.float32)
    _known(out, want)
    for name, (shp, dt) in want.items():
        out[name] = _out(out.get(name), x, shp, dt, name)
    h, scale = out.get("h"), out.get("scale")
    _call(fn, d_,
        _at(x), _dtype_code(x), _at(res), _at(h), _dtype_code(x if res is None else res), _at(gamma),
        *map(_at, more), float(eps), rows, d, _at(out["y"]), code, _at(scale), group)
    return out


def sdm_residual_norm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor,
                               dh: Optional[torch.Tensor] = None, eps: float = 1e-6,
                               out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of sdm_residual_norm from the stored h (x where there was no residual).

    dy, dh [..., d] of one dtype (dh: what arrives at h from behind, or None), h [..., d],
    gamma [d] fp32. Returns a dict with dx (the gradient of x and of res, in dy's dtype) and
    dgamma [d] fp32; ``out`` may pass them preallocated, dx may be dy, dh or h.
    """
    return _norm_backward("sdm_residual_norm_backward", ("dgamma",), dy, h, gamma, dh, eps, out, workspace)


def _norm_backward(fn, sums, dy, h, gamma, dh, eps, out, workspace):
    d_ = _gpu(dy, h, gamma, dh)
    if dy.dim() < 1 or gamma.shape != dy.shape[-1:] or gamma.dtype != torch.float32 or h.shape != dy.shape \
            or (dh is not None and (dh.shape != dy.shape or dh.dtype != dy.dtype)):
        raise ValueError(f"shape or dtype mismatch in {fn}")
    d = dy.shape[-1]
    rows = dy.numel() // d if d else 0
    out = dict(out or {})
    _known(out, ("dx", *sums))
    got = {"dx": _out(out.get("dx"), dy, dy.shape, dy.dtype, "dx")}
    for name in sums:
        got[name] = _out(out.get(name), dy, (d,), torch.float32, name)
        if rows == 0:
            got[name].zero_()
    n = getattr(lib(), fn + "_workspace_bytes")(rows, d)
    ws = _workspace(workspace, max(n, 0), d_)
    _call(fn, d_,
        _at(dy), _at(dh), _dtype_code(dy), _at(h), _dtype_code(h), _at(gamma), float(eps), rows, d,
        *map(_at, got.values()), _at(ws), ws.numel())
    return got


def sdm_residual_layer_norm(x: torch.Tensor, gamma: torch.Tensor, bias: Optional[torch.Tensor] = None,
                            res: Optional[torch.Tensor] = None, eps: float = 1e-5, dtype: str = "bf16", group: int = 0,
                            out: Optional[dict] = None) -> dict:
    """h = x + res and its layer norm y = (h - mean h) / sqrt(var h + eps) * gamma + bias, per row.

    bias [d] fp32 or None; everything else, outputs among it, as in sdm_residual_norm.
    """
    return _norm("sdm_residual_layer_norm", x, gamma, (bias,), res, eps, dtype, group, out)


def sdm_residual_layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor,
                                     dh: Optional[torch.Tensor] = None, eps: float = 1e-5,
                                     out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of sdm_residual_layer_norm from the stored h: dx, dgamma and dbias [d] fp32 (as
    sdm_residual_norm_backward)."""
    return _norm_backward("sdm_residual_layer_norm_backward", ("dgamma", "dbias"), dy, h, gamma, dh, eps, out, workspace)


def sdm_balance_workspace_bytes(B: int, H: int, T: int, K: int, N: int) -> int:
    n = lib().sdm_balance_workspace_bytes(B, H, T, K, N)
    if n < 0:
        raise ValueError("invalid sizes for the balance workspace")
    return n


def _mask(mask, B, T, idx):
    if mask is None:
        return
    if tuple(mask.shape) != (B, T) or mask.dtype not in (torch.uint8, torch.bool):
        raise ValueError("mask must be [B, T], uint8 or bool")
    _gpu(idx, mask)


def sdm_balance_forward(idx: torch.Tensor, wt: torch.Tensor, N: int, mask: Optional[torch.Tensor] = None,
                        out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Slot counts and balance loss of an addressing result, per head over the kept tokens.

    idx [B,H,T,K] int32, wt [B,H,T,K] fp32 (as sdm_address gives them), mask [B,T] uint8 or
    bool (non-zero: kept) or None. Returns a dict with counts [H,N] int32, mass [H,N] fp32,
    tokens [1] int32 and loss [H] fp32 (1 when even); ``out`` may pass them preallocated.
    """
    d = _gpu(idx, wt)
    B, H, T, K = idx.shape
    if wt.shape != idx.shape or idx.dtype != torch.int32 or wt.dtype != torch.float32:
        raise ValueError("shape or dtype mismatch in sdm_balance_forward")
    _mask(mask, B, T, idx)
    out = dict(out or {})
    want = {"counts": ((H, N), torch.int32), "mass": ((H, N), torch.float32),
            "tokens": ((1,), torch.int32), "loss": ((H,), torch.float32)}
    _known(out, want)
    for name, (shp, dt) in want.items():
        out[name] = _out(out.get(name), idx, shp, dt, name)
    if H == 0:
        out["tokens"].zero_()
    workspace = _workspace(workspace, sdm_balance_workspace_bytes(B, H, T, K, N), d)
    _call("sdm_balance_forward", d,
        _at(idx), _at(wt), _at(mask), B, H, T, K, N, _at(out["counts"]), _at(out["mass"]),
        _at(out["tokens"]), _at(out["loss"]), _at(workspace), workspace.numel())
    return out


def sdm_balance_backward(idx: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor, dloss: torch.Tensor,
                         mask: Optional[torch.Tensor] = None, dwt: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The balance loss's gradient to the weights: dwt [B,H,T,K] fp32 from dloss [H] fp32 and the
    counts [H,N] and tokens [1] of sdm_balance_forward on the same idx and mask."""
    d = _gpu(idx, counts, tokens, dloss)
    B, H, T, K = idx.shape
    if idx.dtype != torch.int32 or counts.dtype != torch.int32 or tokens.dtype != torch.int32 \
            or dloss.dtype != torch.float32 or counts.dim() != 2 or counts.shape[0] != H \
            or tuple(tokens.shape) != (1,) or tuple(dloss.shape) != (H,):
        raise ValueError("shape or dtype mismatch in sdm_balance_backward")
    _mask(mask, B, T, idx)
    dwt = _out(dwt, idx, (B, H, T, K), torch.float32, "dwt")
    _call("sdm_balance_backward", d,
        _at(idx), _at(mask), _at(counts), _at(tokens), _at(dloss), B, H, T, K, counts.shape[1],
        _at(dwt))
    return dwt


# Rows by strides: consecutive channels, the other dimensions at any stride.

ACTS = {None: 0, "silu": 1}
_I3, _I12, _I14 = (ctypes.c_int64 * n for n in (3, 12, 14))


def _rows(name: str, t: torch.Tensor, like: torch.Tensor, shape):
    """Checks a tensor by strides (batch, head or token, token or group first, channels last)."""
    if t.get_device() != like.get_device() or t.get_device() < 0:
        raise ValueError("all tensors must be on the same GPU")
    if t.shape != shape or t.dtype != like.dtype:
        raise ValueError(f"{name} has the wrong shape or dtype")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the channels of {name} must be consecutive")


def _sequences(start, lengths, B, T, like):
    if start is not None:
        if start.shape != (B, T) or start.dtype not in (torch.uint8, torch.bool):
            raise ValueError("start must be [B, T], uint8 or bool")
        _gpu(like, start)
    if lengths is not None:
        if lengths.shape != (B,) or lengths.dtype != torch.int32:
            raise ValueError("lengths must be [B], int32")
        _gpu(like, lengths)


def _conv_inputs(fn, x, w, bias, act, S0, S, start, lengths):
    shape, st = x.shape, x.stride()
    if len(shape) == 3:
        (B, T, d), H, s = shape, 1, _I3(st[0], 0, st[1])
        per = (d,)
    elif len(shape) == 4:
        (B, H, T, d), s = shape, _I3(st[0], st[1], st[2])
        per = (H, d)
    else:
        raise ValueError("x must be [B, T, d] or [B, H, T, d]")
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    if st[-1] != 1 and d > 1:
        raise ValueError("the channels of x must be consecutive")
    if w.dim() != len(shape) - 1 or w.shape[:-1] != per or w.dtype != torch.float32 \
            or (bias is not None and (bias.shape != per or bias.dtype != torch.float32)):
        raise ValueError(f"shape or dtype mismatch in {fn}")
    K = w.shape[-1]
    if K < 2:
        raise ValueError("w must hold at least 2 taps")
    dev = _gpu(w, bias, S0, S)
    if x.get_device() != dev.index:
        raise ValueError("all tensors must be on the same GPU")
    state = (*shape[:-2], K - 1, d)
    for name, t in (("S0", S0), ("S", S)):
        if t is not None and (t.shape != state or t.dtype != x.dtype):
            raise ValueError(f"{name} has the wrong shape or dtype")
    if start is not None or lengths is not None:
        _sequences(start, lengths, B, T, w)
    return dev, (B, H, T, d, K), state, s


def sdm_causal_conv_forward(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                            act: Optional[str] = "silu", S0: Optional[torch.Tensor] = None,
                            S: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                            lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Short causal convolution y_t = act(bias + sum_j w_j x_{t-K+1+j}) over time of every channel.

    x [B,T,d] or [B,H,T,d] (fp32 or bf16; channels consecutive, the rest at any stride: a part of a
    projection or its heads transposed need no copy), w [d,K] or [H,d,K] and bias [d] or [H,d] fp32,
    act "silu" or None. S0: the K-1 inputs in front, [B,K-1,d] or [B,H,K-1,d] in x's dtype, or None
    (zeros). start [B,T] uint8 or bool: tokens that begin a sequence; lengths [B] int32: the tokens that
    are there (y is 0 behind them). Returns (y, S): y contiguous in x's shape and dtype, S the last K-1
    inputs; both may be passed preallocated, and S may be S0 (updated in place).
    """
    d_, sizes, state, xs = _conv_inputs("sdm_causal_conv_forward", x, w, bias, act, S0, S, start, lengths)
    if S is None:
        S = x.new_empty(state)
    y = _out(y, w, x.shape, x.dtype, "y")
    _call("sdm_causal_conv_forward", d_,
        _at(x), _dtype_code(x), xs, _at(w), _at(bias), ACTS[act], _at(S0), _at(S), _at(start), _at(lengths), _at(y), *sizes)
    return y, S


def sdm_causal_conv_backward_workspace_bytes(B: int, H: int, T: int, d: int, K: int) -> int:
    n = lib().sdm_causal_conv_backward_workspace_bytes(B, H, T, d, K)
    if n < 0:
        raise ValueError("invalid sizes for the convolution's backward workspace")
    return n


def sdm_causal_conv_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                             act: Optional[str] = "silu", S0: Optional[torch.Tensor] = None,
                             dS: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                             lengths: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                             workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of one sdm_causal_conv_forward call (nothing is kept from it).

    dy contiguous in x's shape and dtype; dS, the gradient of the last state, or None. Returns a dict with
    dx (x's dtype, in x's order of dimensions), dw, dbias (fp32) and dS0 (x's dtype); ``out`` may pass those
    preallocated, dx at any strides with consecutive channels (a part of a projection's gradient).
    """
    d_, sizes, state, xs = _conv_inputs("sdm_causal_conv_backward", x, w, bias, act, S0, dS, start, lengths)
    B, H, T, d, K = sizes
    _out(dy, w, x.shape, x.dtype, "dy")
    out = dict(out or {})
    _known(out, ("dx", "dw", "dbias", "dS0"))
    dx = out.get("dx")
    if dx is None:
        dx = torch.empty_like(x)
    _rows("dx", dx, x, x.shape)
    gs = (dx.stride(0), dx.stride(1) if x.dim() == 4 else 0, dx.stride(-2))
    dw = _out(out.get("dw"), w, w.shape, torch.float32, "dw")
    dbias = _out(out.get("dbias"), w, w.shape[:-1], torch.float32, "dbias")
    dS0 = _out(out.get("dS0"), w, state, x.dtype, "dS0")
    if B == 0:
        dw.zero_()
        dbias.zero_()
    ws = _workspace(workspace, sdm_causal_conv_backward_workspace_bytes(*sizes), d_)
    _call("sdm_causal_conv_backward", d_,
        _at(dy), _at(x), _dtype_code(x), xs, _at(w), _at(bias), ACTS[act], _at(S0), _at(dS), _at(start), _at(lengths),
        _at(dx), _I3(*gs), _at(dw), _at(dbias), _at(dS0), *sizes, _at(ws), ws.numel())
    return {"dx": dx, "dw": dw, "dbias": dbias, "dS0": dS0}


def sdm_selective_scan_workspace_bytes(B: int, T: int, D: int, G: int, N: int) -> int:
    """Workspace of one forward call; fewer sequences or tokens can need more than many, so one workspace for calls of
    several sizes takes the largest of their answers."""
    n = lib().sdm_selective_scan_workspace_bytes(B, T, D, G, N)
    if n < 0:
        raise ValueError("invalid sizes for the selective scan workspace")
    return n


def _selective_inputs(fn, x, dt, A, Bm, Cm, D, z, dt_bias, states, start, lengths, dy=None):
    if x.dim() != 3 or Bm.dim() not in (3, 4) or A.dim() != 2:
        raise ValueError("x must be [B, T, D], A [D, N], Bm and Cm [B, T, N] or [B, T, G, N]")
    shape, dtype = x.shape, x.dtype
    B, T, n = shape
    N, four = A.shape[1], Bm.dim() == 4
    G = Bm.shape[2] if four else 1
    groups = (B, T, G, N) if four else (B, T, N)
    dev = _gpu(A, D, dt_bias, *(t for _, t in states))
    s = []
    for name, t, shp in (("x", x, shape), ("dt", dt, shape), ("z", z, shape), ("Bm", Bm, groups), ("Cm", Cm, groups), ("dy", dy, shape)):
        if t is None:
            if name == "z":
                s += (0, 0)
            continue
        st = t.stride()
        if t.shape != shp or t.dtype != dtype:
            raise ValueError(f"{name} has the wrong shape or dtype")
        if st[-1] != 1 and shp[-1] > 1:
            raise ValueError(f"the channels of {name} must be consecutive")
        if t.get_device() != dev.index:
            raise ValueError("all tensors must be on the same GPU")
        s += st[:-1]
        if shp is groups and not four:
            s.append(0)
    if G < 1 or n % G or A.shape[0] != n or A.dtype != torch.float32 \
            or any(p is not None and (p.shape != (n,) or p.dtype != torch.float32) for p in (D, dt_bias)):
        raise ValueError(f"shape or dtype mismatch in {fn}")
    for name, t in states:
        if t is not None and (t.shape != (B, n, N) or t.dtype != torch.float32):
            raise ValueError(f"{name} has the wrong shape or dtype")
    if start is not None or lengths is not None:
        _sequences(start, lengths, B, T, A)
    return dev, (B, T, n, G, N), (_I12 if dy is None else _I14)(*s)


def sdm_selective_scan_forward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                               D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                               dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                               S0: Optional[torch.Tensor] = None, S: Optional[torch.Tensor] = None,
                               start: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                               y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Selective state-space scan: delta = softplus(dt + dt_bias) (or dt + dt_bias), h_t = exp(delta_t A) h_{t-1} +
    delta_t x_t B_t, y_t = (C_t h_t + D x_t) silu(z_t).

    x, dt, z [B,T,D] and Bm, Cm [B,T,N] or [B,T,G,N] (channels in G groups), one dtype (fp32 or bf16; last
    dimension consecutive, the rest at any stride), A [D,N], D and dt_bias [D] fp32, S0 [B,D,N] fp32 or None
    (zeros). start and lengths as in sdm_causal_conv_forward. Returns (y [B,T,D] in x's dtype, S the last
    state); both may be passed preallocated, and S may be S0 (updated in place).
    """
    d_, sizes, s = _selective_inputs("sdm_selective_scan_forward", x, dt, A, Bm, Cm, D, z, dt_bias,
                                     (("S0", S0), ("S", S)), start, lengths)
    B, T, n, G, N = sizes
    if S is None:
        S = A.new_empty((B, n, N))
    y = _out(y, A, x.shape, x.dtype, "y")
    need = sdm_selective_scan_workspace_bytes(*sizes)
    ws = _workspace(workspace, need, d_) if need or workspace is not None else None
    _call("sdm_selective_scan_forward", d_,
        _at(x), _at(dt), _at(z), _at(Bm), _at(Cm), _dtype_code(x), s, _at(A), _at(D), _at(dt_bias), int(softplus),
        _at(S0), _at(S), _at(start), _at(lengths), _at(y), *sizes, _at(ws), ws.numel() if ws is not None else 0)
    return y, S


def sdm_selective_scan_backward_workspace_bytes(B: int, T: int, D: int, G: int, N: int) -> int:
    n = lib().sdm_selective_scan_backward_workspace_bytes(B, T, D, G, N)
    if n < 0:
        raise ValueError("invalid sizes for the selective scan's backward workspace")
    return n


def sdm_selective_scan_backward(dy: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                                Cm: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                                dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                                S0: Optional[torch.Tensor] = None, dS: Optional[torch.Tensor] = None,
                                start: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                                out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of one sdm_selective_scan_forward call (nothing is kept from it).

    dy [B,T,D] in x's dtype, at any stride; dS [B,D,N] fp32, the gradient of the last state, or None. Returns
    a dict with dx, ddt, dz (with z) in x's dtype, dA, dB, dC, dD, ddt_bias and dS0 in fp32, named after the
    formula's letters and shaped as the inputs; ``out`` may pass those tensors preallocated.
    """
    d_, sizes, s = _selective_inputs("sdm_selective_scan_backward", x, dt, A, Bm, Cm, D, z, dt_bias,
                                     (("S0", S0), ("dS", dS)), start, lengths, dy)
    B, T, n, G, N = sizes
    out = dict(out or {})
    want = {"dx": (x.shape, x.dtype), "ddt": (x.shape, x.dtype), "dz": (x.shape, x.dtype), "dA": (A.shape, torch.float32),
            "dB": (Bm.shape, torch.float32), "dC": (Bm.shape, torch.float32), "dD": ((n,), torch.float32),
            "ddt_bias": ((n,), torch.float32), "dS0": ((B, n, N), torch.float32)}
    if z is None:
        del want["dz"]
    _known(out, want)
    for name, (shp, dtype) in want.items():
        out[name] = _out(out.get(name), A, shp, dtype, name)
        if B == 0:
            out[name].zero_()
    ws = _workspace(workspace, sdm_selective_scan_backward_workspace_bytes(*sizes), d_)
    _call("sdm_selective_scan_backward", d_,
        _at(dy), _at(x), _at(dt), _at(z), _at(Bm), _at(Cm), _dtype_code(x), s, _at(A), _at(D), _at(dt_bias), int(softplus),
        _at(S0), _at(dS), _at(start), _at(lengths), *(_at(out.get(k)) for k in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dS0")),
        *sizes, _at(ws), ws.numel())
    return out
