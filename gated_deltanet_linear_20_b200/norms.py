"""Norms around a layer: binding of the gdn_gated_norm and gdn_residual_norm calls.

Argument marshalling only, as in ``gdn.py``.  ``gated_norm`` is the RMS norm of
each row times a gate (o of a prefill or decode per head, or a plain norm
without a gate); ``residual_norm`` is the step between two blocks.  Tensors may
have any leading dimensions; the last one is normalised.  Calls run on the
current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .gdn import _lib
from .recurrence import _F32, _begin, _call, _code, _expect, _fits, _optional, _out

_vp, _ci, _cz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
for _name, _args in (
        ("gdn_gated_norm", [_vp, _ci] + [_vp] * 3 + [_ci] * 3 + [_vp] * 2),
        ("gdn_gated_norm_backward", [_vp, _vp, _ci] + [_vp] * 5 + [_ci] * 3 + [_vp, _cz, _vp, _vp]),
        ("gdn_residual_norm", [_vp] * 8 + [_ci] * 4 + [_vp] * 2),
        ("gdn_residual_norm_backward", [_vp] * 14 + [_ci] * 4 + [_vp, _cz, _vp, _vp])):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci
_lib.gdn_norm_workspace_bytes.argtypes = [_ci] * 3
_lib.gdn_norm_workspace_bytes.restype = _cz

GATES = {"silu": 0, "sigmoid": 1}  # gdn_gate


class NormOptions(ctypes.Structure):
    """gdn_norm_options (include/gdn.h)."""
    _fields_ = [("size", ctypes.c_int), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("gate", ctypes.c_int)]


def _options(eps: float, weight_offset: float, gate: str):
    code = GATES.get(gate)
    if code is None:
        raise ValueError(f"gate must be one of {sorted(GATES)}, got {gate!r}")
    if code == 0 and eps == 1e-6 and weight_offset == 0.0:
        return None  # the library's defaults
    return ctypes.byref(NormOptions(ctypes.sizeof(NormOptions), eps, weight_offset, code))


def _rows(x: torch.Tensor, shape):
    if len(shape) < 1:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    return (x.numel() // D if D else 0), D


def workspace_bytes(rows: int, D: int, weights: int = 1) -> int:
    """Bytes of workspace of a backward call with that many weight arrays."""
    _fits("workspace_bytes", rows, D)
    return int(_lib.gdn_norm_workspace_bytes(rows, D, weights))


def _workspace(workspace, rows, D, weights, dev):
    if workspace is None:
        need = workspace_bytes(rows, D, weights)
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace, workspace.numel()


def gated_norm(x: torch.Tensor, w: torch.Tensor, z: Optional[torch.Tensor] = None, *,
               gate: str = "silu", eps: float = 1e-6, weight_offset: float = 0.0,
               out_dtype: Optional[torch.dtype] = None,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = a(z) (w + weight_offset) x / sqrt(mean(x^2) + eps) over the last dimension.

    x [..., D] fp32 or bf16; w [D] fp32; z like x in shape, fp32 or bf16, or None
    (no gate); a is ``gate``: "silu" or "sigmoid".  y has z's type, or without z
    ``out_dtype`` (x's by default)."""
    shape, xd, xt, dev = _begin(x, "gated_norm", "")
    rows, D = _rows(x, shape)
    if out_dtype is None:
        out_dtype = xd if z is None else z.dtype
    px = _expect(x, "x", xd, shape, dev)
    pw = _expect(w, "w", _F32, (D,), dev)
    pz = _optional(z, "z", out_dtype, shape, dev)
    y = _out(y, "y", out_dtype, shape, dev, x)
    _call(_lib.gdn_gated_norm, dev, px, xt, pw, pz, y.data_ptr(), rows, D, _code(out_dtype, "y"),
          _options(eps, weight_offset, gate))
    return y


def gated_norm_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                        z: Optional[torch.Tensor] = None, *, gate: str = "silu",
                        eps: float = 1e-6, weight_offset: float = 0.0,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients of ``gated_norm``: returns (dx, dz, dw), dz None without z.  dx has
    x's type, dz dy's (which is z's), dw [D] is fp32, summed over the rows."""
    shape, xd, xt, dev = _begin(x, "gated_norm_backward", "")
    rows, D = _rows(x, shape)
    px = _expect(x, "x", xd, shape, dev)
    dt = _code(dy.dtype, "dy")
    pdy = _expect(dy, "dy", dy.dtype, shape, dev)
    pw = _expect(w, "w", _F32, (D,), dev)
    pz = _optional(z, "z", dy.dtype, shape, dev)
    dx = torch.empty_like(x)
    dz = torch.empty_like(z) if z is not None else None
    dw = torch.empty_like(w)
    ws, have = _workspace(workspace, rows, D, 1, dev)
    _call(_lib.gdn_gated_norm_backward, dev, pdy, px, xt, pw, pz, dx.data_ptr(),
          None if dz is None else dz.data_ptr(), dw.data_ptr(), rows, D, dt, ws.data_ptr(), have,
          _options(eps, weight_offset, gate))
    return dx, dz, dw


def residual_norm(x: torch.Tensor, r: torch.Tensor, w: torch.Tensor, *,
                  z: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, gate: str = "silu", eps: float = 1e-6,
                  weight_offset: float = 0.0, y: Optional[torch.Tensor] = None,
                  r_out: Optional[torch.Tensor] = None):
    """The step between two blocks: returns (y, r_out) with

        u = (w_post + weight_offset) x / rms(x)   (x itself without w_post)
        r_out = r + scale a(z) u                  y = (w + weight_offset) r_out / rms(r_out)

    x (the block's output), z [..., D] fp32 or bf16; r [..., D] of that type or
    fp32; w, w_post, scale [D] fp32; z, w_post, scale may be None (no gate, no
    norm behind the block, 1).  ``r_out`` may be ``r``."""
    shape, xd, dt, dev = _begin(x, "residual_norm", "")
    rows, D = _rows(x, shape)
    px = _expect(x, "x", xd, shape, dev)
    rt = _code(r.dtype, "r")
    pr = _expect(r, "r", r.dtype, shape, dev)
    pw = _expect(w, "w", _F32, (D,), dev)
    pz = _optional(z, "z", xd, shape, dev)
    pp = _optional(w_post, "w_post", _F32, (D,), dev)
    ps = _optional(scale, "scale", _F32, (D,), dev)
    y = _out(y, "y", xd, shape, dev, x)
    r_out = _out(r_out, "r_out", r.dtype, shape, dev, r)
    _call(_lib.gdn_residual_norm, dev, px, pr, pw, pz, pp, ps, y.data_ptr(), r_out.data_ptr(), rows,
          D, dt, rt, _options(eps, weight_offset, gate))
    return y, r_out


def residual_norm_backward(dy: torch.Tensor, dr_out: Optional[torch.Tensor], x: torch.Tensor,
                           r_out: torch.Tensor, w: torch.Tensor, *,
                           z: Optional[torch.Tensor] = None,
                           w_post: Optional[torch.Tensor] = None,
                           scale: Optional[torch.Tensor] = None, gate: str = "silu",
                           eps: float = 1e-6, weight_offset: float = 0.0,
                           workspace: Optional[torch.Tensor] = None):
    """Gradients of ``residual_norm`` at the kept sum ``r_out``: returns (dx, dr, dz,
    dw, dw_post, dscale), each None where its input is.  dr_out (of r_out's type,
    None: zeros) is the gradient that reaches r_out from what follows besides y."""
    shape, xd, dt, dev = _begin(x, "residual_norm_backward", "")
    rows, D = _rows(x, shape)
    px = _expect(x, "x", xd, shape, dev)
    rt = _code(r_out.dtype, "r_out")
    pr = _expect(r_out, "r_out", r_out.dtype, shape, dev)
    pdy = _expect(dy, "dy", xd, shape, dev)
    pdr = _optional(dr_out, "dr_out", r_out.dtype, shape, dev)
    pw = _expect(w, "w", _F32, (D,), dev)
    pz = _optional(z, "z", xd, shape, dev)
    pp = _optional(w_post, "w_post", _F32, (D,), dev)
    ps = _optional(scale, "scale", _F32, (D,), dev)
    dx, dr, dw = torch.empty_like(x), torch.empty_like(r_out), torch.empty_like(w)
    dz = torch.empty_like(z) if z is not None else None
    dwp = torch.empty_like(w_post) if w_post is not None else None
    dsc = torch.empty_like(scale) if scale is not None else None
    ws, have = _workspace(workspace, rows, D, 1 + (dwp is not None) + (dsc is not None), dev)
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(_lib.gdn_residual_norm_backward, dev, pdy, pdr, px, pr, pw, pz, pp, ps, dx.data_ptr(),
          dr.data_ptr(), at(dz), dw.data_ptr(), at(dwp), at(dsc), rows, D, dt, rt, ws.data_ptr(),
          have, _options(eps, weight_offset, gate))
    return dx, dr, dz, dw, dwp, dsc
