"""Channel recurrence (gated linear recurrence): binding of the gdn_scan calls.

    h_t = exp(g_t) h_{t-1} + beta_t x_t        per sequence and channel

Argument marshalling only, as in ``gdn.py``: the arithmetic is in the library's
CUDA kernels.  ``scan`` / ``scan_varlen`` run whole sequences, ``scan_step`` one
token with the state in place, and the ``*_backward`` calls return gradients.
Calls run on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .gdn import GDN_OK, GDNError, _check, _lib

_vp, _ci = ctypes.c_void_p, ctypes.c_int
for _name, _args in (("gdn_scan", [_vp] * 7 + [_ci] * 4 + [_vp, _vp]),
                     ("gdn_scan_varlen", [_vp] * 8 + [_ci] * 4 + [_vp, _vp]),
                     ("gdn_scan_step", [_vp] * 5 + [_ci] * 3 + [_vp]),
                     ("gdn_scan_backward", [_vp] * 11 + [_ci] * 5 + [_vp, _vp]),
                     ("gdn_scan_varlen_backward", [_vp] * 11 + [_ci, _vp] + [_ci] * 4 + [_vp, _vp])):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci
_lib.gdn_scan_carry_bytes.argtypes = [_ci] * 4
_lib.gdn_scan_carry_bytes.restype = ctypes.c_size_t

CARRY_TOKENS = 16  # GDN_SCAN_CARRY_TOKENS
DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # gdn_dtype
_F32, _I32 = torch.float32, torch.int32


def _expect(t, name, dtype, shape, device):
    """_check with its common answer first (the calls of one token are short), and
    the tensor's address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, dtype, shape, device)
    return t.data_ptr()


def _optional(t, name, dtype, shape, device):
    return None if t is None else _expect(t, name, dtype, shape, device)


def _code(dtype: torch.dtype, name: str) -> int:
    code = DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")
    return code


_MOST = 2 ** 31 - 1  # of a size: the library's are C ints, and ctypes keeps their low bits


def _fits(what: str, *sizes: int) -> None:
    if max(sizes, default=0) > _MOST:
        raise ValueError(f"{what}: sizes must be below 2^31, got {max(sizes)}")


def _begin(x: torch.Tensor, what: str, layout: str):
    """x's shape, type, type code and device; ``layout``: its dimensions, e.g. "[B,C]"
    ("": rows of its last dimension)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    shape, dtype, device = x.shape, x.dtype, x.device
    count = x.numel()
    if count > _MOST or count == 0:
        _fits(what, *(shape if layout else (*shape[-1:], count // max(1, shape[-1]) if shape else 0)))
    if device.type != "cuda":
        raise ValueError(f"{what} runs on CUDA tensors only (no CPU path)")
    if layout and len(shape) != layout.count(",") + 1:
        raise ValueError(f"x must be {layout}")
    return shape, dtype, _code(dtype, "x"), device


def _call(fn, device: torch.device, *args):
    """Calls the library on the tensors' device and that device's current stream.
    (The stream's handle is asked for directly: torch.cuda.current_stream builds
    an object first, 2.2 us against 0.1 of a call that takes 8 in all.)"""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != GDN_OK:
        raise GDNError(rc, fn.__name__)


def _out(t, name, dtype, shape, device, like=None):
    """A given output, checked, or a new one (``like``: a tensor of its shape, which
    is quicker to copy the shape from)."""
    if t is None:
        if like is not None:
            return torch.empty_like(like) if like.dtype is dtype else torch.empty_like(like, dtype=dtype)
        return torch.empty(shape, dtype=dtype, device=device)
    _check(t, name, dtype, shape, device)
    return t


def _carry_shape(N: int, tokens: int, C: int, packed: bool):
    if packed:
        return (tokens // CARRY_TOKENS + N, C)
    return (N, -(-(tokens // N if N else 0) // CARRY_TOKENS), C)


def scan(x: torch.Tensor, g: torch.Tensor, beta: Optional[torch.Tensor] = None,
         h0: Optional[torch.Tensor] = None, *, h: Optional[torch.Tensor] = None,
         h_T: Optional[torch.Tensor] = None, save_carries: bool = False,
         status: Optional[torch.Tensor] = None):
    """The recurrence over B sequences of T tokens: returns (h [B,T,C], h_T [B,C] fp32).

    x, beta [B,T,C] fp32 or bf16 (beta None: 1); g [B,T,C] fp32 natural-log
    decays; h0 [B,C] fp32 or None (zeros).  h has x's type.  ``h`` / ``h_T`` may
    be given preallocated (``h_T`` may be ``h0``).  ``save_carries`` also returns
    the states before every 16th token ([B, ceil(T/16), C] fp32), which
    ``scan_backward`` takes."""
    shape, xt, dt, dev = _begin(x, "scan", "[B,T,C]")
    B, T, C = shape
    px = _expect(x, "x", xt, shape, dev)
    pg = _expect(g, "g", _F32, shape, dev)
    pb = _optional(beta, "beta", xt, shape, dev)
    p0 = _optional(h0, "h0", _F32, (B, C), dev)
    pst = _optional(status, "status", _I32, (1,), dev)
    h = _out(h, "h", xt, shape, dev, x)
    h_T = _out(h_T, "h_T", _F32, (B, C), dev)
    carries = torch.empty(_carry_shape(B, B * T, C, False), dtype=_F32, device=dev) \
        if save_carries else None
    _call(_lib.gdn_scan, dev, px, pg, pb, p0, h.data_ptr(), h_T.data_ptr(),
          None if carries is None else carries.data_ptr(), B, T, C, dt, pst)
    return (h, h_T, carries) if save_carries else (h, h_T)


def _packed(cu_seqlens, status, dev):
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N+1]")
    N = cu_seqlens.numel() - 1
    _fits("cu_seqlens", N)
    return (N, _expect(cu_seqlens, "cu_seqlens", _I32, (N + 1,), dev),
            _optional(status, "status", _I32, (1,), dev))


def scan_varlen(x: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor,
                beta: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None, *,
                h: Optional[torch.Tensor] = None, h_T: Optional[torch.Tensor] = None,
                save_carries: bool = False, status: Optional[torch.Tensor] = None):
    """``scan`` of N packed sequences: x, g, beta [total_T,C], cu_seqlens int32
    [N+1] on the device, h0 [N,C]; returns (h [total_T,C], h_T [N,C] fp32), and
    with ``save_carries`` the kept states ([total_T // 16 + N, C] fp32).  Tokens of no
    sequence are not written in h: give ``h`` if what is there matters."""
    shape, xt, dt, dev = _begin(x, "scan_varlen", "[total_T,C]")
    T, C = shape
    N, pcu, pst = _packed(cu_seqlens, status, dev)
    px = _expect(x, "x", xt, shape, dev)
    pg = _expect(g, "g", _F32, shape, dev)
    pb = _optional(beta, "beta", xt, shape, dev)
    p0 = _optional(h0, "h0", _F32, (N, C), dev)
    h = _out(h, "h", xt, shape, dev, x)
    h_T = _out(h_T, "h_T", _F32, (N, C), dev)
    carries = torch.empty(_carry_shape(N, T, C, True), dtype=_F32, device=dev) \
        if save_carries else None
    _call(_lib.gdn_scan_varlen, dev, px, pg, pb, p0, h.data_ptr(), h_T.data_ptr(),
          None if carries is None else carries.data_ptr(), pcu, N, T, C, dt, pst)
    return (h, h_T, carries) if save_carries else (h, h_T)


def scan_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
              beta: Optional[torch.Tensor] = None, *,
              h: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of B sequences; ``state`` [B,C] fp32 is updated in place.
    Returns h [B,C], the new state in x's type.

    x, beta [B,C] fp32 or bf16 (beta None: 1); g [B,C] fp32."""
    shape, xt, dt, dev = _begin(x, "scan_step", "[B,C]")
    B, C = shape
    px = _expect(x, "x", xt, shape, dev)
    pg = _expect(g, "g", _F32, shape, dev)
    ps = _expect(state, "state", _F32, shape, dev)
    pb = _optional(beta, "beta", xt, shape, dev)
    h = _out(h, "h", xt, shape, dev, x)
    _call(_lib.gdn_scan_step, dev, px, pg, pb, ps, h.data_ptr(), B, C, dt)
    return h


def _backward(fn, dh, x, g, beta, h0, dh_T, carries, N, tokens, packed, sizes, tail, begun):
    shape, xt, dt, dev = begun
    C = shape[-1]
    px = _expect(x, "x", xt, shape, dev)
    pg = _expect(g, "g", _F32, shape, dev)
    pb = _optional(beta, "beta", xt, shape, dev)
    p0 = _optional(h0, "h0", _F32, (N, C), dev)
    pdh = _expect(dh, "dh", xt, shape, dev)
    pdt = _optional(dh_T, "dh_T", _F32, (N, C), dev)
    kept = carries is not None
    carries = _out(carries, "carries", _F32, _carry_shape(N, tokens, C, packed), dev)
    dx = torch.empty_like(x)
    dg = torch.empty_like(g)
    dbeta = torch.empty_like(beta) if beta is not None else None
    dh0 = torch.empty_like(h0) if h0 is not None else None
    _call(fn, dev, px, pg, pb, p0, pdh, pdt, dx.data_ptr(), dg.data_ptr(),
          None if dbeta is None else dbeta.data_ptr(), None if dh0 is None else dh0.data_ptr(),
          carries.data_ptr(), int(kept), *sizes, C, dt, *tail)
    return dx, dg, dbeta, dh0


def scan_backward(dh: torch.Tensor, x: torch.Tensor, g: torch.Tensor,
                  beta: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                  dh_T: Optional[torch.Tensor] = None, *, carries: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None):
    """Gradients of ``scan``'s inputs: returns (dx, dg, dbeta, dh0), dbeta and dh0
    None where beta and h0 are.

    dh [B,T,C] has x's type, dh_T [B,C] fp32 or None (zeros).  ``carries`` is what
    ``scan(..., save_carries=True)`` returned for the same inputs; without it the
    states are computed again first."""
    begun = _begin(x, "scan_backward", "[B,T,C]")
    B, T, _ = begun[0]
    pst = _optional(status, "status", _I32, (1,), begun[3])
    return _backward(_lib.gdn_scan_backward, dh, x, g, beta, h0, dh_T, carries, B, B * T, False,
                     (B, T), (pst,), begun)


def scan_varlen_backward(dh: torch.Tensor, x: torch.Tensor, g: torch.Tensor,
                         cu_seqlens: torch.Tensor, beta: Optional[torch.Tensor] = None,
                         h0: Optional[torch.Tensor] = None, dh_T: Optional[torch.Tensor] = None, *,
                         carries: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None):
    """Gradients of ``scan_varlen``'s inputs, as ``scan_backward``.  Those of tokens
    before the first sequence and behind the last are zero; those of a sequence with
    invalid offsets (``status`` reports it) are not written."""
    begun = _begin(x, "scan_varlen_backward", "[total_T,C]")
    T = begun[0][0]
    N, pcu, pst = _packed(cu_seqlens, status, begun[3])
    return _backward(_lib.gdn_scan_varlen_backward, dh, x, g, beta, h0, dh_T, carries, N, T, True,
                     (pcu, N, T), (pst,), begun)
