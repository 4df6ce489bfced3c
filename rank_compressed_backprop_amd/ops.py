"""Operators around the linear layer: its forward with bias, activation and residual, its exact
backward from activations kept in 8 bits, and the RMS norm that feeds it (C ABI:
``include/instant_ops.h``, kernels in ``libinstant.so``).

The ``instant_*`` functions marshal arguments to the C entry points of the same names. The
functions below them take and return torch tensors: they check shapes, types and devices,
allocate outputs and workspace (from torch's allocator, on the current stream) and raise
``ValueError``, ``TypeError`` or ``InstantError``. Leading dimensions count as rows: x [..., K]
is a matrix of M rows. Inputs are contiguous, on the current device, and the work is enqueued
on its current stream. None of them is differentiable by itself: ``linear.py`` and ``norm.py``
build the layers.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import INSTANT_BF16, INSTANT_FP32, INSTANT_OK, InstantError, _lib, _ptr, _stream

CKPT_GROUP = 32
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_DTYPES = {torch.float32: INSTANT_FP32, torch.bfloat16: INSTANT_BF16}

_vp, _i, _sz, _st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
_sig = {
    "instant_ckpt_pack": (_st, [_vp, _i, _i, _i, _vp, _vp, _vp]),
    "instant_ckpt_unpack": (_st, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "instant_linear_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "instant_linear_fwd": (_st, [_vp] * 4 + [_i] * 5 + [_vp] * 5 + [_sz, _vp]),
    "instant_act_bwd": (_st, [_vp] * 4 + [_i] * 4 + [_vp] * 3 + [_sz, _vp]),
    "instant_linear_bwd": (_st, [_vp] * 5 + [_i] * 4 + [_vp] * 3 + [_sz, _vp]),
    "instant_rmsnorm_fwd": (_st, [_vp] * 3 + [_i] * 3 + [ctypes.c_float] + [_vp] * 6),
    "instant_rmsnorm_workspace_bytes": (_sz, [_i, _i]),
    "instant_rmsnorm_bwd": (_st, [_vp] * 5 + [_i] * 3 + [_vp] * 3 + [_sz, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


# ----------------------------------------------------------------------------- C names

def instant_ckpt_pack(x, M, C, dtype, q, scale, stream=None) -> int:
    return _lib.instant_ckpt_pack(_ptr(x), M, C, dtype, _ptr(q), _ptr(scale), _stream(stream))


def instant_ckpt_unpack(q, scale, M, C, dtype, x, stream=None) -> int:
    return _lib.instant_ckpt_unpack(_ptr(q), _ptr(scale), M, C, dtype, _ptr(x), _stream(stream))


def instant_linear_workspace_bytes(M, N, K, dtype) -> int:
    return int(_lib.instant_linear_workspace_bytes(M, N, K, dtype))


def instant_linear_fwd(x, w, bias, res, M, N, K, dtype, act, y, z, zq, zscale, workspace, workspace_bytes,
                       stream=None) -> int:
    return _lib.instant_linear_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(res), M, N, K, dtype, act, _ptr(y), _ptr(z),
                                   _ptr(zq), _ptr(zscale), _ptr(workspace), workspace_bytes, _stream(stream))


def instant_act_bwd(gy, z, zq, zscale, M, N, dtype, act, gz, gb, workspace, workspace_bytes, stream=None) -> int:
    return _lib.instant_act_bwd(_ptr(gy), _ptr(z), _ptr(zq), _ptr(zscale), M, N, dtype, act, _ptr(gz), _ptr(gb),
                                _ptr(workspace), workspace_bytes, _stream(stream))


def instant_linear_bwd(gz, w, x, xq, xscale, M, N, K, dtype, gx, gw, workspace, workspace_bytes, stream=None) -> int:
    return _lib.instant_linear_bwd(_ptr(gz), _ptr(w), _ptr(x), _ptr(xq), _ptr(xscale), M, N, K, dtype, _ptr(gx),
                                   _ptr(gw), _ptr(workspace), workspace_bytes, _stream(stream))


def instant_rmsnorm_fwd(x, res, g, M, C, dtype, eps, h, y, yq, yscale, rstd, stream=None) -> int:
    return _lib.instant_rmsnorm_fwd(_ptr(x), _ptr(res), _ptr(g), M, C, dtype, eps, _ptr(h), _ptr(y), _ptr(yq),
                                    _ptr(yscale), _ptr(rstd), _stream(stream))


def instant_rmsnorm_workspace_bytes(M, C) -> int:
    return int(_lib.instant_rmsnorm_workspace_bytes(M, C))


def instant_rmsnorm_bwd(gy, h, g, rstd, gh, M, C, dtype, gx, gg, workspace, workspace_bytes, stream=None) -> int:
    return _lib.instant_rmsnorm_bwd(_ptr(gy), _ptr(h), _ptr(g), _ptr(rstd), _ptr(gh), M, C, dtype, _ptr(gx), _ptr(gg),
                                    _ptr(workspace), workspace_bytes, _stream(stream))


# ----------------------------------------------------------------------------- checks

def _ok(status, where):
    if status != INSTANT_OK:
        raise InstantError(status, where)


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _on_device(t, name):
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")


def _matrix(t, name):
    """The first tensor of a call: (rows, columns, dtype code)."""
    code = _dtype(t, name)
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on_device(t, name)
    C = t.shape[-1]
    if C < 8 or C % 8:
        raise ValueError(f"{name}'s last dimension must be a positive multiple of 8, got {C}")
    M = t.numel() // C
    if M > 1 << 26:
        raise ValueError(f"{name} has {M} rows, more than 2^26")
    return M, C, code


def _like(t, shape, dtype, device, name):
    """Another tensor of the call: of this shape and type, beside the first."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(n, device):
    if n == 0:
        raise ValueError("sizes outside what the operator takes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _act(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return code


# ----------------------------------------------------------------------------- checkpoints

class Checkpoint8(NamedTuple):
    """An activation [..., C] in 8 bits: q int8 [..., C] and scale uint8 [..., ceil(C / 32)],
    biased power-of-two exponents. It stands for q * 2^(scale - 127) (see instant_ops.h)."""
    q: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        return self.q.shape


def _groups(C):
    return -(-C // CKPT_GROUP)


def _empty_ckpt(shape, device):
    return Checkpoint8(torch.empty(shape, dtype=torch.int8, device=device),
                       torch.empty((*shape[:-1], _groups(shape[-1])), dtype=torch.uint8, device=device))


def _ckpt(c, shape, device, name):
    _like(c.q, shape, torch.int8, device, f"{name}.q")
    _like(c.scale, torch.Size((*shape[:-1], _groups(shape[-1]))), torch.uint8, device, f"{name}.scale")


def checkpoint_pack(x) -> Checkpoint8:
    """x [..., C] in 8 bits."""
    M, C, dt = _matrix(x, "x")
    c = _empty_ckpt(x.shape, x.device)
    _ok(instant_ckpt_pack(x, M, C, dt, c.q, c.scale), "instant_ckpt_pack")
    return c


def checkpoint_unpack(c: Checkpoint8, dtype=torch.bfloat16) -> torch.Tensor:
    """The values of a checkpoint (exact in both types)."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    if c.q.dim() < 1 or c.q.shape[-1] < 8 or c.q.shape[-1] % 8:
        raise ValueError(f"a checkpoint's last dimension is a positive multiple of 8, got {tuple(c.q.shape)}")
    _on_device(c.q, "q")
    _ckpt(c, c.q.shape, c.q.get_device(), "checkpoint")
    C = c.q.shape[-1]
    x = torch.empty(c.q.shape, dtype=dtype, device=c.q.device)
    _ok(instant_ckpt_unpack(c.q, c.scale, c.q.numel() // C, C, _DTYPES[dtype], x), "instant_ckpt_unpack")
    return x


# ----------------------------------------------------------------------------- linear layer

def linear_forward(x, w, bias=None, residual=None, activation="none", save="none"):
    """y = act(x w^T + bias) + residual for x [..., K], w [N, K], bias [N], residual [..., N].

    save keeps the pre-activation for the backward: "z" in full, "z8" as a Checkpoint8 of the
    unrounded values, "none" not at all. Returns (y, what was kept or None)."""
    M, K, dt = _matrix(x, "x")
    act = _act(activation)
    if save not in ("none", "z", "z8"):
        raise ValueError(f"save must be none, z or z8, got {save!r}")
    if w.dim() != 2:
        raise ValueError(f"w must be [N, K], got {tuple(w.shape)}")
    N, dev = w.shape[0], x.get_device()
    _like(w, torch.Size((N, K)), x.dtype, dev, "w")
    shape = torch.Size((*x.shape[:-1], N))
    if bias is not None:
        _like(bias, torch.Size((N,)), x.dtype, dev, "bias")
    if residual is not None:
        _like(residual, shape, x.dtype, dev, "residual")
    n = instant_linear_workspace_bytes(M, N, K, dt)
    ws = _workspace(n, x.device)
    y = torch.empty(shape, dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if save == "z" else None
    z8 = _empty_ckpt(shape, x.device) if save == "z8" else None
    q, s = z8 if z8 is not None else (None, None)
    _ok(instant_linear_fwd(x, w, bias, residual, M, N, K, dt, act, y, z, q, s, ws, n), "instant_linear_fwd")
    return y, z8 if z8 is not None else z


def activation_backward(gy, z, activation="none", bias_grad=True):
    """(gz, gb): gz = gy * act'(z) and gb = sum over rows of gz (None unless bias_grad), with z a
    tensor like gy or a Checkpoint8 of its shape. With activation "none" gz is gy itself."""
    M, N, dt = _matrix(gy, "gy")
    act, dev = _act(activation), gy.get_device()
    if not act and not bias_grad:
        return gy, None
    q = s = None
    if not act:
        if z is not None:
            raise ValueError("activation 'none' takes no z")
    elif isinstance(z, Checkpoint8):
        _ckpt(z, gy.shape, dev, "z")
        q, s = z
        z = None
    elif z is None:
        raise ValueError(f"activation {activation!r} needs z")
    else:
        _like(z, gy.shape, gy.dtype, dev, "z")
    gz = torch.empty_like(gy) if act else None
    gb = ws = None
    n = 0
    if bias_grad:
        gb = torch.empty(N, dtype=gy.dtype, device=gy.device)
        n = instant_linear_workspace_bytes(M, N, 8, dt)
        ws = _workspace(n, gy.device)
    _ok(instant_act_bwd(gy, z, q, s, M, N, dt, act, gz, gb, ws, n), "instant_act_bwd")
    return gz if act else gy, gb


def linear_backward(gz, w, x, need_gx=True, need_gw=True):
    """(gx, gw) of z = x w^T: gx = gz w [..., K] and gw = gz^T x [N, K] (None where not needed),
    with x a tensor [..., K] or a Checkpoint8 of that shape."""
    M, N, dt = _matrix(gz, "gz")
    if not (need_gx or need_gw):
        return None, None
    if w.dim() != 2:
        raise ValueError(f"w must be [N, K], got {tuple(w.shape)}")
    K, dev = w.shape[1], gz.get_device()
    _like(w, torch.Size((N, K)), gz.dtype, dev, "w")
    shape = torch.Size((*gz.shape[:-1], K))
    q = s = None
    if isinstance(x, Checkpoint8):
        _ckpt(x, shape, dev, "x")
        q, s = x
        x = None
    elif need_gw:
        _like(x, shape, gz.dtype, dev, "x")
    else:
        x = None
    n = instant_linear_workspace_bytes(M, N, K, dt)
    ws = _workspace(n, gz.device)
    gx = torch.empty(shape, dtype=gz.dtype, device=gz.device) if need_gx else None
    gw = torch.empty((N, K), dtype=gz.dtype, device=gz.device) if need_gw else None
    _ok(instant_linear_bwd(gz, w, x, q, s, M, N, K, dt, gx, gw, ws, n), "instant_linear_bwd")
    return gx, gw


# ----------------------------------------------------------------------------- RMS norm

class NormOut(NamedTuple):
    """y (or None), h = x + residual (x itself without one), rstd float32 [...], y in 8 bits
    (or None)."""
    y: Optional[torch.Tensor]
    h: torch.Tensor
    rstd: torch.Tensor
    y8: Optional[Checkpoint8]


def rmsnorm_forward(x, weight, residual=None, eps=1e-6, y=True, y8=False) -> NormOut:
    """h = x + residual; y = h (mean(h^2) + eps)^(-1/2) * weight for x, residual [..., C] and
    weight [C]. y8 also (or with y=False only) writes y as a Checkpoint8."""
    M, C, dt = _matrix(x, "x")
    dev = x.get_device()
    if not (y or y8):
        raise ValueError("one of y and y8 has to be asked for")
    if not 0.0 <= eps < float("inf"):
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    _like(weight, torch.Size((C,)), x.dtype, dev, "weight")
    if residual is not None:
        _like(residual, x.shape, x.dtype, dev, "residual")
    h = torch.empty_like(x) if residual is not None else None
    out = torch.empty_like(x) if y else None
    c = _empty_ckpt(x.shape, x.device) if y8 else None
    q, s = c if c is not None else (None, None)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _ok(instant_rmsnorm_fwd(x, residual, weight, M, C, dt, eps, h, out, q, s, rstd), "instant_rmsnorm_fwd")
    return NormOut(out, x if h is None else h, rstd, c)


def rmsnorm_backward(gy, h, weight, rstd, gh=None, need_gweight=True):
    """(gx, gweight) for the gradient gy of y, with h and rstd from rmsnorm_forward. gh, the
    gradient that reaches h past the norm, is added to gx. gx is the gradient of x and of the
    residual."""
    M, C, dt = _matrix(gy, "gy")
    dev = gy.get_device()
    _like(h, gy.shape, gy.dtype, dev, "h")
    _like(weight, torch.Size((C,)), gy.dtype, dev, "weight")
    _like(rstd, gy.shape[:-1], torch.float32, dev, "rstd")
    if gh is not None:
        _like(gh, gy.shape, gy.dtype, dev, "gh")
    gx = torch.empty_like(gy)
    gw = ws = None
    n = 0
    if need_gweight:
        gw = torch.empty(C, dtype=gy.dtype, device=gy.device)
        n = instant_rmsnorm_workspace_bytes(M, C)
        ws = _workspace(n, gy.device)
    _ok(instant_rmsnorm_bwd(gy, h, weight, rstd, gh, M, C, dt, gx, gw, ws, n), "instant_rmsnorm_bwd")
    return gx, gw
