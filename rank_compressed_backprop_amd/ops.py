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
import functools
from typing import NamedTuple, Optional

import torch
from torch import Tensor

from . import INSTANT_BF16, INSTANT_FP32, INSTANT_OK, InstantError, _lib, _ptr, _stream

CKPT_GROUP = 32
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_DTYPES = {torch.float32: INSTANT_FP32, torch.bfloat16: INSTANT_BF16}

_vp, _i, _sz, _st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
_sig = {
    "instant_ckpt_pack": (_st, [_vp, _i, _i, _i, _vp, _vp, _vp]),
    "instant_ckpt_unpack": (_st, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "instant_linear_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "instant_linear_fwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "instant_linear_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "instant_linear_gx_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "instant_linear_gw_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "instant_act_bwd_workspace_bytes": (_sz, [_i, _i, _i]),
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


def instant_linear_fwd_workspace_bytes(M, N, K, dtype) -> int:
    return int(_lib.instant_linear_fwd_workspace_bytes(M, N, K, dtype))


def instant_linear_bwd_workspace_bytes(M, N, K, dtype, x_ckpt) -> int:
    return int(_lib.instant_linear_bwd_workspace_bytes(M, N, K, dtype, int(x_ckpt)))


def instant_linear_gx_workspace_bytes(M, N, K, dtype) -> int:
    return int(_lib.instant_linear_gx_workspace_bytes(M, N, K, dtype))


def instant_linear_gw_workspace_bytes(M, N, K, dtype, x_ckpt) -> int:
    return int(_lib.instant_linear_gw_workspace_bytes(M, N, K, dtype, int(x_ckpt)))


def instant_act_bwd_workspace_bytes(M, N, dtype) -> int:
    return int(_lib.instant_act_bwd_workspace_bytes(M, N, dtype))


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


def _foreign(t, name):
    raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")


def _dtype(t, name):
    if not isinstance(t, Tensor):
        _foreign(t, name)
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
    if not isinstance(t, Tensor):
        _foreign(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# Sizes depend on the shapes alone.
_fwd_bytes = functools.lru_cache(4096)(instant_linear_fwd_workspace_bytes)
_gx_bytes = functools.lru_cache(4096)(instant_linear_gx_workspace_bytes)
_gw_bytes = functools.lru_cache(4096)(instant_linear_gw_workspace_bytes)
_act_bytes = functools.lru_cache(4096)(instant_act_bwd_workspace_bytes)
_norm_bytes = functools.lru_cache(4096)(instant_rmsnorm_workspace_bytes)


def _workspace(n, like):
    """n bytes of workspace (None if none are needed) and their address. The caller keeps the
    tensor until its launches are enqueued; the allocator orders its reuse after them."""
    if n == 0:
        return None, None
    ws = like.new_empty(n, dtype=torch.uint8)
    return ws, ws.data_ptr()


# The current stream of the current device, on which every input lies.
def _current(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _p(t):
    return None if t is None else t.data_ptr()


def _act(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return code


def differentiated_once(backward):
    """Decorator of a layer's backward pass on these operators. Its results have no graph, so a
    second derivative would silently lack the layer's terms: create_graph=True (which runs
    backward passes with gradients enabled) is refused."""
    @functools.wraps(backward)
    def checked(ctx, *grads):
        if torch.is_grad_enabled():
            raise RuntimeError("the backward pass of this layer cannot be differentiated again (create_graph=True)")
        return backward(ctx, *grads)
    return checked


# ----------------------------------------------------------------------------- checkpoints

class Checkpoint8(NamedTuple):
    """An activation [..., C] in 8 bits: q int8 [..., C] and scale uint8 [..., ceil(C / 32)],
    biased power-of-two exponents. It stands for q * 2^(scale - 127) (see instant_ops.h)."""
    q: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        return self.q.shape


def _empty_ckpt(shape, like):
    return Checkpoint8(like.new_empty(shape, dtype=torch.int8),
                       like.new_empty((*shape[:-1], -(-shape[-1] // CKPT_GROUP)), dtype=torch.uint8))


def check_checkpoint(c, shape, device, name):
    """Raises unless c is a checkpoint of a tensor of this shape on this device (its index)."""
    _like(c.q, shape, torch.int8, device, name + ".q")
    _like(c.scale, (*shape[:-1], -(-shape[-1] // CKPT_GROUP)), torch.uint8, device, name + ".scale")


def checkpoint_pack(x) -> Checkpoint8:
    """x [..., C] in 8 bits."""
    M, C, dt = _matrix(x, "x")
    c = _empty_ckpt(x.shape, x)
    _ok(_lib.instant_ckpt_pack(x.data_ptr(), M, C, dt, c.q.data_ptr(), c.scale.data_ptr(), _current(x.get_device())),
        "instant_ckpt_pack")
    return c


def checkpoint_unpack(c: Checkpoint8, dtype=torch.bfloat16) -> torch.Tensor:
    """The values of a checkpoint (exact in both types)."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    if not isinstance(c, Checkpoint8):
        raise TypeError(f"a checkpoint must be a Checkpoint8, got {type(c).__name__}")
    if not isinstance(c.q, Tensor):
        _foreign(c.q, "checkpoint.q")
    q, shape = c.q, c.q.shape
    if q.dim() < 1 or shape[-1] < 8 or shape[-1] % 8:
        raise ValueError(f"a checkpoint's last dimension is a positive multiple of 8, got {tuple(shape)}")
    _on_device(q, "q")
    dev = q.get_device()
    check_checkpoint(c, shape, dev, "checkpoint")
    C = shape[-1]
    x = torch.empty_like(q, dtype=dtype)
    _ok(_lib.instant_ckpt_unpack(q.data_ptr(), c.scale.data_ptr(), q.numel() // C, C, code, x.data_ptr(),
                                 _current(dev)), "instant_ckpt_unpack")
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
    if not isinstance(w, Tensor):
        _foreign(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w must be [N, K], got {tuple(w.shape)}")
    N, dev = w.shape[0], x.get_device()
    _like(w, (N, K), x.dtype, dev, "w")
    if N < 8 or N % 8:
        raise ValueError(f"w must have a positive multiple of 8 rows, got {N}")
    shape = (*x.shape[:-1], N)
    if bias is not None:
        _like(bias, (N,), x.dtype, dev, "bias")
    if residual is not None:
        _like(residual, shape, x.dtype, dev, "residual")
    n = _fwd_bytes(M, N, K, dt)
    ws, wp = _workspace(n, x)
    y = x.new_empty(shape)
    kept = z = q = s = None
    if save == "z":
        kept = torch.empty_like(y)
        z = kept.data_ptr()
    elif save == "z8":
        kept = _empty_ckpt(shape, x)
        q, s = kept.q.data_ptr(), kept.scale.data_ptr()
    _ok(_lib.instant_linear_fwd(x.data_ptr(), w.data_ptr(), _p(bias), _p(residual), M, N, K, dt, act, y.data_ptr(), z,
                                q, s, wp, n, _current(dev)), "instant_linear_fwd")
    return y, kept


def activation_backward(gy, z, activation="none", bias_grad=True):
    """(gz, gb): gz = gy * act'(z) and gb = sum over rows of gz (None unless bias_grad), with z a
    tensor like gy or a Checkpoint8 of its shape. With activation "none" gz is gy itself."""
    M, N, dt = _matrix(gy, "gy")
    act, dev = _act(activation), gy.get_device()
    zp = q = s = None
    if not act:
        if z is not None:
            raise ValueError("activation 'none' takes no z")
        if not bias_grad:
            return gy, None
    elif isinstance(z, Checkpoint8):
        check_checkpoint(z, gy.shape, dev, "z")
        q, s = z.q.data_ptr(), z.scale.data_ptr()
    elif z is None:
        raise ValueError(f"activation {activation!r} needs z")
    else:
        _like(z, gy.shape, gy.dtype, dev, "z")
        zp = z.data_ptr()
    gz = torch.empty_like(gy) if act else None
    gb = ws = wp = None
    n = 0
    if bias_grad:
        gb = gy.new_empty(N)
        n = _act_bytes(M, N, dt)
        ws, wp = _workspace(n, gy)
    _ok(_lib.instant_act_bwd(gy.data_ptr(), zp, q, s, M, N, dt, act, _p(gz), _p(gb), wp, n, _current(dev)),
        "instant_act_bwd")
    return gz if act else gy, gb


def linear_backward(gz, w, x, need_gx=True, need_gw=True):
    """(gx, gw) of z = x w^T: gx = gz w [..., K] and gw = gz^T x [N, K] (None where not needed),
    with x a tensor [..., K] or a Checkpoint8 of that shape."""
    M, N, dt = _matrix(gz, "gz")
    if not (need_gx or need_gw):
        return None, None
    if not isinstance(w, Tensor):
        _foreign(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w must be [N, K], got {tuple(w.shape)}")
    K, dev = w.shape[1], gz.get_device()
    _like(w, (N, K), gz.dtype, dev, "w")
    if K < 8 or K % 8:
        raise ValueError(f"w must have a positive multiple of 8 columns, got {K}")
    shape = (*gz.shape[:-1], K)
    xp = q = s = None
    if isinstance(x, Checkpoint8):
        check_checkpoint(x, shape, dev, "x")
        q, s = x.q.data_ptr(), x.scale.data_ptr()
    elif need_gw:
        if x is None:
            raise ValueError("x is needed for the weight's gradient")
        _like(x, shape, gz.dtype, dev, "x")
        xp = x.data_ptr()
    n = max(_gx_bytes(M, N, K, dt) if need_gx else 0, _gw_bytes(M, N, K, dt, q is not None) if need_gw else 0)
    ws, wp = _workspace(n, gz)
    gx = gz.new_empty(shape) if need_gx else None
    gw = torch.empty_like(w) if need_gw else None
    _ok(_lib.instant_linear_bwd(gz.data_ptr(), w.data_ptr(), xp, q, s, M, N, K, dt, _p(gx), _p(gw), wp, n,
                                _current(dev)), "instant_linear_bwd")
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
    _like(weight, (C,), x.dtype, dev, "weight")
    if residual is not None:
        _like(residual, x.shape, x.dtype, dev, "residual")
    h = torch.empty_like(x) if residual is not None else None
    out = torch.empty_like(x) if y else None
    c = q = s = None
    if y8:
        c = _empty_ckpt(x.shape, x)
        q, s = c.q.data_ptr(), c.scale.data_ptr()
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    _ok(_lib.instant_rmsnorm_fwd(x.data_ptr(), _p(residual), weight.data_ptr(), M, C, dt, eps, _p(h), _p(out), q, s,
                                 rstd.data_ptr(), _current(dev)), "instant_rmsnorm_fwd")
    return NormOut(out, x if h is None else h, rstd, c)


def rmsnorm_backward(gy, h, weight, rstd, gh=None, need_gweight=True):
    """(gx, gweight) for the gradient gy of y, with h and rstd from rmsnorm_forward. gh, the
    gradient that reaches h past the norm, is added to gx. gx is the gradient of x and of the
    residual."""
    M, C, dt = _matrix(gy, "gy")
    dev = gy.get_device()
    _like(h, gy.shape, gy.dtype, dev, "h")
    _like(weight, (C,), gy.dtype, dev, "weight")
    _like(rstd, gy.shape[:-1], torch.float32, dev, "rstd")
    if gh is not None:
        _like(gh, gy.shape, gy.dtype, dev, "gh")
    gx = torch.empty_like(gy)
    gw = ws = wp = None
    n = 0
    if need_gweight:
        gw = torch.empty_like(weight)
        n = _norm_bytes(M, C)
        ws, wp = _workspace(n, gy)
    _ok(_lib.instant_rmsnorm_bwd(gy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), _p(gh), M, C, dt,
                                 gx.data_ptr(), _p(gw), wp, n, _current(dev)), "instant_rmsnorm_bwd")
    return gx, gw
