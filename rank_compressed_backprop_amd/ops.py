"""Operators around the linear layer: its forward with bias, activation and residual, its exact
backward from activations kept in 8 bits, and the RMS norm that feeds it; and operators at the
ends of a language model's training step: the embedding and its gradient, log probabilities from
logits and their gradient, the norm over all gradients and clipping (C ABI:
``include/instant_ops.h``, kernels in ``libinstant.so``).

The ``instant_*`` functions marshal arguments to the C entry points of the same names. The
functions below them take and return torch tensors: they check shapes, types and devices,
allocate outputs and workspace (from torch's allocator, on the current stream) and raise
``ValueError``, ``TypeError`` or ``InstantError``. Leading dimensions count as rows: x [..., K]
is a matrix of M rows. Inputs are contiguous, on the current device, and the work is enqueued
on its current stream. None of them is differentiable by itself: ``linear.py``, ``norm.py``,
``embedding.py`` and ``loss.py`` build the layers.
"""
from __future__ import annotations

import array
import ctypes
import functools
import math
from typing import NamedTuple, Optional

import torch
from torch import Tensor

from . import INSTANT_BF16, INSTANT_FP32, INSTANT_OK, InstantError, _lib, _ptr, _stream

CKPT_GROUP = 32
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_DTYPES = {torch.float32: INSTANT_FP32, torch.bfloat16: INSTANT_BF16}

IGNORE = -100  # the target of a row without a token
MAX_VOCAB = 1 << 18
MAX_TOP = 32
_TOKENS = {torch.int64: 8, torch.int32: 4}

_vp, _i, _sz, _st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
_f, _l = ctypes.c_float, ctypes.c_int64
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
    "instant_embed_fwd": (_st, [_vp, _i, _i, _vp, _i, _i, _i, _f, _vp, _vp]),
    "instant_embed_workspace_bytes": (_sz, [_i, _i, _i]),
    "instant_embed_bwd": (_st, [_vp, _vp] + [_i] * 5 + [_f, _l, _i, _vp, _vp, _sz, _vp]),
    "instant_logprobs_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "instant_logprobs_fwd": (_st, [_vp, _vp] + [_i] * 5 + [_l, _i] + [_vp] * 7 + [_sz, _vp]),
    "instant_logprobs_bwd": (_st, [_vp, _vp] + [_i] * 5 + [_l] + [_vp] * 7),
    "instant_grad_norm_workspace_bytes": (_sz, [_i]),
    "instant_grad_norm": (_st, [_vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "instant_clip_grads": (_st, [_vp] * 5 + [_i, _f, _vp, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

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


def instant_embed_fwd(tokens, token_bytes, M, table, V, C, dtype, scale, y, stream=None) -> int:
    return _lib.instant_embed_fwd(_ptr(tokens), token_bytes, M, _ptr(table), V, C, dtype, scale, _ptr(y),
                                  _stream(stream))


def instant_embed_workspace_bytes(M, V, C) -> int:
    return int(_lib.instant_embed_workspace_bytes(M, V, C))


def instant_embed_bwd(gy, tokens, token_bytes, M, V, C, dtype, scale, padding, accumulate, gtable, workspace,
                      workspace_bytes, stream=None) -> int:
    return _lib.instant_embed_bwd(_ptr(gy), _ptr(tokens), token_bytes, M, V, C, dtype, scale, padding, int(accumulate),
                                  _ptr(gtable), _ptr(workspace), workspace_bytes, _stream(stream))


def instant_logprobs_workspace_bytes(M, V, dtype, k) -> int:
    return int(_lib.instant_logprobs_workspace_bytes(M, V, dtype, k))


def instant_logprobs_fwd(logits, targets, token_bytes, M, W, V, dtype, ignore, k, logp, lse, entropy, stats, top_logp,
                         top_index, workspace, workspace_bytes, stream=None) -> int:
    return _lib.instant_logprobs_fwd(_ptr(logits), _ptr(targets), token_bytes, M, W, V, dtype, ignore, k, _ptr(logp),
                                     _ptr(lse), _ptr(entropy), _ptr(stats), _ptr(top_logp), _ptr(top_index),
                                     _ptr(workspace), workspace_bytes, _stream(stream))


def instant_logprobs_bwd(logits, targets, token_bytes, M, W, V, dtype, ignore, stats, entropy, g_logp, g_lse,
                         g_entropy, gz, stream=None) -> int:
    return _lib.instant_logprobs_bwd(_ptr(logits), _ptr(targets), token_bytes, M, W, V, dtype, ignore, _ptr(stats),
                                     _ptr(entropy), _ptr(g_logp), _ptr(g_lse), _ptr(g_entropy), _ptr(gz),
                                     _stream(stream))


class _Host:
    """A host array of the call ('Q' addresses, 'q' int64, 'i' int32) and its address (NULL for None). The
    caller keeps it until the call returns."""
    __slots__ = ("held", "at")

    def __init__(self, code, values):
        self.held = None if values is None else array.array(code, values)
        self.at = None if values is None else self.held.buffer_info()[0]


def _addresses(tensors):
    return None if tensors is None else [_ptr(t) or 0 for t in tensors]


def instant_grad_norm_workspace_bytes(n) -> int:
    return int(_lib.instant_grad_norm_workspace_bytes(n))


def instant_grad_norm(grads, count, dtype, n, norm, workspace, workspace_bytes, stream=None) -> int:
    """grads (tensors or addresses), count and dtype are sequences of n."""
    g, c, d = _Host("Q", _addresses(grads)), _Host("q", count), _Host("i", dtype)
    return _lib.instant_grad_norm(g.at, c.at, d.at, n, _ptr(norm), _ptr(workspace), workspace_bytes, _stream(stream))


def instant_clip_grads(grads, count, dtype, out, out_dtype, n, max_norm, norm, workspace, workspace_bytes,
                       stream=None) -> int:
    """grads, count, dtype, out and out_dtype are sequences of n."""
    g, c, d = _Host("Q", _addresses(grads)), _Host("q", count), _Host("i", dtype)
    o, e = _Host("Q", _addresses(out)), _Host("i", out_dtype)
    return _lib.instant_clip_grads(g.at, c.at, d.at, o.at, e.at, n, max_norm, _ptr(norm), _ptr(workspace),
                                   workspace_bytes, _stream(stream))


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


def _tokens(t, name):
    """Bytes of an integer of a token tensor."""
    if not isinstance(t, Tensor):
        _foreign(t, name)
    size = _TOKENS.get(t.dtype)
    if size is None:
        raise TypeError(f"{name} must be int64 or int32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return size


def _beside(t, shape, device, name):
    """A token tensor beside the first tensor of the call."""
    size = _tokens(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    return size


def _finite(v, name):
    if not math.isfinite(v) or abs(v) > 3.4028234663852886e38:
        raise ValueError(f"{name} must be a finite float32, got {v}")


# A kernel writes through an address, which autograd does not see: a call that writes a tensor of
# its caller's says so, and a backward pass that has saved it raises instead of using what it holds now.
_written = torch.autograd.graph.increment_version

# Sizes depend on the shapes alone.
_fwd_bytes = functools.lru_cache(4096)(instant_linear_fwd_workspace_bytes)
_gx_bytes = functools.lru_cache(4096)(instant_linear_gx_workspace_bytes)
_gw_bytes = functools.lru_cache(4096)(instant_linear_gw_workspace_bytes)
_act_bytes = functools.lru_cache(4096)(instant_act_bwd_workspace_bytes)
_norm_bytes = functools.lru_cache(4096)(instant_rmsnorm_workspace_bytes)
_logprobs_bytes = functools.lru_cache(4096)(instant_logprobs_workspace_bytes)
_embed_bytes = functools.lru_cache(4096)(instant_embed_workspace_bytes)
_grads_bytes = functools.lru_cache(4096)(instant_grad_norm_workspace_bytes)


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


def weight_parameter(weight, device, dtype) -> torch.nn.Parameter:
    """A layer's weight from the one that its caller hands over. A Parameter of this device and type,
    contiguous, is taken as it is: handed to two layers, it is one leaf with one gradient. Anything
    else is copied: no two Parameters share memory, which would each get a part of the gradient and
    an optimizer would step twice."""
    if (isinstance(weight, torch.nn.Parameter) and weight.dtype == dtype and weight.is_contiguous()
            and weight.device == torch.empty(0, device=device).device):
        return weight
    return torch.nn.Parameter(weight.detach().to(device=device, dtype=dtype, copy=True,
                                                 memory_format=torch.contiguous_format))


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


# ----------------------------------------------------------------------------- embedding

def embedding_forward(tokens, table, scale=1.0):
    """y = scale * table[tokens] [..., C] for tokens [...] (int64 or int32) and table [V, C]. A
    token outside 0 .. V - 1 gives a row of NaN."""
    size = _tokens(tokens, "tokens")
    dt = _dtype(table, "table")
    if table.dim() != 2:
        raise ValueError(f"table must be [V, C], got {tuple(table.shape)}")
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    V, C = table.shape
    _vocab(V, "table")
    if C < 8 or C % 8:
        raise ValueError(f"table's last dimension must be a positive multiple of 8, got {C}")
    _finite(scale, "scale")
    M = tokens.numel()
    if M > 1 << 26:
        raise ValueError(f"tokens are {M}, more than 2^26")
    _on_device(table, "table")
    dev = table.get_device()
    if tokens.get_device() != dev:
        raise ValueError(f"tokens must be on the current CUDA device, got {tokens.device}")
    y = table.new_empty((*tokens.shape, C))
    _ok(_lib.instant_embed_fwd(tokens.data_ptr(), size, M, table.data_ptr(), V, C, dt, scale, y.data_ptr(),
                               _current(dev)), "instant_embed_fwd")
    return y


def _vocab(V, name):
    if not 1 <= V <= MAX_VOCAB:
        raise ValueError(f"{name}: a vocabulary is of 1 to {MAX_VOCAB} tokens, got {V}")


def embedding_backward(gy, tokens, vocab, scale=1.0, padding=None, into=None):
    """The table's gradient [vocab, C]: scale * the sums of gy's rows [..., C] by their tokens
    [...], with the same bits every time; rows of the token `padding` take no part, nor does a token
    outside the vocabulary. into: a gradient [vocab, C] that the sums are added to, in place (rows
    without a token are not touched), and which is returned. At most 2^22 tokens."""
    M, C, dt = _matrix(gy, "gy")
    dev = gy.get_device()
    size = _beside(tokens, gy.shape[:-1], dev, "tokens")
    _vocab(vocab, "vocab")
    _finite(scale, "scale")
    if padding is None:
        padding = -1
    elif not 0 <= padding < vocab:
        raise ValueError(f"padding must be a token of the vocabulary, got {padding}")
    if M > 1 << 22:
        raise ValueError(f"gy has {M} rows, more than 2^22")
    if into is not None:
        _like(into, (vocab, C), gy.dtype, dev, "into")
    gw = gy.new_empty((vocab, C)) if into is None else into
    n = _embed_bytes(M, vocab, C)
    ws, wp = _workspace(n, gy)
    _ok(_lib.instant_embed_bwd(gy.data_ptr(), tokens.data_ptr(), size, M, vocab, C, dt, scale, padding,
                               into is not None, gw.data_ptr(), wp, n, _current(dev)), "instant_embed_bwd")
    if into is not None:
        _written(into)
    return gw


# ----------------------------------------------------------------------------- log probabilities

class TokenLogprobs(NamedTuple):
    """Of logits [..., W] (float32 but for the places): logp, the log probability of the target
    (None without targets), lse = log sum exp, entropy [...]; the alternatives' top_logp and
    top_index (int64) [..., k], likeliest first (None unless asked for); stats [..., 2], what the
    gradient needs."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_index: Optional[torch.Tensor]
    stats: torch.Tensor


def _logits(z, vocab):
    """(rows, width, vocabulary, dtype code) of logits, whose rows may have any width."""
    dt = _dtype(z, "logits")
    if z.dim() < 1:
        raise ValueError("logits must have at least one dimension")
    if not z.is_contiguous():
        raise ValueError("logits must be contiguous")
    W = z.shape[-1]
    _vocab(W, "logits")
    V = W if vocab is None else vocab
    if not 1 <= V <= W:
        raise ValueError(f"vocab must be 1 to the {W} columns of logits, got {V}")
    M = z.numel() // W
    if M > 1 << 26:
        raise ValueError(f"logits have {M} rows, more than 2^26")
    _on_device(z, "logits")
    return M, W, V, dt


def _int64(v, name):
    if not -(1 << 63) <= v < 1 << 63:
        raise ValueError(f"{name} must be an int64, got {v}")


def token_logprobs(logits, targets=None, vocab=None, top=0, ignore=IGNORE) -> TokenLogprobs:
    """Log probabilities of the tokens targets [...] (int64 or int32) under logits [..., W], the
    entropy, and the `top` <= 32 likeliest alternatives (equal logits by their place). vocab: only
    the first vocab columns count (a padded vocabulary). Where the target is `ignore` its log
    probability is 0; where it is outside the vocabulary, NaN. A logit of -inf has probability 0;
    a row of nothing else has lse -inf and entropy 0."""
    M, W, V, dt = _logits(logits, vocab)
    shape, dev = logits.shape[:-1], logits.get_device()
    size = 8 if targets is None else _beside(targets, shape, dev, "targets")
    if not 0 <= top <= min(MAX_TOP, V):
        raise ValueError(f"top must be 0 to {min(MAX_TOP, V)}, got {top}")
    _int64(ignore, "ignore")
    lse = logits.new_empty(shape, dtype=torch.float32)
    entropy = torch.empty_like(lse)
    logp = torch.empty_like(lse) if targets is not None else None
    stats = logits.new_empty((*shape, 2), dtype=torch.float32)
    tl = ti = None
    if top:
        tl = logits.new_empty((*shape, top), dtype=torch.float32)
        ti = logits.new_empty((*shape, top), dtype=torch.int64)
    n = _logprobs_bytes(M, V, dt, top)
    ws, wp = _workspace(n, logits)
    _ok(_lib.instant_logprobs_fwd(logits.data_ptr(), _p(targets), size, M, W, V, dt, ignore, top, _p(logp),
                                  lse.data_ptr(), entropy.data_ptr(), stats.data_ptr(), _p(tl), _p(ti), wp, n,
                                  _current(dev)), "instant_logprobs_fwd")
    return TokenLogprobs(logp, lse, entropy, tl, ti, stats)


def token_logprobs_backward(logits, targets, stats, g_logp=None, g_lse=None, g_entropy=None, entropy=None, vocab=None,
                            ignore=IGNORE, in_place=False):
    """The gradient of logits (of their shape and type) for the gradients g_logp, g_lse and
    g_entropy [...] of token_logprobs' results, with its stats and (for g_entropy) its entropy:
    g_logp (1[j = target] - p) + g_lse p - g_entropy p (log p + entropy), zeros behind the
    vocabulary. A row whose gradients are all 0 gets zeros, whatever it holds (with g_logp, unless its
    target is outside the vocabulary: NaN). in_place: it is written over logits and logits are
    returned; a later backward pass that has saved them raises."""
    M, W, V, dt = _logits(logits, vocab)
    shape, dev = logits.shape[:-1], logits.get_device()
    if g_logp is None and g_lse is None and g_entropy is None:
        raise ValueError("one of g_logp, g_lse and g_entropy has to be given")
    if targets is None and g_logp is not None:
        raise ValueError("targets are needed for g_logp")
    if entropy is None and g_entropy is not None:
        raise ValueError("entropy is needed for g_entropy")
    size = 8 if targets is None else _beside(targets, shape, dev, "targets")
    _like(stats, (*shape, 2), torch.float32, dev, "stats")
    for t, name in ((g_logp, "g_logp"), (g_lse, "g_lse"), (g_entropy, "g_entropy"), (entropy, "entropy")):
        if t is not None:
            _like(t, shape, torch.float32, dev, name)
    _int64(ignore, "ignore")
    gz = logits if in_place else torch.empty_like(logits)
    _ok(_lib.instant_logprobs_bwd(logits.data_ptr(), _p(targets), size, M, W, V, dt, ignore, stats.data_ptr(),
                                  _p(entropy), _p(g_logp), _p(g_lse), _p(g_entropy), gz.data_ptr(), _current(dev)),
        "instant_logprobs_bwd")
    if in_place:
        _written(logits)
    return gz


# ----------------------------------------------------------------------------- gradients of a model

def _grads(tensors, name):
    """Of a sequence of tensors: a list of them, and of each the address, the elements and the dtype code
    (a model has hundreds: each question is put to all of them at once)."""
    if isinstance(tensors, Tensor):
        raise TypeError(f"{name} must be a sequence of tensors, got a tensor")
    tensors = list(tensors)
    if not tensors:
        raise ValueError(f"{name} must hold a tensor at least")
    try:
        codes = [_DTYPES[t.dtype] for t in tensors]
        devices = set(map(Tensor.get_device, tensors))
    except (KeyError, AttributeError, TypeError):
        for t in tensors:  # says which it is
            _dtype(t, name)
        raise
    if devices != {torch.cuda.current_device() if torch.cuda.is_available() else None}:
        raise ValueError(f"{name} must be on the current CUDA device, got {[str(t.device) for t in tensors]}")
    if not all(map(Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    return tensors, list(map(Tensor.data_ptr, tensors)), list(map(Tensor.numel, tensors)), codes


def grad_norm(tensors) -> torch.Tensor:
    """The Euclidean norm over all elements of a sequence of tensors (float32 and bfloat16 in any
    mixture, of any shapes), a float32 scalar on the device. Squares are summed in float64."""
    tensors, at, count, codes = _grads(tensors, "tensors")
    first, n = tensors[0], len(at)
    norm = first.new_empty((), dtype=torch.float32)
    size = _grads_bytes(n)
    ws, wp = _workspace(size, first)
    g, c, d = _Host("Q", at), _Host("q", count), _Host("i", codes)
    _ok(_lib.instant_grad_norm(g.at, c.at, d.at, n, norm.data_ptr(), wp, size, _current(first.get_device())),
        "instant_grad_norm")
    return norm


def clip_grads(tensors, max_norm, out=None) -> torch.Tensor:
    """Scales a sequence of tensors so that the norm over all their elements is at most max_norm:
    by max_norm / (norm + 1e-6) where that is below 1, else not at all. Returns the norm before (a
    float32 scalar on the device; nothing waits for it). out: as many tensors of as many elements each,
    float32 or bfloat16, that receive the result; None: the tensors themselves. Outputs may not share memory
    with each other or with another tensor of the call."""
    tensors, at, count, codes = _grads(tensors, "tensors")
    if not max_norm >= 0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    first, n = tensors[0], len(at)
    to, to_codes = at, codes
    if out is not None:
        out, to, to_count, to_codes = _grads(out, "out")
        if to_count != count:
            raise ValueError(f"out must hold tensors of {count} elements, got {to_count}")
    norm = first.new_empty((), dtype=torch.float32)
    size = _grads_bytes(n)
    ws, wp = _workspace(size, first)
    g, c, d, o, e = _Host("Q", at), _Host("q", count), _Host("i", codes), _Host("Q", to), _Host("i", to_codes)
    _ok(_lib.instant_clip_grads(g.at, c.at, d.at, o.at, e.at, n, max_norm, norm.data_ptr(), wp, size,
                                _current(first.get_device())), "instant_clip_grads")
    _written(tensors if out is None else out)
    return norm
