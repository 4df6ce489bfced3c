"""Training-step integration of the INSTANT low-rank backward: a linear layer y = x w^T
(optionally with bias, activation and residual) whose backward runs through the library (notes "INSTANT: Compressing Gradients
and Activations for Resource-Efficient Training", 整体框架: calibrate every N_t steps,
compress and run the low-rank backward in between; 关键设计 3 for the backward).

Schedule of each window of N_t training steps (the library leaves it to the caller):

  - steps 0 .. N_cal-1 of the window are calibration steps: the forward keeps x, the
    backward is exact (PyTorch GEMMs) and also hands x and g_y to the library's
    statistics; the last of them finalizes, which installs the new P and Q;
  - the other steps keep only x_hat = P x from the forward (the activation memory saving)
    and run the library's low-rank backward.

Until a finalize has succeeded there are no projections, and a step that is not a
calibration step falls back to the exact backward. A failed finalize keeps the previous
projections (the library's rule), so the layer keeps compressing with them.

For the plain layer only the forward GEMM and the exact backward of calibration steps are
PyTorch's; every step of the INSTANT path (statistics, decomposition, truncation, compression,
low-rank backward) runs in the HIP kernels of libinstant.so. With a bias, an activation, a
residual or checkpoints in 8 bits the rest does too (ops.py): the forward is one product with
its epilogue, the exact steps keep x and the pre-activation in 8 bits instead of x in full
(checkpoint="int8"), and the low-rank steps run on the gradient behind the activation. One
forward and one backward per step, in order, on the layer's device.
"""
from __future__ import annotations

import math

import torch

from . import INSTANT_OK, InstantLayer, instant_status_str, make_config, ops


class _InstantLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, mod, mode):
        y = torch.nn.functional.linear(x, w)  # the caller's GEMM
        B = x.shape[0]
        if mode == "compress":
            xhat = torch.empty((B, mod.Rx, mod.Cx), dtype=x.dtype, device=x.device)
            mod.layer.compress_fwd(x, B, xhat)
            ctx.save_for_backward(xhat, w)
        else:
            ctx.save_for_backward(x, w)
        ctx.mod, ctx.mode = mod, mode
        return y

    @staticmethod
    def backward(ctx, gy):
        saved, w = ctx.saved_tensors
        mod, mode = ctx.mod, ctx.mode
        gy = gy.contiguous()
        B = gy.shape[0]
        if mode == "compress":
            gw = torch.empty_like(w)
            gx = torch.empty((B, mod.L, mod.Cx), dtype=gy.dtype, device=gy.device)
            mod.layer.backward(saved, gy, w, B, gw, gx)
            return gx, gw, None, None
        x = saved
        gx = torch.matmul(gy.reshape(-1, mod.Cy), w).reshape(B, mod.L, mod.Cx)
        gw = torch.mm(gy.reshape(-1, mod.Cy).t().contiguous(), x.reshape(-1, mod.Cx))
        if mode in ("calibrate", "finalize"):
            mod._calibrate(x, gy, B, finalize=(mode == "finalize"))
        return gx, gw, None, None


class _FusedLinearFn(torch.autograd.Function):
    """y = act(x w^T + b) + r on the library's products. In 8 bits x is kept as q, scale (x8, or
    packed here) and its statistics are taken in the forward, while x is at hand; the gradient's
    are taken in the backward either way (split and joint calls sum identically)."""

    @staticmethod
    def forward(ctx, x, w, b, r, q, scale, mod, mode):
        eight = mod.checkpoint == "int8"
        save = "none" if mod.activation == "none" else "z8" if eight else "z"
        y, z = ops.linear_forward(x, w, b, r, mod.activation, save)
        B = x.shape[0]
        kept = [x]
        if mode == "compress":
            xhat = torch.empty((B, mod.Rx, mod.Cx), dtype=x.dtype, device=x.device)
            mod.layer.compress_fwd(x, B, xhat)
            kept = [xhat]
        elif eight:
            kept = [q, scale] if q is not None else list(ops.checkpoint_pack(x))
            if mode in ("calibrate", "finalize"):
                mod.layer.calibrate(x, None, B)
        ctx.n_kept = len(kept)
        kept += [] if z is None else list(z) if save == "z8" else [z]
        ctx.save_for_backward(w, *kept)
        ctx.mod, ctx.mode, ctx.has_bias, ctx.has_res = mod, mode, b is not None, r is not None
        return y

    @staticmethod
    @ops.differentiated_once
    def backward(ctx, gy):
        w, *kept = ctx.saved_tensors
        mod, mode, n = ctx.mod, ctx.mode, ctx.n_kept
        gy = gy.contiguous()
        B = gy.shape[0]
        x, z = kept[:n], kept[n:]
        z = None if not z else z[0] if len(z) == 1 else ops.Checkpoint8(*z)
        need_gx, need_gw, need_gb, need_gr = ctx.needs_input_grad[:4]
        gz, gb = ops.activation_backward(gy, z, mod.activation, ctx.has_bias and need_gb)
        gx = gw = None
        if mode == "compress":
            gw = torch.empty_like(w)
            gx = torch.empty((B, mod.L, mod.Cx), dtype=gy.dtype, device=gy.device)
            mod.layer.backward(x[0], gz, w, B, gw, gx)
        else:
            gx, gw = ops.linear_backward(gz, w, x[0] if n == 1 else ops.Checkpoint8(*x), need_gx, need_gw)
            if mode in ("calibrate", "finalize"):
                mod._calibrate(x[0] if n == 1 else None, gz, B, finalize=(mode == "finalize"))
        return gx, gw, gb, gy if ctx.has_res and need_gr else None, None, None, None, None


class InstantLinear(torch.nn.Module):
    """y = act(x w^T + b) + r for x [B, L, Cx] -> y [B, L, Cy], weight [Cy, Cx], with the INSTANT
    backward on the steps between calibrations. By default there is neither bias (bias), nor
    activation (activation: relu, gelu, gelu_tanh, silu), nor residual (an argument of the call):
    y = x w^T.

    checkpoint="int8" keeps x and the pre-activation of the exact steps in 8 bits (one byte a
    value and one per 32 channels, ops.Checkpoint8): half the bf16 activations' memory, for a
    rounding of at most 1/127 of a group's largest value (x enters g_w, the pre-activation the
    activation's slope). A norm that writes its output in 8 bits (norm.InstantRMSNorm) hands
    that over as x8, and nothing is packed here. The low-rank steps keep x_hat as ever.

    weight: where the weight starts. A Parameter of the layer's type and device, contiguous, is taken
    as it is, so one that other layers hold too (an embedding's, say) is tied; anything else is copied.

    The library's backward passes cannot be differentiated again: with any of these options a
    backward pass with create_graph=True raises RuntimeError.

    dtype is the library's I/O dtype ("bf16" or "fp32"); inputs and the weight must have
    it. N_cal calibration steps start every window of N_t steps (N_cal <= N_t).

    comp is the energy compensation of the projections (关键设计 2). The default is the
    ratio reading, c = (E / sum_{i<=R} sigma_i^2)^(1/2) >= 1, which keeps the compressed
    steps' gradients on the scale of the exact ones. The factor as printed ("paper",
    c = (sum_{i<=R} sigma_i^2)^(-1/2)) carries the units of the data: g_w scales by c_P^2
    and g_x by c_Q^2 (about 5e-11 on BERT-sized synthetic data), so the compressed steps of a
    window would get gradients on a different scale from its exact calibration steps; it
    stays selectable. "none" (c = 1) gives the orthogonal projection.
    """

    def __init__(self, L, Cx, Cy, B_max, N_t=100, N_cal=16, p=2, eps=0.95, dtype="bf16", R_max=64,
                 comp="ratio", weight=None, device="cuda", bias=False, activation="none", checkpoint=None):
        super().__init__()
        if not 1 <= N_cal <= N_t:
            raise ValueError("need 1 <= N_cal <= N_t")
        if activation not in ops.ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(ops.ACTIVATIONS)}, got {activation!r}")
        if checkpoint not in (None, "int8"):
            raise ValueError(f"checkpoint must be None or 'int8', got {checkpoint!r}")
        self.L, self.Cx, self.Cy, self.B_max = int(L), int(Cx), int(Cy), int(B_max)
        self.N_t, self.N_cal = int(N_t), int(N_cal)
        self.torch_dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        if weight is None:
            self.weight = torch.nn.Parameter((torch.randn(Cy, Cx, device=device) / math.sqrt(Cx)).to(self.torch_dtype))
        else:
            self.weight = ops.weight_parameter(weight, device, self.torch_dtype)
        self.activation, self.checkpoint = activation, checkpoint
        self.bias = torch.nn.Parameter(torch.zeros(Cy, dtype=self.torch_dtype, device=device)) if bias else None
        self.layer = InstantLayer(make_config(L, Cx, Cy, B_max, R_max=R_max, p=p, N_t=N_t, eps=eps,
                                              dtype=dtype, comp=comp), device=device)
        self.step = 0          # training steps whose forward has run
        self.generation = 0    # successful finalizes so far
        self.Rx = self.Ry = 0
        self.last_status = INSTANT_OK

    def mode_of_step(self, step: int) -> str:
        t = step % self.N_t
        if t < self.N_cal:
            return "finalize" if t == self.N_cal - 1 else "calibrate"
        return "compress" if self.generation > 0 else "exact"

    def _calibrate(self, x, gy, B, finalize):
        s = self.layer.calibrate(x, gy, B, finalize=finalize)
        if finalize:
            self.last_status = s
            if s == INSTANT_OK:
                _, info = self.layer.query()
                self.generation += 1
                self.Rx, self.Ry = info.Rx, info.Ry

    def forward(self, x, residual=None, x8=None):
        if x.dim() != 3 or x.shape[1] != self.L or x.shape[2] != self.Cx or x.shape[0] > self.B_max:
            raise ValueError(f"x must be [B <= {self.B_max}, {self.L}, {self.Cx}], got {tuple(x.shape)}")
        if x.dtype != self.torch_dtype:
            raise TypeError(f"x must be {self.torch_dtype}")
        if x8 is not None:
            if not isinstance(x8, ops.Checkpoint8):
                raise TypeError(f"x8 must be a Checkpoint8, got {type(x8).__name__}")
            if self.checkpoint != "int8":
                raise ValueError("x8 is x in 8 bits, for a layer with checkpoint='int8'")
            ops.check_checkpoint(x8, x.shape, x.get_device(), "x8")
        x = x.contiguous()
        plain = self.bias is None and self.activation == "none" and self.checkpoint is None and residual is None
        if residual is not None:
            residual = residual.contiguous()
        if not (self.training and torch.is_grad_enabled()):
            if plain:
                return torch.nn.functional.linear(x, self.weight)
            if torch.is_grad_enabled():
                # evaluation with gradients: an exact step outside the schedule
                return _FusedLinearFn.apply(x, self.weight, self.bias, residual, *(x8 or (None, None)), self, "exact")
            return ops.linear_forward(x, self.weight, self.bias, residual, self.activation)[0]
        mode = self.mode_of_step(self.step)
        if plain:
            y = _InstantLinearFn.apply(x, self.weight, self, mode)
        else:
            y = _FusedLinearFn.apply(x, self.weight, self.bias, residual, *(x8 or (None, None)), self, mode)
        self.step += 1  # (a call that was refused is no step)
        return y

    def status(self) -> str:
        return instant_status_str(self.last_status)
