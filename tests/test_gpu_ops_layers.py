"""GPU tests of the layers built on the operators around the linear layer: InstantLinear with
bias, activation, residual and checkpoints in 8 bits through its calibration schedule, and
InstantRMSNorm before it."""
import numpy as np
import pytest

import oracle as O
import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _gelu(z):
    return 0.5 * z * (1 + torch.erf(z / 2 ** 0.5))


def _rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_schedule_with_epilogue_fp32(checkpoint):
    """Two windows of the tiny workload: forward, exact steps and low-rank steps against 64 bits.
    Exact steps: float32 sums over at most 128 terms and an erf, 1e-5; in 8 bits a group's rms
    rounding is at most max / 63.5 / 12^0.5 with max under 4 of the group's rms, 1.8e-2, once in x
    and once through the slope."""
    from rank_compressed_backprop_amd.linear import InstantLinear
    wl = W.get_workload("tiny")
    ly = wl.layer(0)
    B, L, N_t, N_cal, R_max = wl.B, wl.L, 5, 2, 32
    d0 = W.make_layer_batch(wl, 0, 0, with_w=True)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    mod = InstantLinear(L, ly.Cx, ly.Cy, B, N_t=N_t, N_cal=N_cal, p=wl.p, eps=wl.eps, dtype="fp32", R_max=R_max,
                        weight=dev(d0["w"]), bias=True, activation="gelu", checkpoint=checkpoint)
    g = torch.Generator().manual_seed(7)
    with torch.no_grad():
        mod.bias.copy_(torch.randn(ly.Cy, generator=g) * 0.1)
    w, b = mod.weight.detach().double(), mod.bias.detach().double()
    stats = {"x": [], "g": []}
    for s in range(2 * N_t):
        d = W.make_layer_batch(wl, 0, s)
        mode = mod.mode_of_step(s)
        print(f"[layer] step {s} {mode} checkpoint={checkpoint}", flush=True)
        x, r = dev(d["x"]).requires_grad_(True), torch.randn(B, L, ly.Cy, generator=g).cuda().requires_grad_(True)
        gy = dev(d["gy"])
        mod.weight.grad = mod.bias.grad = None
        y = mod(x, residual=r)
        y.backward(gy)
        x64 = x.detach().double()
        z64 = (x64 @ w.t() + b).requires_grad_(True)
        y64 = _gelu(z64)
        (gz64,) = torch.autograd.grad(y64, z64, gy.double())
        assert _rel(y.detach(), y64.detach() + r.detach().double()) <= 1e-6
        assert torch.equal(r.grad, gy)
        tol = 1e-5 if checkpoint is None or mode == "compress" else 0.03
        ztol = 1e-5 if checkpoint is None else 0.03
        assert _rel(mod.bias.grad, gz64.sum((0, 1))) <= ztol
        if mode == "compress":
            P = torch.empty((mod.Rx, L), device="cuda")
            Q = torch.empty((mod.Ry, L), device="cuda")
            mod.layer.get_projections(P, Q)
            P64, Q64 = P.cpu().numpy().astype(np.float64), Q.cpu().numpy().astype(np.float64)
            out = O.backward(P64, Q64, O.compress(P64, d["x64"]), gz64.cpu().numpy(), w.cpu().numpy())
            # (the existing path's own tolerance, and the slope's in 8 bits)
            assert _rel(mod.weight.grad, torch.from_numpy(out["gw"]).cuda()) <= max(1e-4, ztol if checkpoint else 0)
            assert _rel(x.grad, torch.from_numpy(out["gx"]).cuda()) <= max(1e-4, ztol if checkpoint else 0)
        else:
            flat = gz64.reshape(-1, ly.Cy)
            assert _rel(mod.weight.grad, flat.t() @ x64.reshape(-1, ly.Cx)) <= max(tol, ztol)
            assert _rel(x.grad, gz64 @ w) <= ztol
            if mode in ("calibrate", "finalize"):
                stats["x"].append(d["x64"])
                stats["g"].append(gz64.cpu().numpy())
        if mode == "finalize":
            assert mod.last_status == 0, mod.status()
            if checkpoint is None:  # (with z in 8 bits the statistics of g are of the rounded slope)
                cal = O.calibrate(stats["x"], stats["g"], wl.eps, wl.p, O.COMP_RATIO, R_max)
                assert (mod.Rx, mod.Ry) == (cal["x"]["R"], cal["g"]["R"])
            else:
                cal = O.calibrate(stats["x"], stats["x"], wl.eps, wl.p, O.COMP_RATIO, R_max)
                assert mod.Rx == cal["x"]["R"]
            stats = {"x": [], "g": []}
    mod.eval()
    x = dev(W.make_layer_batch(wl, 0, 99)["x"])
    with torch.no_grad():
        y = mod(x)
    y2 = mod(x)  # with gradients, outside the schedule
    assert mod.step == 2 * N_t and torch.equal(y, y2.detach())
    y2.sum().backward()
    assert _rel(y, _gelu(x.double() @ w.t() + b)) <= 1e-6


def test_norm_and_two_layers_bf16():
    """A pre-norm MLP block of the layers, x in 8 bits handed from the norm to the first layer,
    against autograd in 64 bits; the same without 8 bits. bf16: about ten roundings of 2^-9 rms
    lie between an input and a gradient, 6e-3; in 8 bits see above."""
    from rank_compressed_backprop_amd.linear import InstantLinear
    from rank_compressed_backprop_amd.norm import InstantRMSNorm
    B, L, C, H = 8, 49, 448, 1792
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).bfloat16().cuda()  # noqa: E731
    w1, w2 = rnd(H, C, sd=C ** -0.5), rnd(C, H, sd=H ** -0.5)
    xs = [rnd(B, L, C) for _ in range(2)]
    gout = rnd(B, L, C)
    for checkpoint in (None, "int8"):
        norm = InstantRMSNorm(C, eps=1e-5, checkpoint=checkpoint)
        up = InstantLinear(L, C, H, B, N_t=4, N_cal=2, weight=w1, bias=True, activation="gelu_tanh", checkpoint=checkpoint)
        down = InstantLinear(L, H, C, B, N_t=4, N_cal=2, weight=w2, bias=True, checkpoint=checkpoint)
        x, r = (t.clone().requires_grad_(True) for t in xs)
        y, h, *x8 = norm(x, r)
        out = down(up(y, x8=x8[0] if x8 else None), residual=h)
        out.backward(gout)
        x64, w1_, w2_, g_ = (t.double().requires_grad_(True) for t in (xs[0], w1, w2, norm.weight.detach()))
        h64 = x64 + xs[1].double()
        n = h64 * (h64.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * g_
        z = n @ w1_.t()
        a = 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
        o64 = a @ w2_.t() + h64
        ref = torch.autograd.grad(o64, (x64, w1_, w2_, g_), gout.double())
        tol = 0.01 if checkpoint is None else 0.03
        assert _rel(out.detach(), o64.detach()) <= 0.01
        for name, got, want in zip(("x", "w1", "w2", "g"), (x.grad, up.weight.grad, down.weight.grad, norm.weight.grad), ref):
            e = _rel(got, want)
            print(f"  checkpoint={checkpoint} {name}: {e:.2e}", flush=True)
            assert e <= tol, (checkpoint, name, e)
        assert torch.equal(x.grad, r.grad)


def test_norm_gradients_of_one_output():
    from rank_compressed_backprop_amd.norm import InstantRMSNorm
    norm = InstantRMSNorm(64, dtype="fp32")
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    r = torch.randn(3, 64, device="cuda", requires_grad=True)
    norm(x, r)[1].sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, x.grad)
    x.grad = None
    norm(x).square().sum().backward()
    x64 = x.detach().double().requires_grad_(True)
    (want,) = torch.autograd.grad((x64 * (x64.square().mean(1, keepdim=True) + 1e-6).rsqrt()).square().sum(), x64)
    # (the sum of squares hardly moves with x: compared on the scale of the terms that cancel)
    assert bool(((x.grad.double() - want).abs() <= 1e-5).all())


def test_wrong_layers_raise():
    from rank_compressed_backprop_amd import ops
    from rank_compressed_backprop_amd.linear import InstantLinear
    from rank_compressed_backprop_amd.norm import InstantRMSNorm
    with pytest.raises(ValueError):
        InstantLinear(8, 16, 16, 1, activation="tanh")
    with pytest.raises(ValueError):
        InstantLinear(8, 16, 16, 1, checkpoint="fp8")
    with pytest.raises(ValueError):
        InstantRMSNorm(64, checkpoint="int4")
    x = torch.zeros(1, 8, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        InstantLinear(8, 16, 16, 1, N_t=2, N_cal=1)(x, x8=ops.checkpoint_pack(x))
    with pytest.raises(ValueError):
        InstantLinear(8, 16, 16, 1, N_t=2, N_cal=1, checkpoint="int8")(x, x8=ops.checkpoint_pack(x[:, :4].contiguous()))
