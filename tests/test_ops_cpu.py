"""The operators around the linear layer (include/instant_ops.h), without a GPU: the boundary is
exported, and what a call may not be is refused on the host before anything is enqueued."""
import ctypes
import os
import random
import re
import types

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "instant_ops.h")

import rank_compressed_backprop_amd as rcb  # noqa: E402
from rank_compressed_backprop_amd import ops  # noqa: E402

A, W = 0x1000, 0x2000  # pointers that are never read: every call here is refused, or has no rows
E_ARG, E_SHAPE, OK = rcb.INSTANT_E_ARG, rcb.INSTANT_E_SHAPE, rcb.INSTANT_OK
BF, FP = rcb.INSTANT_BF16, rcb.INSTANT_FP32


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(instant_[a-z_]+)\s*\(", text))


def test_boundary_is_exported():
    assert declared() == set(ops.EXPORTED)
    lib = ctypes.CDLL(rcb.LIB_PATH)
    for name in declared():
        assert hasattr(lib, name), name


def test_workspace_sizes():
    for bad in [(-1, 8, 8, BF), (4, 0, 8, BF), (4, 8, -8, BF), (4, 12, 8, BF), (4, 8, 20, BF), (4, 8, 8, 2),
                (1 + (1 << 26), 8, 8, BF), (4, 8 + (1 << 18), 8, BF)]:
        assert ops.instant_linear_workspace_bytes(*bad) == 0, bad
    for bad in [(-1, 8), (4, 0), (4, 12), (4, 65544)]:
        assert ops.instant_rmsnorm_workspace_bytes(*bad) == 0, bad
    for M in (0, 1, 7, 1 << 20, 1 << 26):
        for dt in (BF, FP):
            n = ops.instant_linear_workspace_bytes(M, 4096, 1024, dt)
            assert n >= 256 and n % 256 == 0
            assert n < 1 << 31  # the partial sums' size does not grow with the batch
            alone = [ops.instant_linear_fwd_workspace_bytes(M, 4096, 1024, dt),
                     ops.instant_linear_bwd_workspace_bytes(M, 4096, 1024, dt, True),
                     ops.instant_linear_bwd_workspace_bytes(M, 4096, 1024, dt, False),
                     ops.instant_act_bwd_workspace_bytes(M, 4096, dt)]
            assert max(alone) <= n
        n = ops.instant_rmsnorm_workspace_bytes(M, 65536)
        assert n >= 256 and n % 256 == 0


def fwd(x=A, w=A, bias=None, res=None, M=4, N=64, K=64, dtype=BF, act=0, y=A, z=None, zq=None, zs=None, ws=W,
        n=1 << 30):
    return ops.instant_linear_fwd(x, w, bias, res, M, N, K, dtype, act, y, z, zq, zs, ws, n, 0)


def test_linear_fwd_refusals():
    for change in [dict(x=None), dict(w=None), dict(y=None), dict(x=A + 8), dict(w=A + 2), dict(bias=A + 4),
                   dict(res=A + 8), dict(y=A + 8), dict(z=A + 8), dict(zq=A + 8, zs=A), dict(zq=A), dict(zs=A),
                   dict(z=A, zq=A, zs=A), dict(M=-1), dict(N=0), dict(K=-8), dict(dtype=2), dict(act=5),
                   dict(act=-1)]:
        assert fwd(**change) == E_ARG, change
    for change in [dict(N=60), dict(K=68)]:
        assert fwd(**change) == E_SHAPE, change
    assert fwd(M=0, x=None, w=None, y=None, ws=None, n=0) == OK
    # a workspace that the sizes need: absent, misaligned, too small
    big = dict(M=8, N=64, K=8192)
    assert ops.instant_linear_workspace_bytes(8, 64, 8192, FP) > 256
    assert fwd(**big, dtype=FP, ws=None) == E_ARG
    assert fwd(**big, dtype=FP, ws=W + 128) == E_ARG
    assert fwd(**big, dtype=FP, n=64) == E_SHAPE


def act_bwd(gy=A, z=A, zq=None, zs=None, M=4, N=64, dtype=BF, act=2, gz=A, gb=None, ws=W, n=1 << 30):
    return ops.instant_act_bwd(gy, z, zq, zs, M, N, dtype, act, gz, gb, ws, n, 0)


def test_act_bwd_refusals():
    for change in [dict(gy=None), dict(z=None), dict(z=A, zq=A, zs=A), dict(z=None, zq=A), dict(z=None, zs=A),
                   dict(gz=None), dict(act=0), dict(act=0, z=None, zq=A, zs=A), dict(gy=A + 8), dict(z=A + 8),
                   dict(gz=A + 8), dict(gb=A + 8), dict(M=-1), dict(N=0), dict(dtype=7), dict(act=9),
                   dict(gb=A, ws=None, M=1000), dict(gb=A, ws=W + 8, M=1000)]:
        assert act_bwd(**change) == E_ARG, change
    assert act_bwd(N=12) == E_SHAPE
    assert act_bwd(gb=A, M=1000, n=16) == E_SHAPE
    assert act_bwd(M=0, gy=None, z=None) == OK


def bwd(gz=A, w=A, x=A, xq=None, xs=None, M=4, N=64, K=64, dtype=BF, gx=A, gw=A, ws=W, n=1 << 30):
    return ops.instant_linear_bwd(gz, w, x, xq, xs, M, N, K, dtype, gx, gw, ws, n, 0)


def test_linear_bwd_refusals():
    for change in [dict(gz=None), dict(w=None), dict(x=None), dict(xq=A, xs=A), dict(x=None, xq=A),
                   dict(x=None, xs=A), dict(gx=None, gw=None), dict(gz=A + 8), dict(w=A + 8), dict(x=A + 8),
                   dict(gx=A + 8), dict(gw=A + 8), dict(x=None, xq=A + 8, xs=A), dict(M=-2), dict(N=0), dict(K=0),
                   dict(dtype=-1)]:
        assert bwd(**change) == E_ARG, change
    for change in [dict(N=4), dict(K=100)]:
        assert bwd(**change) == E_SHAPE, change
    assert bwd(M=0, gz=None, w=None, x=None, gw=None, ws=None, n=0) == OK  # no rows: gx has none
    big = dict(M=8192, N=8, K=8)
    assert bwd(**big, dtype=FP, ws=None) == E_ARG
    assert bwd(**big, dtype=FP, n=0) == E_SHAPE


def test_ckpt_refusals():
    for change in [dict(x=None), dict(q=None), dict(s=None), dict(x=A + 8), dict(q=A + 8), dict(M=-1), dict(C=0),
                   dict(dtype=5)]:
        a = dict(x=A, M=4, C=64, dtype=BF, q=A, s=A) | change
        assert ops.instant_ckpt_pack(a["x"], a["M"], a["C"], a["dtype"], a["q"], a["s"], 0) == E_ARG, change
        assert ops.instant_ckpt_unpack(a["q"], a["s"], a["M"], a["C"], a["dtype"], a["x"], 0) == E_ARG, change
    assert ops.instant_ckpt_pack(A, 4, 36, BF, A, A, 0) == E_SHAPE
    assert ops.instant_ckpt_unpack(A, A, 4, 36, BF, A, 0) == E_SHAPE
    assert ops.instant_ckpt_pack(None, 0, 64, BF, None, None, 0) == OK
    assert ops.instant_ckpt_unpack(None, None, 0, 64, BF, None, 0) == OK


def test_rmsnorm_refusals():
    def nf(x=A, res=None, g=A, M=4, C=64, dtype=BF, eps=1e-5, h=None, y=A, yq=None, ys=None, rstd=A):
        return ops.instant_rmsnorm_fwd(x, res, g, M, C, dtype, eps, h, y, yq, ys, rstd, 0)
    for change in [dict(x=None), dict(g=None), dict(res=A), dict(h=A), dict(y=None), dict(yq=A), dict(ys=A),
                   dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=A + 8), dict(g=A + 8),
                   dict(y=A + 8), dict(rstd=A + 2), dict(M=-1), dict(C=0), dict(dtype=3), dict(res=A + 8, h=A)]:
        assert nf(**change) == E_ARG, change
    assert nf(C=20) == E_SHAPE and nf(C=65544) == E_SHAPE
    assert nf(M=0) == OK

    def nb(gy=A, h=A, g=A, rstd=A, gh=None, M=4, C=64, dtype=BF, gx=A, gg=A, ws=W, n=1 << 30):
        return ops.instant_rmsnorm_bwd(gy, h, g, rstd, gh, M, C, dtype, gx, gg, ws, n, 0)
    for change in [dict(gy=None), dict(h=None), dict(g=None), dict(rstd=None), dict(gx=None), dict(gy=A + 8),
                   dict(h=A + 8), dict(gh=A + 8), dict(gx=A + 8), dict(gg=A + 8), dict(rstd=A + 1), dict(M=-1),
                   dict(C=0), dict(dtype=3), dict(ws=None), dict(ws=W + 16)]:
        assert nb(**change) == E_ARG, change
    assert nb(C=20) == E_SHAPE and nb(C=65544) == E_SHAPE and nb(n=8) == E_SHAPE
    assert nb(M=0, gg=None) == OK


def test_tensor_functions_refuse_cpu_tensors_and_bad_shapes():
    """Shapes and types are checked before the device, so no GPU is asked."""
    x = torch.zeros(4, 12)
    with pytest.raises(TypeError):
        ops.checkpoint_pack(torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError):
        ops.checkpoint_pack(torch.tensor(1.0))
    with pytest.raises(ValueError):
        ops.checkpoint_pack(torch.zeros(16, 4).t())
    for call in (lambda: ops.checkpoint_pack(x), lambda: ops.linear_forward(x, x),
                 lambda: ops.rmsnorm_forward(x, x[0]), lambda: ops.activation_backward(x, x),
                 lambda: ops.checkpoint_pack(torch.zeros(4, 16))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ops.checkpoint_unpack(ops.Checkpoint8(x, x), torch.float16)


def test_one_workspace_serves_every_call():
    """What instant_linear_workspace_bytes returns is enough for each of the three calls, whichever
    way x is given: a checkpoint is split by chunks of rows, x in full by all of them, so either may
    need more."""
    rng = random.Random(5)
    sizes = [(19142, 3504, 10672, BF), (6613, 3984, 10496, FP), (368011, 456, 18920, BF), (368011, 456, 18920, FP)]
    for _ in range(4000):
        M = int(2 ** rng.uniform(0, 26))
        sizes.append((M, 8 * int(2 ** rng.uniform(0, 12)), 8 * int(2 ** rng.uniform(0, 12)), rng.choice([BF, FP])))
    for s in sizes:
        alone = [ops.instant_linear_fwd_workspace_bytes(*s), ops.instant_act_bwd_workspace_bytes(s[0], s[1], s[3]),
                 *(ops.instant_linear_bwd_workspace_bytes(*s, ckpt) for ckpt in (False, True))]
        assert max(alone) <= ops.instant_linear_workspace_bytes(*s), (s, alone)


def test_layers_refuse_second_derivatives(monkeypatch):
    """The backward passes are launches without a graph: a second derivative would be short of
    their terms, so it is refused. Plain forms stand in for the kernels here."""
    from rank_compressed_backprop_amd.linear import _FusedLinearFn
    from rank_compressed_backprop_amd.norm import _RMSNormFn
    raw = torch.no_grad()
    monkeypatch.setattr(ops, "linear_forward", raw(lambda x, w, b, r, act, save: (
        torch.relu(x @ w.t() + b) + r, x @ w.t() + b)))
    monkeypatch.setattr(ops, "activation_backward", raw(lambda gy, z, act, bias_grad: (
        gy * (z > 0), (gy * (z > 0)).sum((0, 1)))))
    monkeypatch.setattr(ops, "linear_backward", raw(lambda gz, w, x, need_gx, need_gw: (
        gz @ w, gz.flatten(0, 1).t() @ x.flatten(0, 1))))
    monkeypatch.setattr(ops, "rmsnorm_forward", raw(lambda x, w, r, eps, y8: ops.NormOut(
        (x + r) * w, x + r, torch.ones(x.shape[:-1]), None)))
    monkeypatch.setattr(ops, "rmsnorm_backward", raw(lambda gy, h, w, rstd, gh, need: (gy * w, (gy * h).sum((0, 1)))))
    g = torch.Generator().manual_seed(3)
    x, r, b, n, w = (torch.randn(*s, generator=g).requires_grad_(True)
                     for s in ((2, 3, 8), (2, 3, 8), (8,), (8,), (8, 8)))
    layer = types.SimpleNamespace(checkpoint=None, activation="relu")
    for leaves, call in [((x, w, b, r), lambda: _FusedLinearFn.apply(x, w, b, r, None, None, layer, "exact")),
                         ((x, n, r), lambda: _RMSNormFn.apply(x, r, n, 1e-6, False)[0])]:
        torch.autograd.grad(call().square().sum(), leaves)  # once is what they are for
        for loss in (call().square().sum(), call().sum()):  # the incoming gradient with and without a graph
            with pytest.raises(RuntimeError, match="differentiated again"):
                torch.autograd.grad(loss, leaves, create_graph=True)


def test_linear_backward_asks_for_the_workspace_of_its_gradients(monkeypatch):
    """Only the gradients that are asked for take workspace: without the weight's, the values of a
    checkpoint are not unpacked and need no room. (What a call passes is enough, and a byte less is
    not: the library refuses it.)"""
    calls = []

    def record(gz, w, x, xq, xs, M, N, K, dt, gx, gw, ws, n, stream):
        calls.append((gx is not None, gw is not None, xq is not None, n))
        assert (ws is None) == (n == 0)
        return OK
    sizes, real = [(8192, 16, 8), (512, 256, 1024), (2048, 64, 4096), (4, 4096, 64)], ops._lib

    class Lib:
        instant_linear_bwd = staticmethod(record)

        def __getattr__(self, name):
            return getattr(real, name)
    monkeypatch.setattr(ops, "_lib", Lib())
    monkeypatch.setattr(ops, "_on_device", lambda t, name: None)
    monkeypatch.setattr(ops, "_current", lambda dev: None)
    for M, N, K in sizes:
        for dtype, code in ((torch.bfloat16, BF), (torch.float32, FP)):
            gz, w, x = (torch.zeros(s, dtype=dtype) for s in ((M, N), (N, K), (M, K)))
            x8 = ops.Checkpoint8(torch.zeros(M, K, dtype=torch.int8), torch.zeros(M, -(-K // 32), dtype=torch.uint8))
            for xx in (x, x8):
                for gx, gw in ((True, True), (True, False), (False, True)):
                    del calls[:]
                    ops.linear_backward(gz, w, xx, gx, gw)
                    ((has_gx, has_gw, ckpt, n),) = calls
                    assert (has_gx, has_gw) == (gx, gw)
                    need = [ops.instant_linear_gx_workspace_bytes(M, N, K, code)] if gx else []
                    need += [ops.instant_linear_gw_workspace_bytes(M, N, K, code, ckpt)] if gw else []
                    assert n == max(need)
                    assert n <= ops.instant_linear_bwd_workspace_bytes(M, N, K, code, ckpt)
                    if n:  # (a workspace a byte smaller is refused before anything is enqueued)
                        xs = (None, A, A) if ckpt else (A, None, None)
                        a = (A, A, *xs, M, N, K, code, A if gx else None, A if gw else None, W, n - 1, None)
                        assert real.instant_linear_bwd(*a) == E_SHAPE, (M, N, K, dtype, ckpt, gx, gw, n)


def test_missing_and_foreign_arguments(monkeypatch):
    """What is needed and not given, and what is neither a tensor nor a checkpoint, is named."""
    monkeypatch.setattr(ops, "_on_device", lambda t, name: None)
    gz, w, x = torch.zeros(4, 16), torch.zeros(16, 8), torch.zeros(4, 8)
    c = (torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8))  # a pair, no Checkpoint8
    for exc, name, call in [(ValueError, "x", lambda: ops.linear_backward(gz, w, None)),
                            (TypeError, "x", lambda: ops.linear_backward(gz, w, c)),
                            (TypeError, "z", lambda: ops.activation_backward(gz, c, "relu")),
                            (TypeError, "bias", lambda: ops.linear_forward(x, w, bias=1.0)),
                            (TypeError, "w", lambda: ops.linear_forward(x, None)),
                            (TypeError, "w", lambda: ops.linear_backward(gz, None, x)),
                            (TypeError, "x", lambda: ops.checkpoint_pack(None)),
                            (TypeError, "h", lambda: ops.rmsnorm_backward(x, None, w[0], x[:, 0])),
                            (TypeError, "checkpoint", lambda: ops.checkpoint_unpack(c))]:
        with pytest.raises(exc, match=f"^(a )?{name} "):
            call()


def test_norm_layer_refuses_other_types():
    from rank_compressed_backprop_amd.norm import InstantRMSNorm
    for dtype in ("float16", "bfloat16", torch.bfloat16, None):
        with pytest.raises(ValueError, match="dtype"):
            InstantRMSNorm(64, dtype=dtype, device="cpu")
    assert InstantRMSNorm(64, device="cpu").weight.dtype == torch.bfloat16
    assert InstantRMSNorm(64, dtype="fp32", device="cpu").weight.dtype == torch.float32
    for C in (0, 12, -8):
        with pytest.raises(ValueError, match="C must"):
            InstantRMSNorm(C, device="cpu")
