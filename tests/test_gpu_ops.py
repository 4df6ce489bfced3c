"""GPU tests of the operators around the linear layer (include/instant_ops.h) against plain
64-bit implementations.

Tolerances. u is half a step of the I/O type relative to the value (bf16 2^-8, fp32 2^-24): what
one rounding is off by at most. A float32 sum of n terms, in any order, is off by at most
n 2^-24 times the sum of the terms' magnitudes; GAMMA(n) = 2 (n + 8) 2^-24 leaves a factor of two
for the matrix cores' own additions. An activation or its slope is evaluated to 2^-19 of
max(1, |z|) (hardware exponential and reciprocal, 1 ulp = 2^-23 each, on arguments whose own
rounding enters at most 16-fold), and no activation's slope exceeds 1.13 (its slope's slope 1.2).
"""
import zlib

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
BF, FP = torch.bfloat16, torch.float32


def GAMMA(n):
    return 2.0 * (n + 8) * 2.0 ** -24


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def randn(g, *shape, dtype=FP, sd=1.0):
    return (torch.randn(*shape, generator=g) * sd).to(dtype).cuda()


def act64(z, name):
    z = z.double()
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / 2 ** 0.5)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, name):
    if name == "relu":
        return (z > 0).double()
    z = z.double().detach().requires_grad_(True)
    (s,) = torch.autograd.grad(act64(z, name).sum() + 0 * z.sum(), z)
    return s


def two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def pack64(x):
    """(q, scale) by the definition, for finite x."""
    t = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 32)).unflatten(1, (-1, 32))
    amax = t.abs().amax(2)
    b = torch.ones_like(amax, dtype=torch.int64)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):  # the largest byte that is still too small, plus one
        up = b + step
        b = torch.where((up <= 254) & (amax > 127 * two_to(torch.clamp(up, max=254) - 128)), up, b)
    q = torch.round(t / two_to(b - 127).unsqueeze(2)).flatten(1)[:, :x.shape[1]]
    return q.to(torch.int8), b.to(torch.uint8)


def value64(c):
    s = torch.where(c.scale == 255, torch.nan, two_to(c.scale.to(torch.int64) - 127))
    return c.q.double() * s.repeat_interleave(32, -1)[..., :c.q.shape[-1]]


def within(name, got, ref, bound):
    d = (got.double() - ref).abs()
    worst = (d - bound).max().item() if d.numel() else 0.0
    ratio = (d / bound.clamp(min=1e-300)).max().item() if d.numel() else 0.0
    print(f"  {name}: worst error / bound {ratio:.3f}", flush=True)
    assert worst <= 0 and not torch.isnan(d).any(), f"{name}: {ratio} of the bound"


def bits(t):
    return t.view(torch.int16 if t.dtype == BF else torch.int32) if t.dtype in (BF, FP) else t


# ------------------------------------------------------------------------- checkpoints

CKPT_SHAPES = [(1, 8), (1, 32), (3, 40), (5, 24), (64, 768), (7, 1000), (129, 4096), (2, 8200)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", CKPT_SHAPES, ids=str)
def test_checkpoint(shape, dtype):
    from rank_compressed_backprop_amd import ops
    print(f"[ckpt] {shape} {dtype}", flush=True)
    g = gen("ckpt", shape, str(dtype))
    x = (torch.randn(*shape, generator=g) * torch.exp(4 * torch.randn(shape[0], 1, generator=g))).to(dtype).cuda()
    c = ops.checkpoint_pack(x)
    q, s = pack64(x)
    assert torch.equal(c.scale, s) and torch.equal(c.q, q)
    assert int(c.q.abs().max()) <= 127
    for out in (BF, FP):
        assert torch.equal(ops.checkpoint_unpack(c, out).double(), value64(c))
    # at most half a step, and a step is at most max / 63.5
    top = torch.nn.functional.pad(x.double(), (0, -shape[1] % 32)).unflatten(1, (-1, 32)).abs().amax(2)
    assert bool(((value64(c) - x.double()).abs() <= (top / 127).repeat_interleave(32, 1)[:, :shape[1]]).all())


def test_checkpoint_edges():
    """Borders of the scale, zeros, subnormals, the largest numbers, infinities and NaN."""
    from rank_compressed_backprop_amd import ops
    rows = [[127.0, 1.5, 2.5, -0.5], [127.5, 1.0], [-127.0, 126.5], [128.0, 3.0, 5.0], [0.0], [1e-40, -3e-42],
            [2.0 ** -126, 2.0 ** -127], [3.3e38, -1e38], [2.0 ** -120, 1e-38]]
    x = torch.zeros(len(rows), 64)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r)
        x[i, 40] = 1.0  # the second group of the row goes its own way
    c = ops.checkpoint_pack(x.cuda())
    q, s = pack64(x.cuda())
    assert torch.equal(c.scale, s) and torch.equal(c.q, q)
    for bad in (float("inf"), -float("inf"), float("nan")):
        x = torch.ones(3, 72)
        x[1, 33] = bad
        for dtype in (BF, FP):
            v = ops.checkpoint_unpack(ops.checkpoint_pack(x.to(dtype).cuda()), dtype)
            want = torch.zeros(3, 72, dtype=torch.bool)
            want[1, 32:64] = True  # its group, and nothing else
            assert torch.equal(torch.isnan(v).cpu(), want)
            assert torch.equal(v[~want.cuda()], torch.ones_like(v[~want.cuda()]))


def test_checkpoint_ends_of_the_range():
    """Finite values stay finite: 127 steps of 2^121 are the largest that a checkpoint stands for,
    and what lies above is off by at most a step. The smallest step is 2^-126."""
    from rank_compressed_backprop_amd import ops
    top = 127 * 2.0 ** 121
    for dtype in (BF, FP):
        most = torch.finfo(dtype).max
        rows = [[most, -most, top, -top, 1e38, 2.0 ** 121, 2.0 ** 120, 1.5 * 2.0 ** 121],
                [-most] * 8, [most] + [0.0] * 7, [top, 126.5 * 2.0 ** 121, -125.5 * 2.0 ** 121, 1.0],
                [2.0 ** -126, 2.0 ** -127, -2.0 ** -127, 2.0 ** -128, 1.5 * 2.0 ** -126, 63 * 2.0 ** -126]]
        x = torch.zeros(len(rows), 72, dtype=torch.float64)
        for i, r in enumerate(rows):
            x[i, 32:32 + len(r)] = torch.tensor(r, dtype=torch.float64)
        x = x.to(dtype).cuda()
        w = torch.eye(72, dtype=dtype, device="cuda")
        packed = ops.checkpoint_pack(x)
        # the product with 1 gives the same values, and so the same checkpoint
        _, kept = ops.linear_forward(x, w, save="z8")
        assert torch.equal(packed.q[:4], kept.q[:4]) and torch.equal(packed.scale[:4], kept.scale[:4])
        assert packed.scale[:, 1].tolist() == [248, 248, 248, 248, 1]
        v = ops.checkpoint_unpack(packed, dtype).double()
        assert bool(torch.isfinite(v).all())
        assert torch.equal(v, value64(packed))
        x64 = x.double()
        assert torch.equal(v[:4].abs() == top, x64[:4].abs() > 126.5 * 2.0 ** 121)
        step = torch.where(x64.abs() > top, 2.0 ** 121, 2.0 ** 120)
        step[4] = 2.0 ** -127
        assert bool(((v - x64).abs() <= step).all())
        assert bool(((v - x64)[:4].abs() <= x64[:4].abs().amax(1, keepdim=True) / 127).all())


# ------------------------------------------------------------------------- linear, forward

def check_forward(ops, M, N, K, dtype, act, bias, res, save, key=0):
    print(f"[linear] M={M} N={N} K={K} {dtype} {act} bias={bias} res={res} save={save}", flush=True)
    g = gen("fwd", M, N, K, str(dtype), act, key)
    x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype, sd=K ** -0.5)
    b = randn(g, N, dtype=dtype) if bias else None
    r = randn(g, M, N, dtype=dtype) if res else None
    y, z = ops.linear_forward(x, w, b, r, act, save)
    z64 = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if bias:
        z64, mag = z64 + b.double(), mag + b.double().abs()
    ez = GAMMA(K) * mag
    y64 = act64(z64, act)
    ey = 1.13 * ez + (0 if act in ("none", "relu") else 2.0 ** -19 * z64.abs().clamp(min=1))
    if res:
        y64 = y64 + r.double()
    ey = ey + 2.0 ** -23 * (y64.abs() + (r.double().abs() if res else 0))
    u = U[dtype]
    within("y", y, y64, u * y64.abs() + (1 + u) * ey + 1e-38)
    if save == "z":
        within("z", z, z64, u * z64.abs() + (1 + u) * ez + 1e-38)
    elif save == "z8":
        # a value near a border may fall on either side: half a step, of the larger of the two
        # scales that the group's largest may round to
        top = torch.nn.functional.pad(z64.abs() + ez, (0, -N % 32)).unflatten(1, (-1, 32)).amax(2)
        _, s = pack64(top.repeat_interleave(32, 1))
        step = two_to(s.to(torch.int64) - 127).repeat_interleave(32, 1)[:, :N]
        within("z8", value64(z), z64, step / 2 + ez)
    else:
        assert z is None


FWD_SHAPES = [(1, 8, 8), (1, 768, 768), (2, 1000, 40), (3, 72, 4096), (8, 11008, 512), (16, 136, 2056), (17, 64, 72),
              (33, 264, 1032), (49, 448, 448), (64, 64, 64), (65, 8, 1024), (127, 256, 96), (128, 128, 64),
              (129, 136, 520), (257, 520, 264), (300, 1792, 448), (1000, 72, 8), (4100, 776, 200)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("i", range(len(FWD_SHAPES)), ids=lambda i: "x".join(map(str, FWD_SHAPES[i])))
def test_linear_forward(i, dtype):
    from rank_compressed_backprop_amd import ops
    M, N, K = FWD_SHAPES[i]
    # every shape with its own mix of options, and each with its opposite
    check_forward(ops, M, N, K, dtype, ACTS[i % 5], bool(i % 2), bool(i % 3), ("none", "z", "z8")[i % 3])
    check_forward(ops, M, N, K, dtype, ACTS[(i + 2) % 5], not i % 2, not i % 3, ("z8", "none", "z")[i % 3])


@pytest.mark.parametrize("act", ACTS)
def test_linear_forward_every_option(act):
    from rank_compressed_backprop_amd import ops
    for n, (bias, res, save) in enumerate([(a, b, c) for a in (0, 1) for b in (0, 1) for c in ("none", "z", "z8")]):
        check_forward(ops, (5, 70, 200)[n % 3], 104, 96, BF, act, bias, res, save, n)


@pytest.mark.parametrize("shape", [(16384, 768, 768), (2048, 11008, 4096), (4096, 4096, 11008), (6272, 1792, 448)],
                         ids=str)
def test_linear_forward_workload_sizes(shape):
    from rank_compressed_backprop_amd import ops
    M, N, K = shape
    check_forward(ops, M, N, K, BF, "gelu", True, True, "z8")


# Sizes that reach every tile shape and ring depth of every product, with the contraction whole and
# split, with edges inside a tile: (rows, columns, contraction) of the output.
EVERY_TILE = {
    ("fwd", BF): [(1, 8, 1168), (1, 8, 80), (2897, 8, 1952), (1, 8, 8), (486, 368, 2480), (471, 1096, 352),
                  (422, 2832, 5256), (747, 1360, 1032), (1643, 584, 1768), (10175, 280, 8), (2736, 424, 3320),
                  (1518, 1416, 1720), (3762, 1344, 5384), (19654, 544, 232), (1656, 7912, 616)],
    ("gx", BF): [(1, 8, 1328), (1, 8, 72), (9018, 8, 2480), (1, 8, 8), (459, 360, 2416), (1382, 328, 280),
                 (186, 2768, 3736), (1398, 864, 960), (1126, 920, 2136), (1063, 1968, 208), (985, 1312, 2928),
                 (3748, 560, 1464), (7152, 576, 3680), (1711, 4728, 896), (3629, 1040, 4976), (5338, 2360, 680)],
    ("gw", BF): [(8, 8, 1110), (8, 8, 67), (5824, 8, 3326), (8, 8, 1), (680, 200, 2230), (1720, 264, 257),
                 (424, 1464, 3985), (1392, 744, 925), (848, 1408, 2125), (5464, 528, 6), (776, 1608, 2933),
                 (1560, 1448, 1470), (1232, 2192, 8012), (3632, 2248, 758), (6456, 656, 4537), (6128, 2144, 641)],
    ("fwd", FP): [(3, 8, 296), (1, 8, 8), (450, 344, 1104), (9399, 8, 8), (1700, 1520, 2304), (910, 3280, 8),
                  (1702, 7384, 32)],
    ("gx", FP): [(1, 8, 312), (1, 8, 8), (774, 152, 1280), (9355, 8, 8), (736, 3208, 2112), (3466, 856, 8),
                 (4128, 1224, 3144), (14689, 872, 16)],
    ("gw", FP): [(8, 8, 295), (8, 8, 1), (504, 376, 895), (8480, 16, 1), (728, 3288, 3420), (8696, 336, 1),
                 (6432, 728, 5541), (7808, 1568, 1)],
}


@pytest.mark.parametrize("which", EVERY_TILE, ids=lambda w: f"{w[0]}-{'bf16' if w[1] == BF else 'fp32'}")
def test_every_tile(which):
    from rank_compressed_backprop_amd import ops
    kind, dtype = which
    for i, (a, b, k) in enumerate(EVERY_TILE[which]):
        print(f"[tile] {kind} {dtype} {a} x {b} over {k}", flush=True)
        if kind == "fwd":
            for act, save in (("none", "none"), ("silu", "z8"), ("relu", "z")):
                check_forward(ops, a, b, k, dtype, act, bool(i % 2), bool(i % 3), save)
            continue
        g = gen("tile", which[0], str(dtype), a, b, k)
        M, N, K = (a, k, b) if kind == "gx" else (k, a, b)
        gz, w = randn(g, M, N, dtype=dtype), randn(g, N, K, dtype=dtype)
        d, u = gz.double(), U[dtype]
        if kind == "gx":
            gx, _ = ops.linear_backward(gz, w, None, need_gw=False)
            ref, mag = d @ w.double(), d.abs() @ w.double().abs()
            within("gx", gx, ref, u * ref.abs() + (1 + u) * GAMMA(N) * mag + 1e-38)
        else:
            x = randn(g, M, K, dtype=dtype)
            d = d.t().contiguous()
            for xx, x64 in ((x, x.double()), (ops.checkpoint_pack(x), None)):
                x64 = value64(xx) if x64 is None else x64
                _, gw = ops.linear_backward(gz, w, xx, need_gx=False)
                ref, mag = d @ x64, d.abs() @ x64.abs()
                within("gw", gw, ref, u * ref.abs() + (1 + u) * GAMMA(M) * mag + 1e-38)


# The largest tile with the contraction split, which the forward's lists above do not reach.
LARGEST_SPLIT = {BF: [(3629, 1040, 4976)], FP: [(4128, 1224, 3144)]}


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_linear_forward_largest_tile_split(dtype):
    from rank_compressed_backprop_amd import ops
    for a, b, k in LARGEST_SPLIT[dtype]:
        check_forward(ops, a, b, k, dtype, "none", True, True, "z")
        check_forward(ops, a, b, k, dtype, "none", False, False, "none")


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_residual_in_place_in_every_tile(dtype):
    """The residual may be the output itself: the same bits as beside it, in every tile."""
    import rank_compressed_backprop_amd as rcb
    from rank_compressed_backprop_amd import ops
    code = rcb.INSTANT_BF16 if dtype == BF else rcb.INSTANT_FP32
    for M, N, K in EVERY_TILE["fwd", dtype] + LARGEST_SPLIT[dtype]:
        g = gen("in place", M, N, K)
        x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype, sd=K ** -0.5)
        b, r = randn(g, N, dtype=dtype), randn(g, M, N, dtype=dtype)
        n = ops.instant_linear_fwd_workspace_bytes(M, N, K, code)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        for act in ("none", "silu"):  # (two choices of tiles)
            print(f"[in place] {M} {N} {K} {dtype} {act}", flush=True)
            want, _ = ops.linear_forward(x, w, b, r, act)
            y = r.clone()
            assert ops.instant_linear_fwd(x, w, b, y, M, N, K, code, ops.ACTIVATIONS[act], y, None, None, None, ws, n) == 0
            assert torch.equal(bits(y), bits(want))


def test_linear_forward_nonfinite_stays():
    """An infinity or NaN in one row reaches that row's outputs, and no other row's."""
    from rank_compressed_backprop_amd import ops
    for M, N, K in [(3, 72, 64), (200, 264, 320)]:
        for dtype in (BF, FP):
            for act in ACTS:
                g = gen("inf", M, act)
                x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype)
                clean, _ = ops.linear_forward(x, w, activation=act)
                x[1, 5] = float("nan")
                y, z = ops.linear_forward(x, w, activation=act, save="z8")
                assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(value64(z)[1]).all())
                keep = torch.arange(M) != 1
                assert torch.equal(bits(y[keep]), bits(clean[keep]))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_forward_extreme_values(act, dtype):
    """Infinities, NaN and numbers near the type's end in one row of x, of the residual and of the
    bias: infinite and NaN outputs where the definition in 64 bits has them (an infinity below zero
    times a vanished factor is NaN there too), right values elsewhere, other rows as ever."""
    from rank_compressed_backprop_amd import ops
    u = U[dtype]
    for M, N, K in [(3, 72, 64), (200, 264, 320)]:
        g = gen("extreme", M, act)
        x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype)
        b, r = randn(g, N, dtype=dtype), randn(g, M, N, dtype=dtype)
        clean, _ = ops.linear_forward(x, w, b, r, act)
        keep = torch.arange(M) != 1
        for value in (float("nan"), float("inf"), -float("inf"), 3e19, -3e19, 2e37, -2e37):
            for place in ("x", "r", "b"):
                print(f"[extreme] {M} {N} {K} {dtype} {act} {value} in {place}", flush=True)
                t = {"x": x.clone(), "r": r.clone(), "b": b.clone()}
                if place == "b":
                    t["b"][N - 3] = value
                else:
                    t[place][1, 5] = value  # (x: a term of every column's sum)
                y, z = ops.linear_forward(t["x"], w, t["b"], t["r"], act, save="z")
                z64 = t["x"].double() @ w.double().t() + t["b"].double()
                y64 = act64(z64, act) + t["r"].double()
                for got, ref in ((z, z64), (y, y64)):
                    assert torch.equal(torch.isnan(got), torch.isnan(ref))
                    assert torch.equal(torch.isposinf(got), torch.isposinf(ref))
                    assert torch.equal(torch.isneginf(got), torch.isneginf(ref))
                mag = t["x"].double().abs() @ w.double().abs().t() + t["b"].double().abs()
                ez = GAMMA(K) * mag
                ey = 1.13 * ez + 2.0 ** -19 * z64.abs().clamp(min=1) + 2.0 ** -23 * (y64.abs() + t["r"].double().abs())
                fine = torch.isfinite(y64) & torch.isfinite(mag)
                within("y", y[fine], y64[fine], (u * y64.abs() + (1 + u) * ey + 1e-38)[fine])
                if place == "b":
                    other = torch.arange(N) != N - 3
                    assert torch.equal(bits(y[:, other]), bits(clean[:, other]))
                else:
                    assert torch.equal(bits(y[keep]), bits(clean[keep]))


# ------------------------------------------------------------------------- linear, backward

def check_backward(ops, M, N, K, dtype, act, zfull, xfull):
    print(f"[backward] M={M} N={N} K={K} {dtype} {act} z in full={zfull} x in full={xfull}", flush=True)
    g = gen("bwd", M, N, K, str(dtype), act)
    gy, w = randn(g, M, N, dtype=dtype), randn(g, N, K, dtype=dtype, sd=N ** -0.5)
    x, z = randn(g, M, K, dtype=dtype), randn(g, M, N, dtype=dtype, sd=1.5)
    u = U[dtype]
    zz = None if act == "none" else z if zfull else ops.checkpoint_pack(z)
    gz, gb = ops.activation_backward(gy, zz, act)
    if act == "none":
        assert gz is gy
        gz64, egz = gy.double(), torch.zeros_like(gy, dtype=torch.float64)
    else:
        z64 = z.double() if zfull else value64(zz)
        gz64 = gy.double() * slope64(z64, act)
        egz = gy.double().abs() * (0 if act == "relu" else 2.0 ** -19 * z64.abs().clamp(min=1)) + 2.0 ** -23 * gz64.abs()
        within("gz", gz, gz64, u * gz64.abs() + (1 + u) * egz + 1e-38)
    gb64 = gz64.sum(0)
    within("gb", gb, gb64, u * gb64.abs() + (1 + u) * (egz.sum(0) + GAMMA(M) * gz64.abs().sum(0)) + 1e-38)
    xx = x if xfull else ops.checkpoint_pack(x)
    x64 = x.double() if xfull else value64(xx)
    gx, gw = ops.linear_backward(gz, w, xx)
    d = gz.double()
    gx64, gw64 = d @ w.double(), d.t().contiguous() @ x64
    within("gx", gx, gx64, u * gx64.abs() + (1 + u) * GAMMA(N) * (d.abs() @ w.double().abs()) + 1e-38)
    within("gw", gw, gw64, u * gw64.abs() + (1 + u) * GAMMA(M) * (d.abs().t().contiguous() @ x64.abs()) + 1e-38)
    one, none = ops.linear_backward(gz, w, xx, need_gw=False)
    assert none is None and torch.equal(bits(one), bits(gx))
    none, one = ops.linear_backward(gz, w, xx, need_gx=False)
    assert none is None and torch.equal(bits(one), bits(gw))


BWD_SHAPES = [(1, 8, 8), (1, 768, 768), (2, 1000, 40), (7, 72, 2048), (16, 4096, 136), (31, 64, 72), (49, 448, 1792),
              (63, 264, 1032), (64, 64, 64), (65, 8, 1024), (128, 128, 64), (129, 136, 520), (257, 520, 264),
              (1000, 72, 8), (2050, 256, 512), (4099, 200, 776)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("i", range(len(BWD_SHAPES)), ids=lambda i: "x".join(map(str, BWD_SHAPES[i])))
def test_linear_backward(i, dtype):
    from rank_compressed_backprop_amd import ops
    M, N, K = BWD_SHAPES[i]
    check_backward(ops, M, N, K, dtype, ACTS[i % 5], bool(i % 2), bool((i // 2) % 2))
    check_backward(ops, M, N, K, dtype, ACTS[(i + 3) % 5], not i % 2, not (i // 2) % 2)


@pytest.mark.parametrize("shape", [(16384, 768, 768), (2048, 11008, 4096), (6272, 1792, 448), (6272, 448, 1792)],
                         ids=str)
@pytest.mark.parametrize("full", [False, True], ids=["8-bit", "full"])
def test_linear_backward_workload_sizes(shape, full):
    from rank_compressed_backprop_amd import ops
    check_backward(ops, *shape, BF, "gelu_tanh", full, full)


def test_slopes_far_out():
    """Slopes at large, infinite and NaN pre-activations: settled, with no inf * 0."""
    from rank_compressed_backprop_amd import ops
    z = torch.tensor([0.0, -0.0, 30.0, -30.0, 200.0, -200.0, 3e19, -3e19, 1e38, -1e38, float("inf"), -float("inf"),
                      float("nan"), 5.0, -5.0, 88.0]).cuda().reshape(1, 16)
    for dtype in (BF, FP):
        for act in ACTS[1:]:
            gz, _ = ops.activation_backward(torch.ones_like(z).to(dtype), z.to(dtype), act)
            want = torch.where(z == float("inf"), 1.0, torch.where(z == -float("inf"), 0.0, slope64(z, act).float()))
            if act == "relu":
                want = torch.where(torch.isnan(z), z, want)
            want = torch.where((z.abs() > 100) & torch.isfinite(z), (z > 0).float(), want)
            assert torch.equal(torch.isnan(gz[0]), torch.isnan(z[0])), (act, gz)
            fine = ~torch.isnan(z[0])
            assert bool(((gz.float() - want)[0][fine].abs() <= U[dtype] * 1.13 + 2.0 ** -19 * 200).all()), (act, gz)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("act,low", [("gelu", -12.5), ("gelu_tanh", -9.5), ("silu", -80.0)])
def test_activation_tails(act, low, dtype):
    """Far below zero an activation and its slope are small, and still right relative to their
    value. An exponential's argument of up to 88 is built in up to four roundings of 2^-24, 2.1e-5
    of the value, and the distribution function is fitted to 2.1e-5: together within 2^-14, beside
    the output's own rounding."""
    from rank_compressed_backprop_amd import ops
    z = torch.linspace(low, -1.5, 4096).reshape(512, 8).to(dtype).cuda()  # (below the slopes' zeros)
    y, _ = ops.linear_forward(z, torch.eye(8, dtype=dtype, device="cuda"), activation=act)
    gz, _ = ops.activation_backward(torch.ones_like(z), z, act)
    z64 = z.double()
    if act == "gelu":
        y64 = z64 * 0.5 * torch.erfc(-z64 / 2 ** 0.5)
        s64 = 0.5 * torch.erfc(-z64 / 2 ** 0.5) + z64 * torch.exp(-z64 ** 2 / 2) / (2 * np.pi) ** 0.5
    else:  # z sigmoid(v), whose terms do not cancel
        c = 2 * (2 / np.pi) ** 0.5
        v = z64 if act == "silu" else c * (z64 + 0.044715 * z64 ** 3)
        dv = 1.0 if act == "silu" else c * (1 + 3 * 0.044715 * z64 ** 2)
        s = torch.sigmoid(v)
        y64, s64 = z64 * s, s + z64 * s * (1 - s) * dv
    for name, got, ref in (("y", y, y64), ("slope", gz, s64)):
        within(f"{act} {name}", got, ref, (U[dtype] + (1 + U[dtype]) * 2.0 ** -14) * ref.abs())


# ------------------------------------------------------------------------- RMS norm

NORM_SHAPES = [(1, 8), (1, 4096), (3, 40), (5, 512), (4, 520), (2, 1032), (301, 768), (9, 2048), (7, 2056), (6, 4104),
               (3, 8192), (3, 11008), (2, 16384), (3, 16392), (2, 40000), (2, 65536), (4099, 256), (1030, 4096)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_rmsnorm(shape, dtype):
    from rank_compressed_backprop_amd import ops
    M, C = shape
    u = U[dtype]
    for res in (False, True):
        print(f"[rmsnorm] {shape} {dtype} res={res}", flush=True)
        g = gen("norm", shape, str(dtype), res)
        x, w = randn(g, M, C, dtype=dtype), (1 + randn(g, C, sd=0.2)).to(dtype)
        r = randn(g, M, C, dtype=dtype) if res else None
        out = ops.rmsnorm_forward(x, w, r, eps=1e-5, y8=True)
        if res:
            assert torch.equal(bits(out.h), bits((x.float() + r.float()).to(dtype)))
        else:
            assert out.h is x
        h = out.h.double()
        rstd = (h.square().mean(1) + 1e-5).rsqrt()
        er = (0.5 * GAMMA(C) + 2.0 ** -22) * rstd  # a relative error of the mean halves in its root
        within("rstd", out.rstd, rstd, er)
        y = h * rstd[:, None] * w.double()
        within("y", out.y, y, u * y.abs() + (1 + u) * (er / rstd + 2.0 ** -22)[:, None] * y.abs() + 1e-38)
        c = ops.checkpoint_pack(out.y)
        assert torch.equal(c.q, out.y8.q) and torch.equal(c.scale, out.y8.scale)
        only = ops.rmsnorm_forward(x, w, r, eps=1e-5, y=False, y8=True)
        assert only.y is None and torch.equal(only.y8.q, c.q) and torch.equal(only.y8.scale, c.scale)

        gy = randn(g, M, C, dtype=dtype)
        gh = randn(g, M, C, dtype=dtype) if res else None
        gx, gw = ops.rmsnorm_backward(gy, out.h, w, out.rstd, gh)
        rs = out.rstd.double()[:, None]
        t = gy.double() * w.double()
        c1 = (t * h).mean(1, keepdim=True)
        gx64 = rs * (t - h * rs * rs * c1)
        e = 2.0 ** -21 * rs * (t.abs() + (h * rs * rs * c1).abs()) + \
            rs ** 3 * h.abs() * GAMMA(C) * (t * h).abs().mean(1, keepdim=True)
        if res:
            gx64 = gx64 + gh.double()
            e = e + 2.0 ** -23 * gx64.abs()
        within("gx", gx, gx64, u * gx64.abs() + (1 + u) * e + 1e-38)
        p = gy.double() * h * rs
        within("gw", gw, p.sum(0), u * p.sum(0).abs() + (1 + u) * (GAMMA(M) + 2.0 ** -22) * p.abs().sum(0) + 1e-38)
        one, none = ops.rmsnorm_backward(gy, out.h, w, out.rstd, gh, need_gweight=False)
        assert none is None and torch.equal(bits(one), bits(gx))


def test_rmsnorm_gradient_against_differences():
    """The gradient in float32 against central differences of the norm in float64."""
    from rank_compressed_backprop_amd import ops
    g = gen("norm differences")
    x, w, gy = randn(g, 4, 72), 1 + randn(g, 72, sd=0.2), randn(g, 4, 72)
    out = ops.rmsnorm_forward(x, w, eps=1e-3)
    gx, gw = ops.rmsnorm_backward(gy, out.h, w, out.rstd)

    def loss(x, w):
        return (gy.double() * x * (x.square().mean(1, keepdim=True) + 1e-3).rsqrt() * w).sum().item()
    d = 1e-5
    for i in range(0, 72, 7):
        e = torch.zeros(4, 72, dtype=torch.float64, device="cuda")
        e[i % 4, i] = d
        num = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * d)
        assert abs(num - gx[i % 4, i].item()) <= 1e-5 * (1 + abs(num))  # d^2 = 1e-10 and float32's 6e-8 stay below
        e = torch.zeros(72, dtype=torch.float64, device="cuda")
        e[i] = d
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * d)
        assert abs(num - gw[i].item()) <= 1e-5 * (1 + abs(num))


def test_rmsnorm_rows_alone():
    """Zero rows, and rows that hold an infinity or NaN, touch no other row."""
    from rank_compressed_backprop_amd import ops
    for C in (64, 4096):
        g = gen("norm rows", C)
        x, w = randn(g, 6, C, dtype=BF), (1 + randn(g, C, sd=0.2)).to(BF)
        clean = ops.rmsnorm_forward(x, w, y8=True)
        x[1], x[2, 3], x[4, 5] = 0, float("inf"), float("nan")
        out = ops.rmsnorm_forward(x, w, y8=True)
        for m in (0, 3, 5):
            assert torch.equal(bits(out.y[m]), bits(clean.y[m]))
        assert bool((out.y[1] == 0).all()) and bool((out.y8.q[1] == 0).all())
        assert bool(torch.isnan(out.y[2, 3])) and bool(torch.isnan(out.y[4]).all())
        assert int(out.y8.scale[2, 0]) == 255 and bool((out.y8.scale[4] == 255).all())


# ------------------------------------------------------------------------- calls

def test_no_rows():
    from rank_compressed_backprop_amd import ops
    for dtype in (BF, FP):
        x, w = torch.empty(0, 40, dtype=dtype, device="cuda"), torch.ones(24, 40, dtype=dtype, device="cuda")
        y, z = ops.linear_forward(x, w, activation="gelu", save="z8")
        assert y.shape == (0, 24) and z.q.shape == (0, 24)
        gz, gb = ops.activation_backward(y, z, "gelu")
        gx, gw = ops.linear_backward(gz, w, ops.checkpoint_pack(x))
        assert gx.shape == (0, 40)
        assert torch.equal(gb, torch.zeros_like(gb)) and torch.equal(gw, torch.zeros_like(w))
        out = ops.rmsnorm_forward(x, w[0], x, y8=True)
        gx, gg = ops.rmsnorm_backward(x, out.h, w[0], out.rstd)
        assert torch.equal(gg, torch.zeros_like(gg))
        assert ops.checkpoint_unpack(out.y8).shape == (0, 40)


def test_leading_dimensions():
    from rank_compressed_backprop_amd import ops
    g = gen("lead")
    x, w = randn(g, 2, 3, 5, 40, dtype=BF), randn(g, 24, 40, dtype=BF)
    y, z = ops.linear_forward(x, w, activation="silu", save="z8")
    y2, z2 = ops.linear_forward(x.reshape(30, 40), w, activation="silu", save="z8")
    assert y.shape == (2, 3, 5, 24) and z.scale.shape == (2, 3, 5, 1)
    assert torch.equal(bits(y).reshape(30, 24), bits(y2)) and torch.equal(z.q.reshape(30, 24), z2.q)
    gz, gb = ops.activation_backward(y, z, "silu")
    gx, gw = ops.linear_backward(gz, w, ops.checkpoint_pack(x))
    assert gx.shape == x.shape and gw.shape == w.shape
    out = ops.rmsnorm_forward(x, w[0], y8=True)
    assert out.rstd.shape == (2, 3, 5) and out.y8.scale.shape == (2, 3, 5, 2)


def _guarded(shape, dtype, kind=None):
    """A buffer for an output with 256 bytes of a pattern around it: (the view, the whole, the edges)."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((256 + (n + 15) // 16 * 16 + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    return whole[256:256 + n].view(dtype).reshape(shape), whole, n


def _edges_kept(*guarded):
    for _, whole, n in guarded:
        assert bool((whole[:256] == 0x5A).all()) and bool((whole[256 + n:] == 0x5A).all())


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 776, 1544), (5, 136, 72), (17, 1000, 264), (130, 264, 136),
                                   (300, 520, 1032)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_writes_stay_inside_and_in_place_calls(M, N, K, dtype):
    """Nothing outside an output is written (the workspace's end included), and the overlaps that
    the interface allows give the same bits."""
    import rank_compressed_backprop_amd as rcb
    from rank_compressed_backprop_amd import ops
    print(f"[guard] {M} {N} {K} {dtype}", flush=True)
    g = gen("guard", M, N, K)
    code = rcb.INSTANT_BF16 if dtype == BF else rcb.INSTANT_FP32
    x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype)
    b, r, gy = randn(g, N, dtype=dtype), randn(g, M, N, dtype=dtype), randn(g, M, N, dtype=dtype)
    G = (N + 31) // 32
    n = ops.instant_linear_workspace_bytes(M, N, K, code)
    ws = _guarded((n,), torch.uint8)
    y, zq, zs = _guarded((M, N), dtype), _guarded((M, N), torch.int8), _guarded((M, G), torch.uint8)
    assert ops.instant_linear_fwd(x, w, b, r, M, N, K, code, 2, y[0], None, zq[0], zs[0], ws[0], n) == 0
    y2, z2 = ops.linear_forward(x, w, b, r, "gelu", "z8")
    assert torch.equal(bits(y[0]), bits(y2)) and torch.equal(zq[0], z2.q) and torch.equal(zs[0], z2.scale)
    _edges_kept(y, zq, zs, ws)
    acc = r.clone()
    assert ops.instant_linear_fwd(x, w, b, acc, M, N, K, code, 2, acc, None, None, None, ws[0], n) == 0
    assert torch.equal(bits(acc), bits(y2))

    gz, gb = _guarded((M, N), dtype), _guarded((N,), dtype)
    assert ops.instant_act_bwd(gy, None, zq[0], zs[0], M, N, code, 2, gz[0], gb[0], ws[0], n) == 0
    gz2, gb2 = ops.activation_backward(gy, z2, "gelu")
    assert torch.equal(bits(gz[0]), bits(gz2)) and torch.equal(bits(gb[0]), bits(gb2))
    over = gy.clone()
    assert ops.instant_act_bwd(over, None, zq[0], zs[0], M, N, code, 2, over, None, None, 0) == 0
    assert torch.equal(bits(over), bits(gz2))
    x8 = ops.checkpoint_pack(x)
    gx, gw = _guarded((M, K), dtype), _guarded((N, K), dtype)
    assert ops.instant_linear_bwd(gz2, w, None, x8.q, x8.scale, M, N, K, code, gx[0], gw[0], ws[0], n) == 0
    gx2, gw2 = ops.linear_backward(gz2, w, x8)
    assert torch.equal(bits(gx[0]), bits(gx2)) and torch.equal(bits(gw[0]), bits(gw2))
    _edges_kept(gz, gb, gx, gw, ws)

    wn = w[0].contiguous()
    h, yy, q, s = (_guarded((M, K), dtype), _guarded((M, K), dtype), _guarded((M, K), torch.int8),
                   _guarded((M, (K + 31) // 32), torch.uint8))
    rs = _guarded((M,), torch.float32)
    assert ops.instant_rmsnorm_fwd(x, gx2, wn, M, K, code, 1e-5, h[0], yy[0], q[0], s[0], rs[0]) == 0
    out = ops.rmsnorm_forward(x, wn, gx2, 1e-5, y8=True)
    assert torch.equal(bits(h[0]), bits(out.h)) and torch.equal(bits(yy[0]), bits(out.y))
    assert torch.equal(q[0], out.y8.q) and torch.equal(s[0], out.y8.scale) and torch.equal(rs[0], out.rstd)
    for first in (True, False):
        a, c = x.clone(), gx2.clone()
        assert ops.instant_rmsnorm_fwd(a, c, wn, M, K, code, 1e-5, a if first else c, yy[0], None, None, None) == 0
        assert torch.equal(bits(a if first else c), bits(out.h)) and torch.equal(bits(yy[0]), bits(out.y))
    nn = ops.instant_rmsnorm_workspace_bytes(M, K)
    wsn, gxn, ggn = _guarded((nn,), torch.uint8), _guarded((M, K), dtype), _guarded((K,), dtype)
    assert ops.instant_rmsnorm_bwd(x, out.h, wn, out.rstd, gx2, M, K, code, gxn[0], ggn[0], wsn[0], nn) == 0
    gx3, gg3 = ops.rmsnorm_backward(x, out.h, wn, out.rstd, gx2)
    assert torch.equal(bits(gxn[0]), bits(gx3)) and torch.equal(bits(ggn[0]), bits(gg3))
    for which in (0, 1):
        a, c = x.clone(), gx2.clone()
        assert ops.instant_rmsnorm_bwd(a, out.h, wn, out.rstd, c, M, K, code, (a, c)[which], None, None, 0) == 0
        assert torch.equal(bits((a, c)[which]), bits(gx3))
    xq, xs = _guarded((M, K), torch.int8), _guarded((M, (K + 31) // 32), torch.uint8)
    assert ops.instant_ckpt_pack(x, M, K, code, xq[0], xs[0]) == 0
    up = _guarded((M, K), dtype)
    assert ops.instant_ckpt_unpack(xq[0], xs[0], M, K, code, up[0]) == 0
    assert torch.equal(xq[0], x8.q) and torch.equal(xs[0], x8.scale)
    _edges_kept(h, yy, q, s, rs, wsn, gxn, ggn, xq, xs, up)


def _chain(ops, x, r, g, w1, b1, w2, b2, gout):
    """A pre-norm MLP block, forward and backward, from the operators: the norm writes the first
    layer's checkpoint, the first layer its pre-activation's, and the second adds the residual."""
    n = ops.rmsnorm_forward(x, g, residual=r, eps=1e-5, y8=True)
    a, z8 = ops.linear_forward(n.y, w1, b1, activation="gelu_tanh", save="z8")
    a8 = ops.checkpoint_pack(a)
    out, _ = ops.linear_forward(a, w2, b2, residual=n.h)
    _, gb2 = ops.activation_backward(gout, None)
    ga, gw2 = ops.linear_backward(gout, w2, a8)
    gz, gb1 = ops.activation_backward(ga, z8, "gelu_tanh")
    gy, gw1 = ops.linear_backward(gz, w1, n.y8)
    gx, gg = ops.rmsnorm_backward(gy, n.h, g, n.rstd, gh=gout)
    return {"out": out, "gx": gx, "gg": gg, "gw1": gw1, "gb1": gb1, "gw2": gw2, "gb2": gb2}


def _chain_inputs(dtype, M=392, C=448, H=1792):
    g = gen("chain", M, C, H)
    return (randn(g, M, C, dtype=dtype), randn(g, M, C, dtype=dtype), (1 + randn(g, C, sd=0.1)).to(dtype),
            randn(g, H, C, dtype=dtype, sd=C ** -0.5), randn(g, H, dtype=dtype, sd=0.1),
            randn(g, C, H, dtype=dtype, sd=H ** -0.5), randn(g, C, dtype=dtype, sd=0.1), randn(g, M, C, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_block_against_autograd_in_64_bits(dtype):
    from rank_compressed_backprop_amd import ops
    args = _chain_inputs(dtype)
    got = _chain(ops, *args)
    x, r, g, w1, b1, w2, b2, gout = [t.double().detach().requires_grad_(True) for t in args]
    h = x + r
    y = h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g
    out = act64(y @ w1.t() + b1, "gelu_tanh") @ w2.t() + b2 + h
    ref = dict(zip(["gx", "gg", "gw1", "gb1", "gw2", "gb2"],
                   torch.autograd.grad(out, (x, g, w1, b1, w2, b2), gout.detach())), out=out.detach())
    # bf16: about ten roundings of 2^-9 rms lie between an input and a gradient (10^0.5 2^-9 = 6e-3)
    # and the 8-bit steps: a group's rms step is at most max / 63.5 / 12^0.5, with max under 4 of
    # the group's rms, 1.8e-2, and it enters a gradient once (x8, a8) or through the slope (z8).
    # fp32: the 8-bit steps alone.
    for k, v in ref.items():
        e = ((got[k].double() - v).norm() / v.norm()).item()
        print(f"  {k}: {e:.2e}", flush=True)
        assert e <= (0.03 if k != "out" else 0.01 if dtype == BF else 1e-5), (k, e)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_repeatable_and_captured(dtype):
    """The same bits on every call, on another stream, and on every replay of a captured graph
    with the program's own work between the replays; new inputs reach a replay."""
    from rank_compressed_backprop_amd import ops
    args = _chain_inputs(dtype, 200, 264, 1032)
    first = _chain(ops, *args)
    again = _chain(ops, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = _chain(ops, *args)
    torch.cuda.current_stream().wait_stream(side)
    for k in first:
        assert torch.equal(bits(first[k]), bits(again[k])), k
        assert torch.equal(bits(first[k]), bits(third[k])), k
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = _chain(ops, *args)
    other = _chain_inputs(dtype, 200, 264, 1032)
    for rep in range(4):
        if rep == 2:
            args[0].mul_(-0.5)
            first = _chain(ops, *args)
        graph.replay()
        _chain(ops, *other)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(bits(first[k]), bits(kept[k])), (rep, k)


def test_two_graphs_and_an_eager_call_at_once():
    """Every call has its own workspace: two captured graphs and eager calls on three streams."""
    from rank_compressed_backprop_amd import ops
    sets = [_chain_inputs(BF, m, 264, 1032) for m in (40, 72, 104)]
    want = [_chain(ops, *s) for s in sets]
    torch.cuda.synchronize()
    graphs, kept = [], []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(_chain(ops, *s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for rep in range(3):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = _chain(ops, *sets[2])
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(bits(eager[k]), bits(want[2][k])), (rep, k)
            for i in range(2):
                assert torch.equal(bits(kept[i][k]), bits(want[i][k])), (rep, i, k)


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements: the rows behind that border."""
    from rank_compressed_backprop_amd import ops
    M, N = 262400, 8192
    assert M * N > 1 << 31
    g = gen("far")
    tail = randn(g, 200, N, dtype=BF)
    gy = torch.zeros(M, N, dtype=BF, device="cuda")
    gy[-200:] = tail
    c = ops.checkpoint_pack(gy)
    t = ops.checkpoint_pack(tail)
    assert torch.equal(c.q[-200:], t.q) and torch.equal(c.scale[-200:], t.scale)
    assert torch.equal(ops.checkpoint_unpack(c)[-200:], ops.checkpoint_unpack(t))
    gz, gb = ops.activation_backward(gy, c, "silu")
    gz2, gb2 = ops.activation_backward(tail, t, "silu")
    assert torch.equal(bits(gz[-200:]), bits(gz2))
    del c
    w = randn(g, N, 8, dtype=BF, sd=N ** -0.5)
    x = torch.zeros(M, 8, dtype=BF, device="cuda")
    x[-200:] = randn(g, 200, 8, dtype=BF)
    gx, gw = ops.linear_backward(gz, w, x)
    d, x64 = gz2.double(), x[-200:].double()
    within("gx", gx[-200:], d @ w.double(), U[BF] * (d @ w.double()).abs() + 1.01 * GAMMA(N) * (d.abs() @ w.double().abs()))
    # (the zero rows add exactly nothing)
    within("gw", gw, d.t().contiguous() @ x64, U[BF] * (d.t().contiguous() @ x64).abs() +
           1.01 * GAMMA(M) * (d.abs().t().contiguous() @ x64.abs()))
    del gz, gx
    y, z = ops.linear_forward(x, w, activation="gelu", save="z8")
    y2, z2 = ops.linear_forward(x[-200:].contiguous(), w, activation="gelu", save="z8")
    within("y", y[-200:], y2.double(), 2 * U[BF] * y2.double().abs() + 2.0 ** -18)
    assert bool((z.scale[:M - 200] == 1).all())
    del y, z
    out = ops.rmsnorm_forward(gy, w[:, 0].contiguous(), y8=True)
    out2 = ops.rmsnorm_forward(tail, w[:, 0].contiguous(), y8=True)
    assert torch.equal(bits(out.y[-200:]), bits(out2.y)) and torch.equal(out.y8.q[-200:], out2.y8.q)
    gx, _ = ops.rmsnorm_backward(gy, out.h, w[:, 0].contiguous(), out.rstd)
    gx2, _ = ops.rmsnorm_backward(tail, out2.h, w[:, 0].contiguous(), out2.rstd)
    assert torch.equal(bits(gx[-200:]), bits(gx2))


@pytest.mark.parametrize("dtype,M,K", [(BF, 16500, 8192), (FP, 8250, 8192), (BF, 33000, 8192)])
def test_weight_gradient_in_chunks(dtype, M, K):
    """Checkpoints whose values in full pass the workspace's 256 MB: gw adds up over chunks of
    rows, the last of them short."""
    import rank_compressed_backprop_amd as rcb
    from rank_compressed_backprop_amd import ops
    N = 24
    code = rcb.INSTANT_BF16 if dtype == BF else rcb.INSTANT_FP32
    assert M * K * (2 if dtype == BF else 4) > 256 << 20
    assert ops.instant_linear_bwd_workspace_bytes(M, N, K, code, True) < 512 << 20
    g = gen("chunks", M)
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(M)).to(dtype)
    gz = randn(g, M, N, dtype=dtype)
    c = ops.checkpoint_pack(x)
    _, gw = ops.linear_backward(gz, torch.zeros(N, K, dtype=dtype, device="cuda"), c, need_gx=False)
    _, again = ops.linear_backward(gz, torch.zeros(N, K, dtype=dtype, device="cuda"), c, need_gx=False)
    assert torch.equal(bits(gw), bits(again))
    d = gz.double().t().contiguous()
    ref = mag = 0
    for m in range(0, M, 4096):
        v = value64(ops.Checkpoint8(c.q[m:m + 4096], c.scale[m:m + 4096]))
        ref, mag = ref + d[:, m:m + 4096] @ v, mag + d[:, m:m + 4096].abs() @ v.abs()
    within("gw", gw, ref, U[dtype] * ref.abs() + 1.01 * GAMMA(M) * mag + 1e-38)


def test_wrong_arguments_raise():
    from rank_compressed_backprop_amd import ops
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(32, 64, dtype=BF, device="cuda")
    y = torch.zeros(4, 32, dtype=BF, device="cuda")
    c = ops.checkpoint_pack(x)
    for exc, call in [
        (ValueError, lambda: ops.linear_forward(x, w[:, :32])), (ValueError, lambda: ops.linear_forward(x, w.t())),
        (ValueError, lambda: ops.linear_forward(x[:, ::2], w)), (TypeError, lambda: ops.linear_forward(x, w.float())),
        (ValueError, lambda: ops.linear_forward(x, w, bias=x[0])), (ValueError, lambda: ops.linear_forward(x, w, residual=x)),
        (ValueError, lambda: ops.linear_forward(x, w, activation="tanh")), (ValueError, lambda: ops.linear_forward(x, w, save="y")),
        (ValueError, lambda: ops.linear_forward(x, w.cpu())), (ValueError, lambda: ops.linear_forward(x.cpu(), w)),
        (ValueError, lambda: ops.activation_backward(y, None, "gelu")), (ValueError, lambda: ops.activation_backward(y, y)),
        (ValueError, lambda: ops.activation_backward(y, c, "gelu")), (TypeError, lambda: ops.activation_backward(y, y.float(), "gelu")),
        (ValueError, lambda: ops.linear_backward(y, w, y)), (ValueError, lambda: ops.linear_backward(x, w, x)),
        (TypeError, lambda: ops.linear_backward(y, w, ops.Checkpoint8(c.q, c.q))),
        (ValueError, lambda: ops.linear_backward(y, w, ops.Checkpoint8(c.q, c.scale[:, :1]))),
        (ValueError, lambda: ops.rmsnorm_forward(x, w)), (ValueError, lambda: ops.rmsnorm_forward(x, w[0], eps=-1.0)),
        (ValueError, lambda: ops.rmsnorm_forward(x, w[0], y=False)), (ValueError, lambda: ops.rmsnorm_forward(x, w[0], residual=w)),
        (TypeError, lambda: ops.rmsnorm_backward(x, x, w[0], x[:, 0])),
        (ValueError, lambda: ops.rmsnorm_backward(x, x, w[0], torch.zeros(3, device="cuda"))),
    ]:
        with pytest.raises(exc):
            call()
