"""GPU tests of the operators at a training step's ends (include/instant_ops.h): embedding, token
log probabilities, gradient norm and clipping, against plain 64-bit implementations.

Tolerances. u = 2^-24 and U (bf16 2^-8, fp32 2^-24) are half a step relative to the value: what one
rounding is off by at most.

Log probabilities. With t = z - m <= 0 an exponential is taken of log2(e) t, evaluated in float32: at
most three roundings (the difference, log2(e), the product) that reach it |t|-fold, and the hardware's
own 1 ulp, so a term of S is off by at most (3 |t| + 2) u of itself. |t| is at most D, the row's range
(104 at most: below, the term is 0 in float32, which is off by less than V 2^-149). A running sum of n
terms of one sign adds n u, and each of its n / 32 + 12 raises of the maximum (the joins of threads
among them) multiplies by an exponential of its own (4 u and 3 u times the distance, D in all):
REL(n, D) below, with n = V the most that one thread may hold. E has terms of one sign too and the same
bound, relative to itself.
"""
import zlib

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

u = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, FP = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
DTYPES = pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])


def REL(n, D):
    return u * (6 * D + n + 4 * (n / 32 + 12) + 10)


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def randn(g, *shape, dtype=FP, sd=1.0):
    return (torch.randn(*shape, generator=g) * sd).to(dtype).cuda()


def within(name, got, ref, bound):
    """got is within bound of ref; infinities are equal, and NaNs are where ref's are. (A difference
    of two logits of 2^127 and more may be -2^128 and beyond: no float32 is nearer than -inf.)"""
    got, ref = got.double(), ref.double()
    ref = torch.where(ref.abs() >= 2.0 ** 128, ref * INF, ref)
    bound = torch.as_tensor(bound, dtype=torch.float64, device=ref.device).expand(ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    d = torch.where(same, 0.0, (got - ref).abs())
    ratio = (d / bound.clamp(min=1e-300)).max().item() if d.numel() else 0.0
    print(f"  {name}: worst error / bound {ratio:.3f}", flush=True)
    assert bool(((d <= bound) | same).all()), f"{name}: {ratio} of the bound"


def bits(t):
    return t.view(torch.int16) if t.dtype == BF else t.view(torch.int32) if t.dtype == FP else t


# ------------------------------------------------------------------------- log probabilities

def logprobs64(z, t, ignore=-100):
    """(logp, lse, entropy, p, log p) by the definition; rows of -inf have probability 0."""
    z = z.double()
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -INF, 0.0, m)
    e = torch.exp(z - m)
    S = e.sum(1, keepdim=True)
    empty = S == 0
    lp = torch.where(empty, -INF, z - m - torch.log(S))
    p = torch.where(lp == -INF, 0.0, torch.exp(lp))
    H = -torch.where(p == 0, 0.0, p * lp).sum(1)
    lse = (m + torch.log(S))[:, 0]
    V = z.shape[1]
    bad = (t < 0) | (t >= V)
    logp = lp.gather(1, torch.where(bad, 0, t).long()[:, None])[:, 0]
    logp = torch.where(t == ignore, 0.0, torch.where(bad, NAN, logp))
    return logp, lse, H, p, lp


def bounds(z, logp, lse, H):
    """Of logp, lse and H, for finite rows."""
    z = torch.where(z.isinf(), NAN, z.double())
    m = torch.nan_to_num(z, nan=-INF).amax(1)
    low = torch.nan_to_num(z, nan=INF).amin(1)
    D = torch.nan_to_num(m - low, nan=0.0, posinf=0.0, neginf=0.0).clamp(0, 104)
    rel = REL(z.shape[1], D)
    ls = torch.nan_to_num(lse - m, nan=0.0, posinf=0.0, neginf=0.0).abs()
    E = (ls - H).abs()
    small = z.shape[1] * 2.0 ** -140
    b_ls = rel + 2 * u * ls + small
    return (b_ls + 2 * u * (torch.nan_to_num(logp.abs(), posinf=0.0) + 2 * ls), b_ls + u * torch.nan_to_num(lse.abs(), posinf=0.0),
            b_ls + (2 * rel + 4 * u) * E + u * H + 120 * small)


def top64(z, k):
    """The places of the k largest, equal ones by their place, a NaN as -inf."""
    z = torch.where(z.isnan(), -INF, z.double()) + 0.0
    return torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]


def check_forward(z, t, top, vocab=None, ignore=-100, out=None):
    from rank_compressed_backprop_amd import ops
    if out is None:
        out = ops.token_logprobs(z, t, vocab=vocab, top=top, ignore=ignore)
    flat = z.flatten(0, -2)[:, :vocab]
    logp, lse, H, p, lp = logprobs64(flat, t.flatten(), ignore)
    b = bounds(flat, logp, lse, H)
    within("logp", out.logp.flatten(), logp, b[0])
    within("lse", out.lse.flatten(), lse, b[1])
    within("entropy", out.entropy.flatten(), H, b[2])
    assert out.logp.shape == out.lse.shape == out.entropy.shape == t.shape and out.stats.shape == (*t.shape, 2)
    if top:
        i = top64(flat, top)
        assert out.top_index.shape == out.top_logp.shape == (*t.shape, top)
        assert torch.equal(out.top_index.flatten(0, -2), i)
        want = lp.gather(1, i)
        within("top", out.top_logp.flatten(0, -2), want,
               b[0][:, None] + 2 * u * torch.nan_to_num(want.abs(), posinf=0.0, nan=0.0))
    return out


def check_backward(z, t, out, g, gl, gh, vocab=None, ignore=-100, in_place=False, gz=None):
    from rank_compressed_backprop_amd import ops
    V = z.shape[-1] if vocab is None else vocab
    flat, tf = z.flatten(0, -2)[:, :V].clone(), t.flatten()
    logp, lse, H, p, lp = logprobs64(flat, tf, ignore)
    zero = torch.zeros_like(H)
    seen = tf != ignore
    gd = zero if g is None else torch.where(seen, g.flatten().double(), 0.0)
    bad = seen & ((tf < 0) | (tf >= V)) if g is not None else seen & False
    gd = torch.where(bad, NAN, gd)
    gld, ghd = (zero if x is None else x.flatten().double() for x in (gl, gh))
    lp0 = torch.where(p == 0, 0.0, lp)
    ref = p * (gld - gd)[:, None] - torch.where(p == 0, 0.0, ghd[:, None] * p * (lp0 + H[:, None]))
    rows = torch.arange(len(tf), device="cuda")
    ok = seen & (tf >= 0) & (tf < V)
    ref[rows[ok], tf[ok].long()] += gd[ok]
    none = (torch.nan_to_num(gd, nan=1.0) == 0) & (gld == 0) & (ghd == 0)
    ref[none] = 0
    bl = bounds(flat, logp, lse, H)
    ls = (lse - torch.where(flat.isinf(), -INF, flat.double()).amax(1)).abs()
    alp = lp0.abs()
    rp = bl[1][:, None] + u * (torch.nan_to_num(ls)[:, None] * 2 + 5 * alp + 4) + u * (alp + torch.nan_to_num(ls)[:, None])
    size = (gd.abs() + gld.abs())[:, None] + ghd.abs()[:, None] * (alp + H[:, None])
    bound = p * size * (rp + 8 * u) + ghd.abs()[:, None] * p * (rp + bl[2][:, None]) \
        + 2 * u * torch.zeros_like(ref).index_put((rows[ok], tf[ok].long()), gd[ok].abs()) \
        + U[z.dtype] * ref.abs() * (1 + 2.0 ** -20) + 2.0 ** -125 * (1 + size)
    bound = torch.nan_to_num(bound, nan=0.0)
    z0 = z.clone()
    if gz is None:
        gz = ops.token_logprobs_backward(z, t, out.stats, g, gl, gh, out.entropy, vocab, ignore, in_place)
    assert gz.shape == z.shape and gz.dtype == z.dtype
    if in_place:
        assert gz.data_ptr() == z.data_ptr()
    else:
        assert torch.equal(bits(z), bits(z0))
    full = gz.flatten(0, -2)
    assert not full[:, V:].any()
    within("gz", full[:, :V], ref, bound)
    return gz


LOGIT_SHAPES = [(1, 1, 0), (1, 2, 1), (3, 7, 7), (5, 33, 32), (2, 255, 5), (4, 256, 32), (7, 257, 3), (3, 1001, 20),
                (2, 2047, 32), (2, 2048, 32), (3, 2056, 32), (3, 2065, 31), (2, 4099, 1), (3, 30522, 20), (2, 32000, 5),
                (1, 32768, 32), (1, 40001, 32), (300, 16387, 2), (1, 131071, 32), (1, 262144, 32), (65, 2500, 0),
                (2048, 8000, 0), (2050, 8199, 1), (2049, 4099, 32), (2051, 9001, 5), (2048, 16391, 20), (2048, 32771, 2)]


@DTYPES
@pytest.mark.parametrize("shape", LOGIT_SHAPES, ids=str)
def test_token_logprobs(shape, dtype):
    m, v, top = shape
    print(f"[logprobs] {shape} {dtype}", flush=True)
    g = gen("lp", shape, str(dtype))
    z = randn(g, m, v, dtype=dtype, sd=3.0)
    t = torch.randint(0, v, (m,), generator=g).cuda()
    if m > 2:
        t[1] = -100
    out = check_forward(z, t, top)
    k = lambda: randn(g, m)  # noqa: E731
    for which in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        check_backward(z, t, out, *(k() if w else None for w in which))


@DTYPES
@pytest.mark.parametrize("width,vocab", [(8, 3), (64, 57), (1001, 1000), (1003, 640), (4104, 4097), (33000, 32999)])
def test_padded_vocabulary(width, vocab, dtype):
    """What stands behind the vocabulary is not looked at (NaN here), and gets zeros."""
    print(f"[padded] {width} {vocab} {dtype}", flush=True)
    g = gen("pad", width, vocab)
    z = randn(g, 5, 3, width, dtype=dtype)
    z[..., vocab:] = NAN
    t = torch.randint(0, vocab, (5, 3), generator=g, dtype=torch.int32).cuda()
    t[0, 1] = vocab  # outside: NaN
    out = check_forward(z, t, min(vocab, 9), vocab)
    assert out.logp[0, 1].isnan() and not out.lse[0, 1].isnan()
    check_backward(z, t, out, randn(g, 5, 3), randn(g, 5, 3), randn(g, 5, 3), vocab)


@DTYPES
@pytest.mark.parametrize("v", [40, 1000, 5003, 70001])
def test_masked_and_strange_rows(v, dtype):
    """-inf, the type's lowest, whole rows of either, one value left, equal rows, infinities, NaN."""
    print(f"[masked] {v} {dtype}", flush=True)
    g = gen("mask", v)
    z, t = strange_rows(g, v, dtype)
    rows = len(t)
    out = check_forward(z, t, 32 if v >= 32 else v)
    assert out.lse[1] == -INF and out.entropy[1] == 0 and out.logp[1] == -INF
    assert out.logp[9] == -INF and out.logp[10] == 0 and out.logp[11] == 0
    assert out.lse[7].isnan() and out.logp[8].isnan() and out.entropy[7].isnan()
    gz = check_backward(z, t, out, randn(g, rows), None, randn(g, rows))
    assert gz[7].isnan().all() and not gz[1][t[1]].isnan()
    gz = check_backward(z, t, out, randn(g, rows), None, None)
    assert not gz[10].any() and not gz[11].any()  # padding: zeros, whatever the row holds


def strange_rows(g, v, dtype):
    low = torch.finfo(dtype).min
    rows = 14
    z = randn(g, rows, v, dtype=dtype, sd=2.0)
    t = torch.randint(0, v, (rows,), generator=g).cuda()
    half = torch.rand(v, generator=g).cuda() < 0.5
    z[0, half] = -INF
    z[1] = -INF                       # nothing is left
    z[2, half] = low
    z[3] = low                        # uniform
    z[4] = -INF
    z[4, v // 2] = 5.0                # one is left
    z[5] = 1.5                        # equal throughout
    z[6] = 0.0
    z[6, 1::2] = -0.0
    z[7, v - 1] = NAN
    z[8, v // 3] = INF
    z[9, 0] = -INF
    t[9] = 0                          # a target of probability 0
    z[10] = -INF
    t[10] = -100                      # an empty row without a target
    z[11] = NAN
    t[11] = -100                      # a row of rubbish without a target
    z[12] = low
    z[12, v - 2] = torch.finfo(dtype).max / 2   # differences beyond float's range
    z[13] = torch.finfo(dtype).max
    return z, t


@DTYPES
@pytest.mark.parametrize("v", [3000, 33001, 131072])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_alternatives_in_hard_orders(v, k, dtype):
    """Rows in order, steps of equal values, and many values that beat the rest in the places of a
    few threads (more than the kernel holds at a time)."""
    print(f"[order] {v} {k} {dtype}", flush=True)
    z = hard_rows(gen("order", v, k), v, dtype)
    check_forward(z, torch.arange(7).cuda(), k)
    one = z[4:5].contiguous()         # (few rows: other blocks)
    check_forward(one, torch.zeros(1, dtype=torch.int64, device="cuda"), k)


@DTYPES
@pytest.mark.parametrize("v", [1000, 8191, 15997, 32700])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_many_hard_and_strange_rows(v, k, dtype):
    """The rows of the two tests before this among two thousand (other kernels take those)."""
    print(f"[many] {v} {k} {dtype}", flush=True)
    g = gen("many", v, k)
    z, t = strange_rows(g, v, dtype)
    z = torch.cat((z, hard_rows(g, v, dtype)))
    t = torch.cat((t, torch.arange(7).cuda()))
    times = 2058 // len(t)
    check_forward(z.repeat(times, 1), t.repeat(times), k)


def hard_rows(g, v, dtype):
    z = torch.zeros(7, v)
    ramp = torch.linspace(-20, 20, v)
    z[0], z[1] = ramp, ramp.flip(0)
    z[2] = torch.floor(ramp)
    z[3] = torch.floor(ramp).flip(0)
    z[4] = -30
    for first in range(0, v, 2048):   # chunks of the same threads
        z[4, first:first + 64] = torch.randn(z[4, first:first + 64].shape, generator=g)
    z[5] = -30
    z[5, v // 2:v // 2 + 2000] = 3.0
    z[6] = torch.randint(0, 3, (v,), generator=g)
    return z.to(dtype).cuda()


@DTYPES
def test_logprobs_largest_magnitudes_and_tails(dtype):
    """Logits of magnitude 1e4 (differences count, not magnitudes) and peaked rows."""
    g = gen("large")
    z = randn(g, 6, 777, sd=2.0)
    z[0] += 1e4
    z[1] -= 1e4
    z[2, 5] = 60.0
    z[3, 770] = 200.0
    z[4] *= 30
    z = z.to(dtype)
    t = torch.tensor([1, 2, 5, 0, 9, 776]).cuda()
    out = check_forward(z, t, 20)
    check_backward(z, t, out, randn(g, 6), randn(g, 6), randn(g, 6))


@DTYPES
@pytest.mark.parametrize("v", [40, 1000, 5003])
def test_gradient_of_large_equal_logits(v, dtype):
    """Two equal logits, far above all others: p is 1/2 whatever they are, so the gradient is half of
    what comes in. The exponents of the two are rests of roundings, exact, and sums of magnitude 1: 16 u
    hold them, log S and both exponentials (2 u each) in forward and backward pass."""
    from rank_compressed_backprop_amd import ops
    tops = [100.0, 1000.0, 4096.0, 12345.0, 65536.0, 100000.0, 523000.0, 1048576.0, 3e6, 1e9, -1000.0, -70000.0]
    z = torch.full((len(tops), v), -INF, dtype=dtype)
    z[:, 3] = z[:, v - 2] = torch.tensor(tops).to(dtype)
    z[:, 7] = z[:, 3] * torch.tensor([0.5 if x > 0 else 2.0 for x in tops])
    z, t = z.cuda(), torch.full((len(tops),), 3).cuda()
    g = randn(gen("equal", v), len(tops))
    out = ops.token_logprobs(z, t)
    within("logp", out.logp, torch.full((len(tops),), 0.5, dtype=torch.float64).log().cuda(), 16 * u)
    for gl, p_of in ((None, -0.5), (g.clone(), 0.0)):
        gz = ops.token_logprobs_backward(z, t, out.stats, g, gl).double()
        want = torch.zeros_like(gz)
        want[:, v - 2], want[:, 3] = g.double() * p_of, g.double() * (1 + p_of)
        within("gz", gz, want, U[dtype] * want.abs() * (1 + 2.0 ** -20) + 32 * u * g.abs().double()[:, None])


@DTYPES
@pytest.mark.parametrize("m,v", [(5, 57), (33, 1001), (3, 40007)])
def test_gradient_in_place_and_inside(m, v, dtype):
    """Outputs at odd places stay inside their rows; in place gives the same bits."""
    from rank_compressed_backprop_amd import ops
    g = gen("inside", m, v)
    n = m * v
    room = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    z = room[3:n + 3].view(m, v)  # (its gradient elsewhere has another alignment)
    z.copy_(randn(g, m, v, dtype=dtype))
    t = torch.randint(0, v, (m,), generator=g).cuda()
    out = check_forward(z, t, 3)
    gs = randn(g, m), None, randn(g, m)
    apart = check_backward(z, t, out, *gs)
    inside = ops.token_logprobs_backward(z, t, out.stats, *gs, out.entropy, in_place=True)
    assert torch.equal(bits(inside), bits(apart)) and bool((room[:3] == 7.0).all() and (room[n + 3:] == 7.0).all())
    dst = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    s = ops.instant_logprobs_bwd(apart, t, 8, m, v, v, int(dtype == BF), -100, out.stats, out.entropy, gs[0], None,
                                 gs[2], dst)
    assert s == 0 and bool((dst[n:] == 7.0).all())
    held = [torch.full((m * w + 32,), 7.0, device="cuda") for w in (1, 1, 1, 2, 3)]
    idx = torch.full((m * 3 + 32,), 7, device="cuda")
    need = ops.instant_logprobs_workspace_bytes(m, v, int(dtype == BF), 3)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    s = ops.instant_logprobs_fwd(apart, t, 8, m, v, v, int(dtype == BF), -100, 3, *held, idx, ws, need)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 7).all())
    assert s == 0 and all(bool((h[m * w:] == 7.0).all()) for h, w in zip(held, (1, 1, 1, 2, 3)))
    assert bool((idx[m * 3:] == 7).all())


def test_logprobs_gradient_against_differences():
    """d/dz of a weighted sum of logp, lse and H by central differences of the 64-bit definition."""
    from rank_compressed_backprop_amd.loss import token_logprobs
    g = gen("fd")
    z = randn(g, 3, 11).requires_grad_(True)
    t = torch.tensor([4, -100, 10]).cuda()
    a, b, c = (randn(g, 3) for _ in range(3))
    out = token_logprobs(z, t, top=2)
    (out.logp * a + out.lse * b + out.entropy * c).sum().backward()

    def f(x):
        logp, lse, H, *_ = logprobs64(x, t)
        return (logp * a + lse * b + H * c).sum()
    h, x = 1e-5, z.detach().double()
    for i in range(3):
        for j in range(11):
            d = torch.zeros_like(x)
            d[i, j] = h
            # (central differences: third derivatives below 50 times h^2 / 6; rounding 2^-52 40 / h)
            assert abs(((f(x + d) - f(x - d)) / (2 * h) - z.grad[i, j]).item()) < 3e-6


# ------------------------------------------------------------------------- embedding

def embed_back64(gy, t, V, scale, padding):
    """(gradient, sums of the terms' magnitudes, terms) of each row."""
    keep = (t >= 0) & (t < V)
    if padding is not None:
        keep &= t != padding
    rows, tok = gy[keep].double(), t[keep].long()
    ref = torch.zeros(V, gy.shape[1], dtype=torch.float64, device="cuda").index_add_(0, tok, rows)
    mag = torch.zeros_like(ref).index_add_(0, tok, rows.abs())
    n = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, tok, torch.ones_like(tok, dtype=torch.float64))
    return ref * scale, mag * abs(scale), n


def check_embed_back(gy, t, V, scale, padding, into=None):
    from rank_compressed_backprop_amd import ops
    C = gy.shape[-1]
    ref, mag, n = embed_back64(gy.view(-1, C), t.flatten(), V, scale, padding)
    before = None if into is None else into.clone()
    got = ops.embedding_backward(gy, t, V, scale, padding, into)
    bound = u * (n[:, None] + 2) * mag
    if into is not None:
        assert got is into
        ref = ref + before.double()
        assert torch.equal(bits(got[n == 0]), bits(before[n == 0]))
    else:
        assert not got[n == 0].any()
    within("gtable", got, ref, bound + (U[gy.dtype] + u) * ref.abs() + 2.0 ** -133)
    again = ops.embedding_backward(gy, t, V, scale, padding, None if into is None else before)
    assert torch.equal(bits(again), bits(got))
    return got


EMBED_SHAPES = [(1, 1, 8), (1, 1000, 64), (2, 3, 8), (8, 128000, 512), (31, 50, 136), (32, 7, 64), (33, 5, 72),
                (100, 1, 128), (1000, 30522, 768), (4095, 97, 264), (4096, 4096, 64), (4097, 300, 2056),
                (9000, 262144, 8), (16384, 32000, 128), (20000, 2, 40),
                (1024, 5000, 16), (1025, 1025, 24), (2049, 262144, 8)]


@DTYPES
@pytest.mark.parametrize("shape", EMBED_SHAPES, ids=str)
def test_embedding(shape, dtype):
    from rank_compressed_backprop_amd import ops
    m, V, C = shape
    print(f"[embed] {shape} {dtype}", flush=True)
    g = gen("emb", shape)
    w = randn(g, V, C, dtype=dtype)
    t = (torch.rand(m, generator=g) ** 3 * V).long().clamp(max=V - 1).cuda()
    for scale, tok in ((1.0, t), (C ** 0.5, t.int()), (-0.37, t)):
        y = ops.embedding_forward(tok, w, scale)
        ref = w[t].double() * scale
        if scale == 1.0:
            assert torch.equal(bits(y), bits(w[t]))
        within("y", y, ref, (U[dtype] + 2 * u) * ref.abs() + 2.0 ** -133)
    gy = randn(g, m, C, dtype=dtype)
    check_embed_back(gy, t, V, 1.0, None)
    check_embed_back(gy, t.int(), V, C ** 0.5, 0)
    check_embed_back(gy, t, V, -0.37, V - 1, randn(g, V, C, dtype=dtype))


@DTYPES
def test_embedding_tokens_outside(dtype):
    """A token outside the vocabulary gives NaN forward, and takes no part backward."""
    from rank_compressed_backprop_amd import ops
    g = gen("out")
    V, C = 50, 64
    w, gy = randn(g, V, C, dtype=dtype), randn(g, 6, C, dtype=dtype)
    t = torch.tensor([0, -1, 49, 50, 1 << 40, -(1 << 62)]).cuda()
    y = ops.embedding_forward(t, w)
    assert torch.equal(y[[0, 2]], w[[0, 49]]) and y[[1, 3, 4, 5]].isnan().all()
    gw = check_embed_back(gy, t, V, 1.0, None)
    assert torch.equal(gw[0], gy[0]) and torch.equal(gw[49], gy[2]) and int((gw != 0).any(1).sum()) == 2
    t32 = torch.tensor([0, -1, 49, 50, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    assert torch.equal(ops.embedding_forward(t32, w).isnan(), y.isnan())
    gy[[1, 3, 4, 5]] = NAN  # what takes no part may hold anything
    assert not check_embed_back(gy, t32, V, 1.0, None).isnan().any()


@DTYPES
@pytest.mark.parametrize("m", [64, 5000, 70000])
def test_embedding_gradient_of_runs(m, dtype):
    """One token throughout, runs that end at the borders of the kernel's tiles, all padding."""
    g = gen("runs", m)
    C, V = 72, 40
    gy = randn(g, m, C, dtype=dtype)
    i = torch.arange(m).cuda()
    for name, t in (("one", i * 0 + 7), ("tiles", (i // 32) % V), ("halves", (i // 16) % V), ("two", (i >= m - 33).long()),
                    ("odd", (i // 31) % V), ("turns", i % V)):
        print(f"[runs] {m} {name}", flush=True)
        check_embed_back(gy, t, V, 1.0, None)
    check_embed_back(gy, i * 0 + 3, V, 1.0, 3)
    check_embed_back(gy, i * 0 + 3, V, 1.0, 3, randn(g, V, C, dtype=dtype))


def test_embedding_gradient_against_differences():
    from rank_compressed_backprop_amd.embedding import InstantEmbedding
    g = gen("efd")
    e = InstantEmbedding(7, 8, scale=1.5, padding=2, dtype="fp32")
    t = torch.tensor([[1, 2, 1], [6, 0, 1]]).cuda()
    a = randn(g, 2, 3, 8)
    (e(t) * a).sum().backward()
    x = e.weight.detach().double()
    keep = (t != 2)[..., None]

    def f(w):
        return (1.5 * w[t] * a * keep).sum()
    for i in range(7):
        d = torch.zeros_like(x)
        d[i, 3] = 1.0  # (linear in the table: differences are exact but for rounding)
        assert abs((f(x + d) - f(x - d)).item() / 2 - e.weight.grad[i, 3].item()) < 1e-5


# ------------------------------------------------------------------------- norm and clipping

def mixture(g, sizes, kinds):
    return [randn(g, *s, dtype=d) for s, d in zip(sizes, kinds)]


def check_clip(ts, max_norm, outs=None):
    """outs: types of other outputs, or None (in place)."""
    from rank_compressed_backprop_amd import ops
    ref = sum((t.double().square().sum() for t in ts), torch.zeros((), dtype=torch.float64, device="cuda")).sqrt()
    before = [t.clone() for t in ts]
    norm = ops.grad_norm(ts)
    within("norm", norm, ref, 2.0 ** -23 * ref)
    out = None if outs is None else [torch.full_like(t, 7.0, dtype=d) for t, d in zip(ts, outs)]
    n2 = ops.clip_grads(ts, max_norm, out)
    assert torch.equal(norm, n2) and norm.dtype == FP and norm.shape == ()
    c = torch.where(norm + 1e-6 <= max_norm, 1.0, max_norm / (norm.double() + 1e-6))
    for b, t, o in zip(before, ts, ts if out is None else out):
        want = b.double() * c
        if c == 1:
            assert torch.equal(o, b.to(o.dtype))
        within(f"out {tuple(b.shape)}", o, want, (U[o.dtype] + 4 * u) * want.abs() + 2.0 ** -133)
        if out is not None:
            assert torch.equal(bits(t), bits(b))


CLIP_LISTS = {
    "one": ([(1,)], [FP]),
    "mixed": ([(3, 5), (1,), (0,), (64, 64), (7,), (1000, 33), (8,), (40000,)], [FP, BF, BF, BF, BF, FP, BF, FP]),
    "pieces": ([(32768,), (32769,), (32767,), (3, 65537)], [BF, FP, BF, BF]),
    "many": ([(1 + i % 37, 1 + i % 11) for i in range(300)], [(BF, FP)[i % 3 == 0] for i in range(300)]),
    "large": ([(4096, 5000), (11, 7)], [BF, BF]),
    "empty": ([(0,), (0, 5)], [BF, FP]),
}


@pytest.mark.parametrize("name", CLIP_LISTS)
def test_clip(name):
    print(f"[clip] {name}", flush=True)
    sizes, kinds = CLIP_LISTS[name]
    for max_norm in (0.5, 1e9, INF, 0.0):
        for outs in (None, [FP] * len(sizes), [BF] * len(sizes), kinds):
            check_clip(mixture(gen("clip", name), sizes, kinds), max_norm, outs)


def test_clip_at_odd_places():
    """Tensors that start anywhere, next to others, which stay as they are; outputs of another
    alignment than their gradients."""
    from rank_compressed_backprop_amd import ops
    g = gen("odd")
    for dtype in (BF, FP):
        for k in range(1, 9):
            a, b = randn(g, 5000, dtype=dtype), torch.full((5000,), 7.0, dtype=dtype, device="cuda")
            t, keep = a[k:k + 4001 + k], a.clone()
            for to in (b[2 * k + 1:2 * k + 4002 + k], t):
                c = 0.5 / (t.double().square().sum().sqrt() + 1e-6)
                want = t.double() * c
                ops.clip_grads([t], 0.5, [to])
                within(f"{k}", to, want, (U[dtype] + 4 * u) * want.abs())
            assert torch.equal(a[:k], keep[:k]) and torch.equal(a[4001 + 2 * k:], keep[4001 + 2 * k:])
            assert bool((b[:2 * k + 1] == 7).all()) and bool((b[4002 + 3 * k:] == 7).all())


def test_norm_extremes():
    """Values whose squares leave float32's range, and what is not finite."""
    from rank_compressed_backprop_amd import ops
    for v in (1e30, 1e-30, 2.0 ** -140, 3e38):
        t = torch.full((4,), v, device="cuda")
        want = torch.tensor(v, dtype=FP).double() * 2
        got = ops.grad_norm([t]).double().cpu()
        assert got == INF if v == 3e38 else abs(got - want) <= 2.0 ** -23 * want + 2.0 ** -149
    t = torch.tensor([1.0, NAN, 2.0], device="cuda")
    assert ops.clip_grads([t], 1.0).isnan() and t.isnan().all()
    t = torch.tensor([1.0, INF, -2.0], device="cuda")
    assert ops.clip_grads([t], 1.0) == INF
    assert t[0] == 0 and t[1].isnan() and t[2] == 0
    t = torch.zeros(5, device="cuda")
    assert ops.clip_grads([t], 1.0) == 0 and not t.any()


def test_clip_grad_norm_of_parameters():
    from rank_compressed_backprop_amd.clip import clip_grad_norm_
    g = gen("params")
    ps = [torch.nn.Parameter(randn(g, 30, 17, dtype=d)) for d in (BF, FP, FP)] + [torch.nn.Parameter(randn(g, 4))]
    for p in ps[:3]:
        p.grad = randn(g, 30, 17, dtype=p.dtype)
    before = [p.grad.clone() for p in ps[:3]]
    ref = torch.stack([b.double().square().sum() for b in before]).sum().sqrt()
    norm = clip_grad_norm_(ps + [ps[0]], 2.0)  # one is listed twice
    within("norm", norm, ref, 2.0 ** -23 * ref)
    for p, b in zip(ps, before):
        want = b.double() * 2.0 / (ref + 1e-6)
        within("grad", p.grad, want, (U[p.dtype] + 6 * u) * want.abs())
    assert ps[3].grad is None
    assert clip_grad_norm_([ps[3]], 1.0) == 0 and clip_grad_norm_([], 1.0) == 0
    clip_grad_norm_(ps[1], 1e-3)


# ------------------------------------------------------------------------- all of them

def test_no_rows():
    from rank_compressed_backprop_amd import ops
    t = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    w = torch.ones(5, 8, device="cuda")
    assert ops.embedding_forward(t, w).shape == (0, 3, 8)
    gw = ops.embedding_backward(torch.zeros(0, 3, 8, device="cuda"), t, 5)
    assert gw.shape == (5, 8) and not gw.any()
    assert torch.equal(ops.embedding_backward(torch.zeros(0, 3, 8, device="cuda"), t, 5, into=w), torch.ones_like(w))
    z = torch.zeros(0, 3, 9, device="cuda")
    out = ops.token_logprobs(z, t, top=2)
    assert out.logp.shape == (0, 3) and out.top_index.shape == (0, 3, 2)
    assert ops.token_logprobs_backward(z, t, out.stats, out.logp).shape == z.shape
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Logits and a table of more than 2^31 elements (and 2^32 bytes)."""
    print("[offsets]", flush=True)
    from rank_compressed_backprop_amd import ops
    g = gen("far")
    m, v = 16500, 131071
    assert m * v > 1 << 31
    z = torch.zeros(m, v, dtype=BF, device="cuda")
    z[-2:] = randn(g, 2, v, dtype=BF)
    t = torch.randint(0, v, (m,), generator=g).cuda()
    out = ops.token_logprobs(z, t, top=4)
    # (the same rows alone are summed in another order, so they are held to the reference, not to bits)
    tail = check_forward(z[-2:], t[-2:], 4, out=ops.TokenLogprobs(*(x[-2:] for x in out)))
    gr = torch.ones(m, device="cuda")
    gz = ops.token_logprobs_backward(z, t, out.stats, gr)
    check_backward(z[-2:], t[-2:], tail, gr[-2:], None, None, gz=gz[-2:])
    del z, gz
    V, C = 262144, 8256
    assert V * C > 1 << 31
    w = torch.zeros(V, C, dtype=BF, device="cuda")
    w[-1] = 3.0
    tok = torch.tensor([V - 1, 0, V - 1]).cuda()
    y = ops.embedding_forward(tok, w, 2.0)
    assert bool((y[[0, 2]] == 6.0).all()) and not y[1].any()
    gw = ops.embedding_backward(y, tok, V, into=w)
    assert bool((gw[-1] == 15.0).all()) and not gw[-2].any()
    del gw, w
    flat = torch.ones((1 << 31) + 5, dtype=BF, device="cuda")
    norm = ops.clip_grads([flat], 1.0)
    assert abs(norm.item() - ((1 << 31) + 5) ** 0.5) < 0.01
    assert bool((flat[-5:] == flat[0]).all()) and flat[0] < 1e-4


def run_all(ops, s):
    """Every operator once: a step's ends on a small table."""
    y = ops.embedding_forward(s["t"], s["w"], 2.0)
    out = ops.token_logprobs(s["z"], s["t"], top=3)
    gz = ops.token_logprobs_backward(s["z"], s["t"], out.stats, s["g"], None, s["g"], out.entropy)
    gw = ops.embedding_backward(s["gy"], s["t"], s["w"].shape[0], 2.0, 0)
    to = [torch.empty_like(gw), torch.empty_like(gz, dtype=FP)]
    return [y, *out, gz, gw, *to, ops.clip_grads([gw, gz], 0.1, to)]


def some(dtype, m=700, v=1001, c=136):
    g = gen("some", m, v, c)
    return {"t": torch.randint(0, v, (m,), generator=g).cuda(), "w": randn(g, v, c, dtype=dtype),
            "z": randn(g, m, v, dtype=dtype), "g": randn(g, m), "gy": randn(g, m, c, dtype=dtype)}


@DTYPES
@pytest.mark.parametrize("m", [9, 5000])
def test_captured_and_replayed(m, dtype):
    """A graph of all of them: every replay, with other inputs and eager work between, gives the
    eager call's bits; two graphs and an eager call at once on streams of their own too."""
    from rank_compressed_backprop_amd import ops
    print(f"[graph] {m} {dtype}", flush=True)
    states = [some(dtype, m, v) for v in (1001, 1000)]
    graphs, outs = [], []
    for s in states:
        run_all(ops, s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run_all(ops, s))
        graphs.append(gr)
    for r in range(4):
        for s in states:
            gen2 = gen("again", r)
            for k in ("z", "g", "gy"):
                s[k].copy_(randn(gen2, *s[k].shape, dtype=s[k].dtype))
            s["t"].copy_(torch.randint(0, 1000, (m,), generator=gen2).cuda())
        want = [run_all(ops, s) for s in states]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for gr, st, o in zip(graphs, streams, outs):
            for x in o:
                x.fill_(7)
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                gr.replay()
        eager = run_all(ops, states[0])
        torch.cuda.synchronize()
        for o, w in zip(outs + [eager], want + [want[0]]):
            for i, (a, b) in enumerate(zip(o, w)):
                assert torch.equal(bits(a), bits(b)), (r, i)


def test_layers_on_another_stream():
    from rank_compressed_backprop_amd import ops
    s = some(BF)
    want = run_all(ops, s)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = run_all(ops, s)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))


def test_layers_refuse_second_derivatives_and_bad_arguments():
    from rank_compressed_backprop_amd import InstantError, ops
    from rank_compressed_backprop_amd.embedding import InstantEmbedding
    from rank_compressed_backprop_amd.loss import token_logprobs
    e = InstantEmbedding(16, 8, dtype="fp32")
    t = torch.arange(4).cuda()
    with pytest.raises(RuntimeError, match="differentiated again"):
        torch.autograd.grad(e(t).square().sum(), e.weight, create_graph=True)
    z = torch.randn(4, 16, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        torch.autograd.grad(token_logprobs(z, t).logp.sum(), z, create_graph=True)
    x = z.detach()
    for call in (lambda: ops.token_logprobs(x, t.cpu()), lambda: ops.token_logprobs(x, t[:3]),
                 lambda: ops.token_logprobs(x, t, top=17), lambda: ops.token_logprobs(x, t, vocab=17),
                 lambda: ops.token_logprobs(x.t(), t), lambda: ops.embedding_forward(t.cpu(), x),
                 lambda: ops.embedding_backward(x, t, 0), lambda: ops.embedding_backward(x, t, 4, padding=4),
                 lambda: ops.clip_grads([x, x.cpu()], 1.0), lambda: ops.clip_grads([x], -1.0),
                 lambda: ops.clip_grads([x], NAN), lambda: ops.clip_grads([x], 1.0, [x[:2]]),
                 lambda: ops.grad_norm([x.t()]), lambda: ops.grad_norm([])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.token_logprobs(x, t.float()), lambda: ops.token_logprobs(x.half(), t),
                 lambda: ops.embedding_forward(t.short(), x), lambda: ops.grad_norm(x),
                 lambda: ops.grad_norm([x, None])):
        with pytest.raises(TypeError):
            call()
    y = torch.zeros(64, device="cuda")
    for ts, out in (([y, y], None), ([y[:32], y[16:]], None), ([y[:32]], [y[16:48]]),
                    ([y[:8], y[32:40]], [y[32:40], y[40:48]])):
        with pytest.raises(InstantError):  # outputs that share memory
            ops.clip_grads(ts, 1.0, out)
    assert ops.grad_norm([y, y]) == 0
    w = torch.zeros(16, 8, device="cuda")
    with pytest.raises(InstantError):  # a gradient that is added to itself
        ops.embedding_backward(w, torch.arange(16).cuda(), 16, into=w)


def test_alternatives_take_no_gradient():
    from rank_compressed_backprop_amd.loss import token_logprobs
    z = torch.randn(4, 16, device="cuda", requires_grad=True)
    out = token_logprobs(z, torch.arange(4).cuda(), top=3)
    assert out.logp.requires_grad and out.lse.requires_grad and out.entropy.requires_grad
    assert not (out.top_logp.requires_grad or out.top_index.requires_grad or out.stats.requires_grad)
    with pytest.raises(RuntimeError):
        out.top_logp.sum().backward()


@pytest.mark.parametrize("tied", [False, True])
def test_a_training_step(tied):
    """Tokens to clipped gradients, as they are used together: embedding, norm, a layer of the
    library, norm, product with the vocabulary, log probabilities, backward, clipping; against
    autograd in 64 bits. float32: sums of at most 200 terms in three products, each within 1e-5."""
    from rank_compressed_backprop_amd.clip import clip_grad_norm_
    from rank_compressed_backprop_amd.embedding import InstantEmbedding
    from rank_compressed_backprop_amd.linear import InstantLinear
    from rank_compressed_backprop_amd.loss import token_logprobs
    from rank_compressed_backprop_amd.norm import InstantRMSNorm
    print(f"[step] tied {tied}", flush=True)
    g = gen("step")
    B, L, C, V, Vp = 2, 64, 64, 187, 192
    emb = InstantEmbedding(Vp, C, scale=C ** 0.5, padding=0, dtype="fp32", weight=randn(g, Vp, C, sd=0.1))
    norm1, norm2 = (InstantRMSNorm(C, dtype="fp32") for _ in range(2))
    mid = InstantLinear(L, C, C, B, N_t=4, N_cal=2, dtype="fp32", weight=randn(g, C, C, sd=C ** -0.5), bias=True,
                        activation="gelu")
    head = InstantLinear(L, C, Vp, B, N_t=4, N_cal=2, dtype="fp32", weight=randn(g, Vp, C, sd=C ** -0.5), bias=True)
    if tied:
        head.weight = emb.weight
    t = torch.randint(0, V, (B, L), generator=g).cuda()
    t[1, 40:] = 0
    want = torch.roll(t, -1, 1)
    want[1, 39:] = -100

    def loss_of(out):
        n = (want != -100).sum()
        return -out.logp.sum() / n + 1e-3 * out.lse.square().mean() - 0.01 * out.entropy.mean()
    x = emb(t)
    h = mid(norm1(x), residual=x)
    out = token_logprobs(head(norm2(h)), want, vocab=V, top=5)
    loss_of(out).backward()
    ps = list({id(p): p for m in (emb, norm1, mid, norm2, head) for p in m.parameters()}.values())
    grads = [p.grad.clone() for p in ps]
    norm = clip_grad_norm_(ps, 0.1)

    d = {id(p): p.detach().double().requires_grad_(True) for p in ps}
    rms = lambda v, w: v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    w = d[id(emb.weight)]
    x = torch.where((t == 0)[..., None], w[t].detach(), w[t]) * C ** 0.5
    z = rms(x, d[id(norm1.weight)]) @ d[id(mid.weight)].t() + d[id(mid.bias)]
    h = x + 0.5 * z * (1 + torch.erf(z / 2 ** 0.5))
    zz = (rms(h, d[id(norm2.weight)]) @ d[id(head.weight)].t() + d[id(head.bias)])[..., :V]
    lse = torch.logsumexp(zz, -1)
    lp = zz - lse[..., None]
    import types
    o64 = types.SimpleNamespace(logp=torch.where(want == -100, 0.0, lp.gather(-1, want.clamp(min=0)[..., None])[..., 0]),
                                lse=lse, entropy=-(lp.exp() * lp).sum(-1))
    for k in ("logp", "lse", "entropy"):
        assert ((getattr(out, k).double() - getattr(o64, k)).abs() <= 1e-4).all(), k
    assert torch.equal(out.top_index[..., 0], zz.argmax(-1))
    ref = torch.autograd.grad(loss_of(o64), [d[id(p)] for p in ps])
    total = torch.sqrt(sum(r.square().sum() for r in ref))
    assert abs(norm.double() - total) <= 1e-5 * total
    for p, got, r in zip(ps, grads, ref):
        assert (got.double() - r).norm() <= 3e-5 * r.norm() + 1e-9, tuple(p.shape)
        assert (p.grad.double() - r * 0.1 / (total + 1e-6)).norm() <= 4e-5 * r.norm() * 0.1 / total + 1e-9


@pytest.mark.parametrize("given", ["parameter", "layer"])
def test_a_tied_step_through_the_constructors(given):
    """One Parameter handed to both ends, or one end's weight to the other: one leaf with the sum of
    both gradients, one norm, one step of the optimizer. (float32 sums of at most 192 terms: 1e-5.)"""
    from rank_compressed_backprop_amd.clip import clip_grad_norm_
    from rank_compressed_backprop_amd.embedding import InstantEmbedding
    from rank_compressed_backprop_amd.linear import InstantLinear
    from rank_compressed_backprop_amd.loss import token_logprobs
    print(f"[tied] {given}", flush=True)
    g = gen("tied", given)
    B, L, C, V = 2, 64, 64, 192
    w = torch.nn.Parameter(randn(g, V, C, sd=0.3))
    emb = InstantEmbedding(V, C, scale=2.0, dtype="fp32", weight=w if given == "parameter" else w.detach())
    head = InstantLinear(L, C, V, B, N_t=4, N_cal=2, dtype="fp32", weight=w if given == "parameter" else emb.weight,
                         bias=True)
    assert head.weight is emb.weight and (emb.weight is w) == (given == "parameter")
    t = torch.randint(0, V, (B, L), generator=g).cuda()
    want = torch.randint(0, V, (B, L), generator=g).cuda()
    (-token_logprobs(head(emb(t)), want).logp.mean()).backward()
    d = w.detach().double().requires_grad_(True)
    lp = (2 * d[t] @ d.t()).log_softmax(-1).gather(-1, want[..., None])
    (ref,) = torch.autograd.grad(-lp.mean(), d)
    assert (emb.weight.grad.double() - ref).norm() <= 1e-5 * ref.norm()
    ps = [emb.weight, head.weight]
    norm = clip_grad_norm_(ps, 0.01)
    assert abs(norm.double() - ref.norm()) <= 1e-5 * ref.norm()
    before, step = emb.weight.detach().clone(), emb.weight.grad.clone()
    torch.optim.SGD({id(p): p for p in ps}.values(), lr=0.5).step()
    assert torch.equal(emb.weight.detach(), torch.add(before, step, alpha=-0.5))


def test_autograd_sees_what_is_written_in_place():
    """A backward pass that has saved what a call overwrote raises, as with torch's own in-place
    operations; a tensor that is only read, or whose call is refused, stays as it was."""
    from rank_compressed_backprop_amd import ops
    from rank_compressed_backprop_amd.clip import clip_grad_norm_
    from rank_compressed_backprop_amd.loss import token_logprobs
    g = gen("version")
    t = torch.arange(4).cuda()
    z = randn(g, 4, 16).requires_grad_(True) * 2
    out = token_logprobs(z, t)
    ops.token_logprobs_backward(z, t, out.stats, torch.ones(4, device="cuda"))
    out.logp.sum().backward(retain_graph=True)  # nothing was written
    ops.token_logprobs_backward(z, t, out.stats, torch.ones(4, device="cuda"), in_place=True)
    with pytest.raises(RuntimeError, match="inplace operation"):
        out.logp.sum().backward()

    def saved(write, read=None):
        """Whether a product that has saved buf refuses its backward pass after write(buf)."""
        buf, w = randn(g, 4, 16), torch.ones(4, 16, device="cuda", requires_grad=True)
        loss = (w * buf).sum()
        write(buf)
        try:
            loss.backward()
        except RuntimeError as e:
            assert "inplace operation" in str(e)
            return True
        assert torch.equal(w.grad, buf)
        return False

    def by_parameter(buf):
        p = torch.nn.Parameter(torch.zeros_like(buf))
        p.grad = buf
        clip_grad_norm_(p, 0.1)

    def refused(buf):
        with pytest.raises(ops.InstantError):
            ops.clip_grads([buf, buf], 0.1)
    other = randn(g, 4, 16)
    for write in (lambda b: ops.embedding_backward(other, t, 4, into=b), lambda b: ops.clip_grads([b], 0.1),
                  lambda b: ops.clip_grads([other], 0.1, [b]), lambda b: ops.clip_grads([other, b[1], b[2:]], 0.1),
                  by_parameter):
        assert saved(write)
    for write in (lambda b: ops.embedding_backward(b, t, 4, into=other), lambda b: ops.grad_norm([b]), refused,
                  lambda b: ops.clip_grads([b], 0.1, [other]), lambda b: ops.embedding_backward(b, t, 4)):
        assert not saved(write)
    with torch.inference_mode():  # (tensors without a version)
        b = randn(g, 4, 16)
        assert ops.clip_grads([b], 0.1) > 0 and b.norm() <= 0.1001
        ops.embedding_backward(b, t, 4, into=b * 0)


def test_logits_gradient_in_place_through_a_product():
    """Without the loss's layer: the gradient is written over the logits and goes on into the product
    that made them. (float32 sums of 24 and 40 terms: 1e-5.)"""
    from rank_compressed_backprop_amd import ops
    g = gen("through")
    x, w = randn(g, 40, 24).requires_grad_(True), randn(g, 56, 24).requires_grad_(True)
    t = torch.randint(0, 56, (40,), generator=g).cuda()
    z = torch.nn.functional.linear(x, w)
    out = ops.token_logprobs(z, t)
    gz = ops.token_logprobs_backward(z, t, out.stats, torch.full((40,), -1 / 40, device="cuda"), in_place=True)
    assert gz is z
    z.backward(gz.detach())
    x64, w64 = (v.detach().double().requires_grad_(True) for v in (x, w))
    ref = torch.autograd.grad(torch.nn.functional.cross_entropy(x64 @ w64.t(), t), (x64, w64))
    for got, r in zip((x.grad, w.grad), ref):
        assert (got.double() - r).norm() <= 1e-5 * r.norm()
