"""GPU tests of the operators at a training step's ends on inputs whose sums are exact in float32,
whatever their order: one term that is lost or counted twice shows, wherever it stands.

Embedding's gradient. Gradients are integers of magnitude 1 to 4, so every partial sum is an integer
below 2^24: the table's gradient is the 64-bit sum, in float32 to the bit and in bfloat16 rounded once.

Log probabilities. Rows hold n zeros among -inf (or among -200, whose exponential is 0 in float32 and
adds less than V e^-200 to S): the exponentials are 1 and 0, S = n < 2^24 and E = 0 exactly. lse and the
entropy are ln 2 log2(n), of which the logarithm is off by at most 1 ulp, 2 u of itself, float32's ln 2 by
u / 16 and the product by u: 4 u log n holds them. One term of n changes log n by 1 / n at least, more than
4 u log n for every n up to 2^18. A row with a single zero has lse and entropy 0 exactly.

Random rows are held to a bound from the additions that a term passes: at most 32 in a step, one for each
of the thread's K steps and 40 in the joins of lanes, waves and slices, u each; each of the K + 40 raises of
the maximum multiplies by an exponential of its own (4 u), and exponents, and the raises' distances, which
add up to the range D at most, are off by 6 u D together. A thread of T (16 up to 128 chunks of CE values, 64
up to 4096, else 256) has n = V / T + 2 CE terms in steps of 16 at least, and at most 10 steps that are
shorter (behind the last whole one, and at the row's ends); one of 1024 has a step for each chunk,
V / 1024 / CE + 2. The logarithm and its product are off by 4 u of themselves, each difference by u.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_step_ends import BF, DTYPES, FP, INF, bits, gen, logprobs64, randn, u, within  # noqa: E402


# ------------------------------------------------------------------------- embedding

def integers(g, *shape, most=4):
    """Integers of magnitude 1 to most."""
    v = torch.randint(1, most + 1, shape, generator=g, dtype=torch.int8)
    return v * (2 * torch.randint(0, 2, shape, generator=g, dtype=torch.int8) - 1)


def check_exact(g, t, V, C, dtype, padding=None, most=4):
    """Dense and added to a gradient; scales are powers of two, which are exact too."""
    from rank_compressed_backprop_amd import ops
    gy = integers(g, len(t), C, most=most).cuda().to(dtype)
    keep = (t >= 0) & (t < V)
    if padding is not None:
        keep &= t != padding
    ref = torch.zeros(V, C, dtype=torch.float64, device="cuda").index_add_(0, t[keep].long(), gy[keep].double())
    got = ops.embedding_backward(gy, t, V, 1.0, padding)
    assert torch.equal(bits(got), bits(ref.to(dtype) + 0.0))  # (no sum is -0: a run's begins with 0)
    held = integers(g, V, C).cuda().to(dtype)
    got = ops.embedding_backward(gy, t, V, 0.5, padding, into=held.clone())
    hit = torch.zeros(V, dtype=torch.bool, device="cuda").index_fill_(0, t[keep].long(), True)
    assert torch.equal(got[~hit], held[~hit])
    want = (held.double() + 0.5 * ref).to(dtype)
    assert torch.equal(got[hit], want[hit])


@DTYPES
@pytest.mark.parametrize("m", [1, 8, 64, 65, 1024, 1025, 5000, 70000])
def test_embedding_gradient_of_integers_in_runs(m, dtype):
    """Runs that end at and beside the borders of eights, waves' rows, tiles, segments and rounds."""
    g = gen("exact runs", m)
    C, V = 72, 40
    i = torch.arange(m).cuda()
    runs = {"one": i * 0 + 7, "turns": i % V, "two": (i >= m - 33).long()}
    runs |= {f"runs of {n}": (i // n) % V for n in (7, 8, 9, 31, 32, 63, 64, 65, 127, 512, 1024, 4096, 4097)}
    for name, t in runs.items():
        print(f"[exact runs] {m} {name}", flush=True)
        check_exact(g, t, V, C, dtype)
    check_exact(g, i % 3, V, C, dtype, padding=1)


@DTYPES
@pytest.mark.parametrize("shape", [(20000, 2, 40), (1000, 30522, 768), (16384, 32000, 128), (4097, 300, 2056),
                                   (262144, 700, 8), (262145, 40000, 8), (300000, 5, 8), (300000, 262144, 8)], ids=str)
def test_embedding_gradient_of_integers(shape, dtype):
    m, V, C = shape
    print(f"[exact] {shape} {dtype}", flush=True)
    g = gen("exact", shape)
    t = (torch.rand(m, generator=g) ** 3 * V).long().clamp(max=V - 1).cuda()
    check_exact(g, t, V, C, dtype)
    check_exact(g, t.int(), V, C, dtype, padding=0)


@pytest.mark.parametrize("m", [5000, 70000, 300000])
def test_embedding_gradient_of_integers_in_one_class(m):
    """Tokens that are equal modulo 1024: one block orders all of them, in several rounds."""
    print(f"[exact class] {m}", flush=True)
    g = gen("class", m)
    i = torch.arange(m).cuda()
    for t in (7 + 1024 * (i % 256), 1023 + 1024 * (i * 256 // m), 1024 * torch.randint(0, 256, (m,), generator=g).cuda()):
        check_exact(g, t, 1 << 18, 8, FP)


def test_embedding_gradient_of_most_tokens():
    """2^22 tokens, the most that are accepted: one throughout, and random ones."""
    g = gen("most")
    m = 1 << 22
    for t, V in ((torch.full((m,), 3), 5), (torch.randint(0, 1500, (m,), generator=g), 1500)):
        print(f"[exact most] {V}", flush=True)
        check_exact(g, t.cuda(), V, 8, FP, most=1)


# ------------------------------------------------------------------------- log probabilities

# sizes for each way through the rows: few lanes a row, a wave, a block of 256 or 1024, slices
WAYS = [(5, 1), (5, 2), (3, 7), (40, 33), (300, 255), (65, 511), (65, 512), (65, 513), (7, 1000), (7, 1024), (7, 1025),
        (9, 2047), (300, 4095), (300, 4097), (2050, 4099), (2050, 8191), (2049, 8193), (2049, 15997), (2048, 16385),
        (300, 16387), (200, 20001), (3, 8200), (3, 32767), (130, 66000), (1, 32768), (1, 65536), (1, 131071), (5, 100003),
        (64, 128000), (128, 65539), (128, 128009), (300, 131071), (1, 262144), (64, 262143), (200, 262144)]


@DTYPES
@pytest.mark.parametrize("m,v", WAYS)
@pytest.mark.parametrize("top", [0, 1, 5])
def test_logprobs_count_every_logit(m, v, top, dtype):
    """Rows of zeros, and of n zeros among -inf or -200."""
    from rank_compressed_backprop_amd import ops
    print(f"[count] {m} {v} {top} {dtype}", flush=True)
    top = min(top, v)
    g = torch.Generator(device="cuda").manual_seed(m * 7 + v)
    full = torch.zeros(m, v, dtype=dtype, device="cuda")
    share = torch.rand(m, 1, generator=g, device="cuda")
    on = torch.rand(m, v, generator=g, device="cuda") < share
    on[torch.arange(m), torch.arange(m) * 977 % v] = True
    for z in (full, full.masked_fill(~on, -INF), full.masked_fill(~on, -200.0)):
        n = (z == 0).sum(1)
        t = (z == 0).int().argmax(1)
        out = ops.token_logprobs(z, t, top=top)
        want = n.double().log()
        assert not out.stats[:, 0].any()
        for name, got in (("log sum", out.stats[:, 1]), ("lse", out.lse), ("entropy", out.entropy), ("logp", -out.logp)):
            within(name, got, want, 4 * u * want)
        if top:
            place = torch.arange(v, dtype=torch.int32, device="cuda")
            order = torch.topk(torch.where(z == 0, place, v + place), top, largest=False).values % v
            assert torch.equal(out.top_index, order.long())
            assert torch.equal(out.top_logp[:, 0], out.logp)


def borders(v, wide):
    """Places at the ends, beside multiples of 1024 (what a block or a wave's step ends at) and beside the
    borders of 2 to 16 slices; all of a short row."""
    if v <= 2100:
        return torch.arange(v)
    at = [0, v, *range(0, v, 1024 if v < 40000 else 4096), *(v * i // n for n in (2, 3, 4, 5, 8, 16) for i in range(n))]
    near = torch.tensor(sorted(set(at)))[:, None] + torch.arange(-wide, wide + 1)
    return torch.unique(near[(near >= 0) & (near < v)])


@DTYPES
@pytest.mark.parametrize("m,v", WAYS)
def test_logprobs_find_a_single_logit(m, v, dtype):
    """Rows of -inf but for one zero, at every border in turn: lse and entropy are 0, it is the target and the
    likeliest, and the others follow by their place."""
    from rank_compressed_backprop_amd import ops
    print(f"[single] {m} {v} {dtype}", flush=True)
    places = borders(v, 9 if m > 4 else 4).cuda()
    z = torch.full((m, v), -INF, dtype=dtype, device="cuda")
    rows = torch.arange(m, device="cuda")
    for b in range(0, len(places), m):
        j = places[torch.arange(b, b + m, device="cuda") % len(places)]
        z[rows, j] = 0.0
        for top in sorted({0, 1, min(2, v)}):
            out = ops.token_logprobs(z, j, top=top)
            assert not (out.lse.any() or out.entropy.any() or out.logp.any() or out.stats.any())
            if top:
                assert torch.equal(out.top_index[:, 0], j) and not out.top_logp[:, 0].any()
            if top == 2:
                assert torch.equal(out.top_index[:, 1], (j == 0).long()) and bool((out.top_logp[:, 1] == -INF).all())
        z[rows, j] = -INF


def chain(v, dtype, D):
    """Relative to S (or E), for random rows (see above)."""
    CE = 8 if dtype == BF else 4
    chunks = v // CE + 2
    T = 16 if chunks <= 130 else 64 if chunks <= 4098 else 256
    K = max((v / T + 2 * CE) / 16 + 10, v / 1024 / CE + 2)
    return u * (6 * D + 32 + K + 40 + 4 * (K + 40) + 10)


@DTYPES
@pytest.mark.parametrize("m,v", WAYS)
def test_logprobs_of_random_rows(m, v, dtype):
    from rank_compressed_backprop_amd import ops
    print(f"[random] {m} {v} {dtype}", flush=True)
    g = gen("chain", m, v)
    z = randn(g, m, v, dtype=dtype, sd=3.0)
    t = torch.randint(0, v, (m,), generator=g).cuda()
    out = ops.token_logprobs(z, t)
    for a in range(0, m, 256):  # (the reference in parts)
        s = slice(a, a + 256)
        logp, lse, H, *_ = logprobs64(z[s], t[s])
        top, low = z[s].double().amax(1), z[s].double().amin(1)
        rel, ls = chain(v, dtype, (top - low).clamp(max=104)), lse - top
        within("log sum", out.stats[s, 1], ls, rel + 4 * u * ls)
        within("lse", out.lse[s], lse, rel + 4 * u * ls + u * lse.abs())
        within("logp", out.logp[s], logp, rel + 4 * u * ls + 2 * u * logp.abs())
        within("entropy", out.entropy[s], H, rel + 4 * u * ls + (2 * rel + 4 * u) * (ls - H).abs() + 2 * u * H)
