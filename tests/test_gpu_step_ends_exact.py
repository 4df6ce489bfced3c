"""GPU tests of the operators at a training step's ends on inputs whose sums are exact in float32,
whatever their order: one term that is lost or counted twice shows, wherever it stands.

Embedding's gradient. Gradients are integers of magnitude 1 to 4, so every partial sum is an integer
below 2^24: the table's gradient is the 64-bit sum, in float32 to the bit and in bfloat16 rounded once.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_step_ends import DTYPES, FP, bits, gen  # noqa: E402


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
