"""The operators at a training step's ends (include/instant_ops.h), without a GPU: what a call may not
be is refused on the host before anything is enqueued, and workspaces are what the sizes need."""
import random

import pytest

torch = pytest.importorskip("torch")

import rank_compressed_backprop_amd as rcb  # noqa: E402
from rank_compressed_backprop_amd import ops  # noqa: E402

A, W, FAR = 0x1000, 0x2000, 1 << 44  # pointers that are never read: every call here is refused, or has no rows
E_ARG, E_SHAPE, OK = rcb.INSTANT_E_ARG, rcb.INSTANT_E_SHAPE, rcb.INSTANT_OK
BF, FP = rcb.INSTANT_BF16, rcb.INSTANT_FP32
INF, NAN = float("inf"), float("nan")


def embed_fwd(tokens=A, size=8, M=4, table=A, V=50, C=64, dtype=BF, scale=1.0, y=A):
    return ops.instant_embed_fwd(tokens, size, M, table, V, C, dtype, scale, y, 0)


def embed_bwd(gy=A, tokens=A, size=8, M=4, V=50, C=64, dtype=BF, scale=1.0, padding=-1, add=0, gt=FAR, ws=W, n=1 << 40):
    return ops.instant_embed_bwd(gy, tokens, size, M, V, C, dtype, scale, padding, add, gt, ws, n, 0)


def test_embed_refusals():
    for change in [dict(tokens=None), dict(table=None), dict(y=None), dict(size=2), dict(tokens=A + 4), dict(size=0),
                   dict(size=4, tokens=A + 2), dict(table=A + 8), dict(y=A + 8), dict(M=-1), dict(V=0), dict(C=0),
                   dict(dtype=2), dict(scale=INF), dict(scale=NAN)]:
        assert embed_fwd(**change) == E_ARG, change
    for change in [dict(C=12), dict(V=(1 << 18) + 1), dict(M=(1 << 26) + 1), dict(C=(1 << 18) + 8)]:
        assert embed_fwd(**change) == E_SHAPE, change
    assert embed_fwd(M=0, tokens=None, table=None, y=None) == OK
    for change in [dict(gy=None), dict(tokens=None), dict(gt=None), dict(size=3), dict(tokens=A + 1), dict(gy=A + 2),
                   dict(gt=FAR + 8), dict(gt=A), dict(gt=A + 496), dict(gy=FAR + 6384), dict(M=-1), dict(V=0), dict(C=-8), dict(dtype=9), dict(scale=INF), dict(padding=-2),
                   dict(ws=None), dict(ws=W + 64)]:
        assert embed_bwd(**change) == E_ARG, change
    for change in [dict(C=20), dict(M=(1 << 22) + 1), dict(M=1 << 22, C=1 << 17), dict(V=(1 << 18) + 8), dict(n=16)]:
        assert embed_bwd(**change) == E_SHAPE, change
    assert embed_bwd(M=0, add=1, gy=None, tokens=None, ws=None, n=0) == OK  # nothing to add


def lp_fwd(z=A, t=A, size=8, M=4, W_=100, V=100, dtype=BF, k=0, logp=A, lse=A, ent=A, stats=A, tl=None, ti=None, ws=W,
           n=1 << 30):
    return ops.instant_logprobs_fwd(z, t, size, M, W_, V, dtype, -100, k, logp, lse, ent, stats, tl, ti, ws, n, 0)


def lp_bwd(z=A, t=A, size=8, M=4, W_=100, V=100, dtype=BF, stats=A, ent=None, g=A, gl=None, gh=None, gz=A):
    return ops.instant_logprobs_bwd(z, t, size, M, W_, V, dtype, -100, stats, ent, g, gl, gh, gz, 0)


def test_logprobs_refusals():
    for change in [dict(z=None), dict(z=A + 1), dict(z=A + 2, dtype=FP), dict(t=None), dict(logp=None),
                   dict(t=None, logp=None, lse=None, ent=None, stats=None), dict(size=1), dict(t=A + 4), dict(M=-1),
                   dict(V=0), dict(V=101), dict(dtype=3), dict(lse=A + 2), dict(k=-1), dict(k=2), dict(k=2, tl=A),
                   dict(k=2, ti=A), dict(tl=A), dict(k=2, tl=A, ti=A + 4), dict(k=2, tl=A + 2, ti=A)]:
        assert lp_fwd(**change) == E_ARG, change
    for change in [dict(k=33, tl=A, ti=A), dict(V=3, k=4, tl=A, ti=A), dict(W_=(1 << 18) + 1), dict(M=(1 << 26) + 1)]:
        assert lp_fwd(**change) == E_SHAPE, change
    assert lp_fwd(M=0, z=None, t=None, logp=None, ws=None, n=0) == OK
    big = dict(M=4, W_=200000, V=200000)
    need = ops.instant_logprobs_workspace_bytes(4, 200000, BF, 0)
    assert need > 0
    assert lp_fwd(**big, ws=None) == E_ARG and lp_fwd(**big, ws=W + 8) == E_ARG and lp_fwd(**big, n=need - 1) == E_SHAPE
    for change in [dict(z=None), dict(stats=None), dict(gz=None), dict(g=None), dict(t=None), dict(gh=A), dict(z=A + 1),
                   dict(gz=A + 1), dict(gz=A + 2, dtype=FP), dict(size=16), dict(g=A + 1), dict(stats=A + 2),
                   dict(V=0), dict(V=200), dict(M=-4), dict(dtype=-1)]:
        assert lp_bwd(**change) == E_ARG, change
    assert lp_bwd(W_=1 << 19) == E_SHAPE
    assert lp_bwd(M=0, z=None, gz=None, stats=None) == OK


def test_logprobs_workspace_sizes():
    for bad in [(-1, 8, BF, 0), (4, 0, BF, 0), (4, 1 << 19, BF, 0), (4, 8, 5, 0), (4, 8, BF, -1), (4, 100, BF, 33),
                (4, 8, BF, 9), ((1 << 26) + 1, 8, BF, 0)]:
        assert ops.instant_logprobs_workspace_bytes(*bad) == 0, bad
    rng = random.Random(3)
    for _ in range(2000):
        M, V = int(2 ** rng.uniform(0, 26)), int(2 ** rng.uniform(5, 18))
        n = ops.instant_logprobs_workspace_bytes(M, V, rng.choice([BF, FP]), rng.randrange(33))
        assert n % 4 == 0 and n < 1 << 20  # only few rows are split
    for bad in [(-1, 8, 8), (4, 0, 8), (4, 8, 12), ((1 << 22) + 1, 8, 8), (1 << 22, 8, 1 << 17)]:
        assert ops.instant_embed_workspace_bytes(*bad) == 0, bad
    for bad in (-1, (1 << 20) + 1):
        assert ops.instant_grad_norm_workspace_bytes(bad) == 0
    assert ops.instant_grad_norm_workspace_bytes(0) > 0


def norm(g=(A,), count=(8,), dtype=(FP,), n=None, out=A, ws=W, size=1 << 30):
    return ops.instant_grad_norm(g, count, dtype, len(g) if n is None else n, out, ws, size, 0)


def clip(g=(A,), count=(8,), dtype=(FP,), out=(A,), out_dtype=(FP,), n=None, max_norm=1.0, norm=A, ws=W, size=1 << 30):
    return ops.instant_clip_grads(g, count, dtype, out, out_dtype, len(g) if n is None else n, max_norm, norm, ws, size, 0)


def test_clip_refusals():
    for change in [dict(g=(None,)), dict(g=(A + 2,)), dict(count=(-1,)), dict(dtype=(2,)), dict(n=-1), dict(out=None),
                   dict(out=A + 2), dict(ws=None), dict(ws=W + 8), dict(g=None, n=1), dict(count=None), dict(dtype=None)]:
        assert norm(**change) == E_ARG, change
    for change in [dict(count=((1 << 40) + 1,)), dict(size=8), dict(n=(1 << 20) + 1)]:
        assert norm(**change) == E_SHAPE, change
    for change in [dict(out=(None,)), dict(out=(A + 2,)), dict(out_dtype=(7,)), dict(max_norm=-1.0), dict(max_norm=NAN),
                   dict(norm=None), dict(norm=A + 1), dict(ws=None), dict(out=None), dict(out_dtype=None)]:
        assert clip(**change) == E_ARG, change
    # outputs that share memory: with each other, with another gradient, in place in another type
    for change in [dict(g=(A, A), count=(8, 8), dtype=(FP, FP), out=(A, A), out_dtype=(FP, FP)),
                   dict(g=(A, A + 64), count=(8, 8), dtype=(FP, FP), out=(0x9000, 0x9010), out_dtype=(FP, FP)),
                   dict(g=(A, A + 32), count=(8, 8), dtype=(FP, FP), out=(A + 16, 0x9000), out_dtype=(FP, FP)),
                   dict(out=(A + 16,)), dict(out_dtype=(BF,)), dict(g=(A + 16,), dtype=(BF,), out=(A,)),
                   dict(g=(A, 0x8000, A), count=(8, 8, 8), dtype=(FP,) * 3, out=(A, 0x8000, 0x9000), out_dtype=(FP,) * 3)]:
        assert clip(**change) == E_ARG, change
    assert clip(size=8) == E_SHAPE


def test_tensor_functions_refuse_on_the_cpu():
    """Types and shapes are checked before the device, so no GPU is asked."""
    x, t = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ops.embedding_forward(t, x), lambda: ops.embedding_forward(t, torch.zeros(4, 12)),
                 lambda: ops.embedding_forward(t, x, scale=INF), lambda: ops.embedding_forward(t, x, scale=1e39),
                 lambda: ops.embedding_forward(t, x.t()), lambda: ops.embedding_forward(t[::2], x),
                 lambda: ops.embedding_forward(t, x[0]), lambda: ops.embedding_backward(x, t, 10),
                 lambda: ops.token_logprobs(x, t), lambda: ops.token_logprobs(x.t()),
                 lambda: ops.token_logprobs(x, vocab=17), lambda: ops.token_logprobs(x, vocab=0),
                 lambda: ops.token_logprobs(torch.zeros(2, 0)), lambda: ops.token_logprobs(torch.tensor(0.0)),
                 lambda: ops.token_logprobs_backward(x, t, torch.zeros(4, 2), g_logp=torch.zeros(4)),
                 lambda: ops.grad_norm([]), lambda: ops.grad_norm([x]), lambda: ops.clip_grads([], 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.embedding_forward(None, x), lambda: ops.embedding_forward(t.float(), x),
                 lambda: ops.embedding_forward(t, None), lambda: ops.embedding_forward(t, x.half()),
                 lambda: ops.token_logprobs(None), lambda: ops.token_logprobs(x.double()), lambda: ops.grad_norm(x),
                 lambda: ops.grad_norm([None]), lambda: ops.clip_grads([x.half()], 1.0), lambda: ops.clip_grads(x, 1.0)):
        with pytest.raises(TypeError):
            call()


def test_layer_refuses_other_sizes():
    from rank_compressed_backprop_amd.embedding import InstantEmbedding
    for bad in [dict(V=0), dict(V=(1 << 18) + 1), dict(C=12), dict(C=0), dict(dtype="fp16"), dict(padding=50),
                dict(padding=-1), dict(weight=torch.zeros(50, 8))]:
        with pytest.raises(ValueError):
            InstantEmbedding(**(dict(V=50, C=16, device="cpu") | bad))
    e = InstantEmbedding(50, 16, padding=3, device="cpu")
    assert e.weight.dtype == torch.bfloat16 and not e.weight[3].any() and e.weight[4].any()


def test_clip_of_no_gradients():
    from rank_compressed_backprop_amd.clip import clip_grad_norm_
    p = torch.nn.Parameter(torch.ones(3))
    assert clip_grad_norm_(p, 1.0) == 0 and clip_grad_norm_([], 1.0) == 0 and p.grad is None


def test_second_derivatives_are_refused(monkeypatch):
    """Plain forms stand in for the kernels here."""
    from rank_compressed_backprop_amd.embedding import _EmbeddingFn
    from rank_compressed_backprop_amd.loss import token_logprobs
    monkeypatch.setattr(ops, "embedding_forward", lambda t, w, s: w[t] * s)
    monkeypatch.setattr(ops, "embedding_backward", lambda gy, t, V, s, p: torch.zeros(V, gy.shape[1]).index_add(0, t, gy))
    monkeypatch.setattr(ops, "token_logprobs", lambda z, t, v, k, i: ops.TokenLogprobs(
        z.log_softmax(1)[torch.arange(len(t)), t], z.logsumexp(1), z.sum(1), None, None, z[:, :2].clone()))
    monkeypatch.setattr(ops, "token_logprobs_backward", lambda z, *a, **k: z * 0)
    w, z = torch.ones(5, 8, requires_grad=True), torch.ones(3, 5, requires_grad=True)
    t = torch.tensor([1, 0, 4])
    for leaf, call in ((w, lambda: _EmbeddingFn.apply(t, w, 1.0, None)), (z, lambda: token_logprobs(z, t).logp)):
        torch.autograd.grad(call().sum(), leaf)
        for loss in (call().square().sum(), call().sum()):
            with pytest.raises(RuntimeError, match="differentiated again"):
                torch.autograd.grad(loss, leaf, create_graph=True)


@pytest.fixture
def layers(monkeypatch):
    """(make, rows, columns) of the layers that take a weight, without a GPU."""
    from rank_compressed_backprop_amd import embedding, linear
    monkeypatch.setattr(linear, "InstantLayer", lambda *a, **k: None)
    return [lambda w, **k: embedding.InstantEmbedding(50, 16, dtype="fp32", weight=w, device="cpu", **k),
            lambda w, **k: linear.InstantLinear(8, 16, 50, 2, dtype="fp32", weight=w, device="cpu", **k)]


def test_a_parameter_is_tied_by_the_constructors(layers):
    """One Parameter handed to both layers is one leaf, with one gradient that both add to."""
    w = torch.nn.Parameter(torch.randn(50, 16))
    made = [make(w) for make in layers]
    assert all(m.weight is w for m in made)
    assert len({id(p) for m in made for p in m.parameters()}) == 1
    (made[0].weight.sum() + 2 * made[1].weight.sum()).backward()
    assert torch.equal(w.grad, torch.full_like(w, 3.0))
    for make, first in zip(layers, reversed(layers)):  # one layer's weight handed to the other
        made = first(None)
        assert make(made.weight).weight is made.weight
    frozen = torch.nn.Parameter(torch.randn(50, 16), requires_grad=False)
    assert all(make(frozen).weight is frozen for make in layers)


def test_two_parameters_never_share_memory(layers):
    """What is not a Parameter of the layer's type, device and layout is copied."""
    base = torch.randn(50, 16)
    others = [base, base.clone().requires_grad_(True), base.bfloat16(), torch.nn.Parameter(base.double()),
              torch.nn.Parameter(base.t().contiguous().t()), torch.randn(100, 16)[::2], torch.randn(60, 16)[5:55]]
    for make in layers:
        for w in others:
            before = w.detach().clone()
            made = make(w).weight
            assert isinstance(made, torch.nn.Parameter) and made.requires_grad and made.is_leaf
            assert made.is_contiguous() and made.dtype == torch.float32 and torch.equal(made, before.float())
            assert made.untyped_storage().data_ptr() != w.untyped_storage().data_ptr()
            assert made.untyped_storage().nbytes() == 50 * 16 * 4
            with torch.no_grad():
                made.zero_()
            assert torch.equal(w.detach(), before)


def test_padding_row_of_a_given_weight(layers):
    """Zeros stand in the padding token's row of a weight that the layer makes; a given one is kept."""
    w = torch.nn.Parameter(torch.ones(50, 16))
    assert layers[0](w, padding=3).weight[3].all() and not layers[0](None, padding=3).weight[3].any()


def test_gradient_that_overlaps_its_logits():
    """In place is the same address; any other overlap is refused, also where both are aligned."""
    for d in (16, 32, 64, 784, 796, 798):  # (4 rows of 100 in bfloat16 are 800 bytes)
        assert lp_bwd(z=FAR, gz=FAR + d) == E_ARG and lp_bwd(z=FAR + d, gz=FAR) == E_ARG, d
    for d in (4, 800, 1596):
        assert lp_bwd(z=FAR, gz=FAR + d, dtype=FP) == E_ARG and lp_bwd(z=FAR + d, gz=FAR, dtype=FP) == E_ARG, d
