"""Host logic of the training-step integration: which kind of step each training step is
(notes "INSTANT: ...", 整体框架: calibration every N_t steps, compression in between)."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


def _modes(N_t, N_cal, generation, steps):
    from rank_compressed_backprop_amd.linear import InstantLinear
    fake = SimpleNamespace(N_t=N_t, N_cal=N_cal, generation=generation)
    return [InstantLinear.mode_of_step(fake, s) for s in range(steps)]


def test_window_schedule():
    assert _modes(5, 2, 1, 10) == ["calibrate", "finalize", "compress", "compress", "compress"] * 2
    assert _modes(4, 1, 3, 8) == ["finalize", "compress", "compress", "compress"] * 2
    # N_cal = N_t: every step calibrates, the last of each window finalizes
    assert _modes(3, 3, 1, 6) == ["calibrate", "calibrate", "finalize"] * 2


def test_no_projections_yet_means_exact_backward():
    assert _modes(5, 2, 0, 5) == ["calibrate", "finalize", "exact", "exact", "exact"]


def _bare_layer(**kw):
    """An InstantLinear without its library handle and its device."""
    from rank_compressed_backprop_amd.linear import InstantLinear
    mod = InstantLinear.__new__(InstantLinear)
    torch.nn.Module.__init__(mod)
    mod.L, mod.Cx, mod.Cy, mod.B_max, mod.N_t, mod.N_cal, mod.step, mod.generation = 4, 8, 8, 2, 5, 2, 0, 0
    mod.torch_dtype, mod.activation, mod.checkpoint, mod.bias = torch.float32, "none", None, None
    mod.weight = torch.nn.Parameter(torch.zeros(8, 8))
    for k, v in kw.items():
        setattr(mod, k, v)
    return mod


@pytest.mark.parametrize("plain", [False, True])
def test_a_refused_call_is_no_step_of_the_schedule(plain):
    """A call whose arguments are refused ran nothing: the next one has its place in the window
    (the step that finalizes among them)."""
    mod = _bare_layer() if plain else _bare_layer(activation="gelu")
    mod.step = 1
    x = torch.zeros(2, 4, 8)
    if plain:
        mod.weight = torch.nn.Parameter(torch.zeros(8, 8, dtype=torch.float64))  # (not the input's type)
        with pytest.raises(RuntimeError):
            mod(x)
    else:
        with pytest.raises(ValueError):
            mod(x, residual=torch.zeros(2, 4, 16))  # (as are tensors on the CPU)
    assert mod.step == 1 and mod.mode_of_step(mod.step) == "finalize"


def test_x8_is_checked_in_the_forward():
    """A checkpoint that does not fit x is refused by the call it is given to, not by the backward
    pass of a step that has run."""
    from rank_compressed_backprop_amd import ops
    x = torch.zeros(2, 4, 8)
    q, s = torch.zeros(2, 4, 8, dtype=torch.int8), torch.zeros(2, 4, 1, dtype=torch.uint8)
    for exc, x8 in [(ValueError, ops.Checkpoint8(q[:1], s)), (ValueError, ops.Checkpoint8(q, s[:1])),
                    (TypeError, ops.Checkpoint8(q.float(), s)), (TypeError, ops.Checkpoint8(q, s.to(torch.int8))),
                    (ValueError, ops.Checkpoint8(q.transpose(0, 1).contiguous().transpose(0, 1), s)),
                    (TypeError, q), (TypeError, (q, s))]:
        mod = _bare_layer(checkpoint="int8")
        with pytest.raises(exc, match="x8"):
            mod(x, x8=x8)
    with pytest.raises(ValueError, match="x8"):
        _bare_layer(activation="gelu")(x, x8=ops.Checkpoint8(q, s))
