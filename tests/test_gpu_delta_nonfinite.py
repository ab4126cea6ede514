"""A reset takes the state before it as zero, whatever it holds, wherever in a
chunk or a segment it stands: the documents behind it give the bits that they give
after a finite state, and the one before it is not made finite. Backward, nothing
of the last state's gradient comes to the documents before the last. Columns of v
do not see one another's states."""
import pytest
import torch

from test_gpu_delta import BF, F32, NAMES, make, run

pytestmark = pytest.mark.gpu

BAD = [float("inf"), float("-inf"), float("nan")]
# a reset around the ends of a chunk (32 steps of fp32, 64 of bf16), and one in a
# later segment of a long axis
CASES = [((2, 150, 1, 1, 40, 48), at) for at in (1, 31, 32, 37, 63, 64, 65, 127, 149)]
CASES += [((1, 100, 2, 4, 136, 20), 37), ((1, 2500, 1, 1, 64, 64), 1300), ((1, 2500, 1, 1, 144, 40), 1301)]


def marks(shape, *at):
    reset = torch.zeros(shape[:2], dtype=torch.bool, device="cuda")
    reset[:, list(at)] = True
    return reset


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,at", CASES, ids=lambda x: str(x) if isinstance(x, int) else "B%dT%dNk%dN%dDk%dDv%d" % x)
def test_state_ahead_of_a_reset(shape, at, dtype):
    p = make(*shape, dtype, seed=21)
    reset = marks(shape, at, min(at + 20, shape[1] - 1))
    ref = dict(zip(NAMES, run(p, reset)))
    for bad in BAD:
        got = dict(zip(NAMES, run(dict(p, state=torch.full_like(p["state"], bad)), reset)))
        assert torch.equal(got["last"], ref["last"]) and torch.equal(got["dstate"], ref["dstate"])
        assert torch.equal(got["dv"], ref["dv"])  # the gradient's state is finite, whatever the state is
        for name in ("o", "dq", "dk", "dg", "dbeta"):
            assert torch.equal(got[name][:, at:], ref[name][:, at:]), name
            assert not torch.isfinite(got[name][:, :at]).any(), name
        o, last = run(dict(p, state=torch.full_like(p["state"], bad)), reset, grads=False)
        clean, clean_last = run(p, reset, grads=False)
        assert torch.equal(last, clean_last) and torch.equal(o[:, at:], clean[:, at:])
        assert not torch.isfinite(o[:, :at]).any()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_columns_keep_to_themselves(dtype):
    """One element of the state: its column of v alone, in o and in the state, until the reset."""
    shape, at = (1, 150, 1, 2, 40, 48), 70
    p = make(*shape, dtype, seed=22)
    state = p["state"].clone()
    state[0, 0, 1, 3, 7] = float("inf")
    for reset in (marks(shape, at), None):
        (o, last), (clean, clean_last) = (run(x, reset, grads=False) for x in (dict(p, state=state), p))
        end = at if reset is not None else 150
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[:, :end, 1, 7] = True
        assert torch.equal(o[~hit], clean[~hit]) and not torch.isfinite(o[hit]).any()
        hit = torch.zeros_like(last, dtype=torch.bool)
        hit[..., 1, :, 7] = reset is None
        assert torch.equal(last[~hit], clean_last[~hit]) and not torch.isfinite(last[hit]).any()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decays_that_end_in_zero(dtype):
    """An infinite state whose decays' product is below the smallest number while the
    document goes on: its steps in that chunk stay what they are, not finite."""
    p = make(1, 64, 1, 1, 32, 32, dtype, seed=23)
    p["g"] = torch.full_like(p["g"], -20.0)
    reset = marks((1, 64), 20)
    ref = run(p, reset)
    got = run(dict(p, state=torch.full_like(p["state"], float("inf"))), reset)
    got, ref = dict(zip(NAMES, got)), dict(zip(NAMES, ref))
    for name in ("o", "dq", "dk", "dg", "dbeta"):
        assert not torch.isfinite(got[name][:, :20]).any(), name
        assert torch.equal(got[name][:, 20:], ref[name][:, 20:]), name
    assert torch.equal(got["last"], ref["last"])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,at", CASES, ids=lambda x: str(x) if isinstance(x, int) else "B%dT%dNk%dN%dDk%dDv%d" % x)
def test_gradient_behind_a_reset(shape, at, dtype):
    p = make(*shape, dtype, seed=24)
    reset = marks(shape, max(at - 20, 0), at)
    ref = dict(zip(NAMES, run(p, reset)))
    for bad in BAD:
        got = dict(zip(NAMES, run(dict(p, dlast=torch.full_like(p["dlast"], bad)), reset)))
        for name in ("o", "last", "dstate", "dq"):
            assert torch.equal(got[name], ref[name]), name
        for name in ("dk", "dv", "dg", "dbeta"):
            assert torch.equal(got[name][:, :at], ref[name][:, :at]), name
        for name in ("dk", "dv", "dbeta"):
            assert not torch.isfinite(got[name][:, at:]).any(), name
        assert torch.isfinite(got["dg"][:, at]).all()  # a reset's own step has no decay
        assert not torch.isfinite(got["dg"][:, at + 1:]).any()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_steps_past_a_length(dtype):
    """o and the gradients there are zero, whatever the state and its gradient hold."""
    for T in (150, 2500):
        p = make(2, T, 1, 1, 40, 48, dtype, seed=25)
        lengths = torch.tensor([T - 13, 70], dtype=torch.int32, device="cuda")
        for name in ("state", "dlast"):
            for bad in BAD:
                got = dict(zip(NAMES, run(dict(p, **{name: torch.full_like(p[name], bad)}), lengths=lengths)))
                for out in ("o", "dq", "dk", "dv", "dg", "dbeta"):
                    for i, n in enumerate(lengths.tolist()):
                        assert (got[out][i, n:] == 0).all(), (name, out)
