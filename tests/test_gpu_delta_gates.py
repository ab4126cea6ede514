"""dg where states are forgotten quickly. dg_t is a_t times a product of the state
before the step and of a gradient, so it becomes small with a_t, and has to keep its
digits: the step's own part of o and of dY, which is not small, is not in it.

Tolerances (L2, over steps of one decay). A sum of products of signed terms has the
terms' relative error, taken as independent, at the sum's own size. fp32: as in
test_gpu_delta.py, and 2^-24 |g| by the rounded exponent: 2^-24 (64 + T / 4 + 3 |g|).
bf16: operands in two bf16 planes, 2^-17 of a value at most (dY, Z, S0, dS1, M or R):
five of them, below 2^-14."""
import pytest
import torch

from test_gpu_delta import BF, F32, make, oracle, run

pytestmark = pytest.mark.gpu

SHAPES = [(1, 200, 1, 2, 40, 48), (2, 130, 2, 4, 128, 128), (1, 100, 1, 1, 200, 72), (1, 2500, 1, 1, 32, 32), (1, 150, 1, 1, 17, 9)]


def off(got, ref):
    assert torch.isfinite(got).all()
    return ((got.double().cpu() - ref).norm() / ref.norm()).item()


def limit(dtype, T, g):
    return 2.0 ** -14 if dtype == BF else 2.0 ** -24 * (64 + T / 4 + 3 * abs(g))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_one_decay(shape, dtype):
    p = make(*shape, dtype, seed=41)
    for g in (-0.1, -0.5, -2.0, -5.0, -10.0, -20.0, -50.0):
        p["g"] = torch.full_like(p["g"], g)
        e = off(run(p)[5], torch.as_tensor(oracle(p)[5]))
        assert e <= limit(dtype, shape[1], g), f"g {g}: {e:.3g}"


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_decays_of_all_sizes(shape, dtype):
    """Long memories with a cut here and there, around the ends of chunks among them, and resets."""
    p = make(*shape, dtype, seed=42)
    B, T, N = p["g"].shape
    gen = torch.Generator().manual_seed(T)
    sizes = torch.tensor([-0.001, -0.02, -0.3, -3.0, -12.0, -40.0])
    pick = torch.multinomial(torch.tensor([0.55, 0.35, 0.04, 0.02, 0.02, 0.02]), B * T * N, True, generator=gen).view(B, T, N)
    for t in (0, 31, 32, 63, 64, 65, 96):
        pick[:, t] = 3 + t % 3
    p["g"] = sizes[pick].cuda()
    reset = torch.rand(B, T, generator=gen) < 0.01
    got, ref = run(p, reset.cuda())[5], torch.as_tensor(oracle(p, reset)[5])
    assert (got[reset.cuda()] == 0).all()
    for k in range(3, 6):
        at = (pick == k) & ~reset[..., None]
        e = off(got[at.cuda()], ref[at])
        assert e <= limit(dtype, T, sizes[k].item()), f"g {sizes[k]}: {e:.3g}"


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_ragged_rows(dtype):
    """Rows of several lengths, whatever stands past them, on a long axis too."""
    for shape in ((4, 150, 1, 2, 40, 48), (2, 2500, 1, 1, 32, 32)):
        p = make(*shape, dtype, seed=43)
        B, T = shape[:2]
        p["g"] = 12 * p["g"] - 2
        lengths = torch.tensor([T - 13, 70, 0, 1][:B], dtype=torch.int32)
        ref = torch.as_tensor(oracle(p, None, lengths)[5])
        for i in range(B):
            for name in ("q", "k", "v", "g", "beta", "do"):
                p[name][i, int(lengths[i]):] = float("nan")
        got = run(p, None, lengths.cuda())[5]
        for i, n in enumerate(lengths.tolist()):
            assert (got[i, n:] == 0).all()
        assert off(got, ref) <= limit(dtype, T, -2.0)
