"""The gated scan against its fp64 oracle where its sums and products are long:
memories of two thousand steps, the sums of db over many items, more items than
CTAs; and its fp32 sigmoids over their whole range."""
import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import gated

from test_gpu_gated import BF, F32, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
def test_long_memories(function, dtype):
    """The carried state and the gradient of the initial state, fp32 for either
    dtype, in channels that remember 2 to 2000 steps; inputs and gradients of one
    sign, so that an error to one side adds up.

    Tolerance: a step rounds 1 + e, f and the sum that f enters, each by at most
    2^-24 relative to either side alike: a standard deviation of 2^-24 together.
    Over a memory of M = 2000 steps they add up with the weights f^k, whose
    squares sum to M / 2: sqrt(1000) 2^-24 = 1.9e-6 of the state, and 1.2e-5 is six
    of them. An error to one side adds up to M of it: an eighth of 2^-23 on
    average would show."""
    B, T, D = 1, 12000, 72
    p = make(function, B, T, 1, D, dtype)
    f = 1 if function == "linear" else 0
    p["Wx"][:, :, f] *= 0.25
    for x in (p["Wx"][:, :, f + 1], p["state"], p["dh"], p["dlast"]):
        x.abs_()
    p["b"][f + 1] = 0
    tau = torch.logspace(np.log10(2), np.log10(2000), D)
    p["b"][f, 0] = torch.log(tau - 1).to(dtype).cuda()
    _, last, _, _, ds = run(p, function)
    _, rlast, before = gated.fwd(p["Wx"], p["b"], p["state"], function)
    _, _, rds = gated.bwd(p["Wx"], p["b"], before, function, p["dh"], p["dlast"])
    for got, ref, what in ((last, rlast, "last"), (ds, rds, "dstate")):
        worst = np.abs(got.detach().double().cpu().numpy() - ref).max() / np.abs(ref).max()
        print(function, dtype, what, worst)
        assert worst <= 1.2e-5, (what, worst)


# (B, T, N, D) and what it reaches: sums of db by a launch of their own (more than
# 64 items a tile of channels, on either side of the limit; more than 8 rows of
# one chunk); several items to a CTA, with TMA's rows and with others
SUMS = [(40, 260, 1, 40), (32, 256, 1, 24), (33, 256, 1, 24), (12, 100, 1, 33), (9, 64, 2, 16), (66, 129, 1, 17)]
MANY = [(24, 520, 1, 600), (24, 520, 1, 601)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("shape", SUMS, ids=lambda s: "B%dT%dN%dD%d" % s)
def test_sums_over_many_items(shape, function, dtype):
    check(make(function, *shape, dtype), function)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "B%dT%dN%dD%d" % s)
def test_more_items_than_blocks(shape, function, dtype):
    check(make(function, *shape, dtype), function)


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_many_items_with_masks(checkpoint):
    B, T, N, D = 24, 520, 1, 600
    p = make("linear", B, T, N, D, BF)
    g = torch.Generator().manual_seed(1)
    reset = torch.rand(B, T, generator=g) < 0.01
    lengths = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    check(p, "linear", reset.cuda(), lengths.cuda(), checkpoint)


def test_fp32_sigmoids_over_their_range():
    """Every sigmoid of the fp32 kernels, and 1 - sigmoid of the coupled cell, read
    off single steps. Tolerance: the base-2 exponential and the product of its
    argument's parts are good to 2^-22, the sum 1 + e and the reciprocal with its
    Newton step to 2^-23 each: 2^-21 relative, and below the normal numbers their
    smallest, 2^-126."""
    z = torch.cat([torch.linspace(-88, 88, 1 << 16), torch.linspace(-1e-3, 1e-3, 1001),
                   torch.tensor([-1e30, -1000.0, -104.0, -88.5, 0.0, 88.5, 104.0, 1000.0, 1e30])])
    n = z.numel()
    want = gated.sigmoid(z.double().numpy())
    rest = gated.sigmoid(-z.double().numpy())
    inf, zero, one = torch.full_like(z, float("inf")), torch.zeros_like(z), torch.ones_like(z)

    def step(function, gates, state):
        Wx = torch.stack(gates).reshape(1, 1, len(gates), 1, n).cuda()
        h, last = rn.gated_scan(Wx, None, state.reshape(1, 1, 1, n).cuda(), function=function)
        pool = state.reshape(1, 1, n).cuda()
        h1 = rn.gated_scan_step(Wx[:, 0], None, pool, function=function)
        assert torch.equal(h1, h[:, 0]) and torch.equal(pool, last[:, 0])
        return h.reshape(-1).double().cpu().numpy(), last.reshape(-1).double().cpu().numpy()

    def near(got, ref, what):
        worst = (np.maximum(np.abs(got - ref) - 2.0 ** -126, 0) / np.maximum(ref, 2.0 ** -1000)).max()
        print(what, np.log2(max(worst, 1e-30)))
        assert np.isfinite(got).all() and worst <= 2.0 ** -21, (what, worst)

    near(step("linear", [-inf, z, one, inf], one)[1], want, "f")
    near(step("linear", [z, -inf, one, inf], zero)[1], want, "i")
    near(step("linear", [-inf, inf, one, z], one)[0], want, "o")
    near(step("linear_coupled", [z, zero], one)[1], want, "coupled f")
    near(step("linear_coupled", [z, one], zero)[1], rest, "coupled 1 - f")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_saturated_coupled_gate(dtype):
    """Logits of +-infinity and of the type's lowest value: f exactly 0 or 1."""
    for low in (float("-inf"), torch.finfo(dtype).min):
        for f, want in ((low, 0.0), (-low, 3e38)):
            Wx = torch.zeros(1, 300, 2, 1, 64, dtype=dtype, device="cuda")
            Wx[:, :, 0] = f
            h, last = rn.gated_scan(Wx, None, torch.full((1, 1, 1, 64), 3e38, device="cuda"), function="linear_coupled")
            assert (last == torch.tensor(want, device="cuda")).all() and (h == torch.tensor(want).to(dtype).cuda()).all()
