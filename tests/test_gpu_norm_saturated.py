"""Slopes of saturated activations: element by element against the 64-bit oracle.

Tolerances. A slope is a product of exp(-|x|) and reciprocals of 1 + exp(-|x|),
none of which cancels. The exponential's argument is rounded: 2^-24 |x|, 2^-18 at
the |x| <= 64 here. fp32: 2^-18 and a few roundings of 2^-24, below 2^-17. bf16:
approximations of 2^-21 besides, and the result's own rounding by 2^-8 at most
(plus products rounded in fp32): 2^-8 (1 + 2^-6). silu's slope s + x s (1 - s) is a sum
that cancels around x = -1.28: only |x| >= 4 is looked at, where its terms differ by
a factor of 3 or more (1 - 4 * 0.98: 2.9), so that errors grow by less than 2."""
import pytest
import torch

import recurrent_networks_gb300 as rn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def slopes(x, act):
    """act'(x) in 64 bits."""
    x = x.double()
    s = torch.sigmoid(x)
    c = torch.sigmoid(x) * torch.sigmoid(-x)
    return c if act == "sigmoid" else s + x * c


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_slopes_of_shut_and_open_gates(act, dtype):
    for width in (64, 1000, 5000):
        at = torch.cat([torch.linspace(4, 64, 200), -torch.linspace(4, 64, 200)])
        z = at.repeat(width // 100 + 1)[:3 * width].to(dtype).cuda().view(3, width).clone().requires_grad_(True)
        x = torch.full((3, width), 2.0, dtype=dtype, device="cuda")  # uncentred, eps 0: n is 1, to a rounding or two
        dy = torch.full_like(x, -3.0)
        y = rn.group_norm(x, 1, gate=z, activation=act, eps=0.0, centered=False)
        (dz,) = torch.autograd.grad(y, z, dy)
        want = -3.0 * slopes(z.detach(), act)
        off = ((dz.double() - want).abs() / want.abs()).max().item()
        assert off <= (2.0 ** -17 if dtype == F32 else 2.0 ** -8 * (1 + 2.0 ** -6)), (width, off)
    # through an activation of the norm itself: t = n w + b with w = 0 is b
    b = torch.cat([torch.linspace(4, 64, 200), -torch.linspace(4, 64, 200)]).to(dtype).cuda().requires_grad_(True)
    x = torch.randn(1, 400, device="cuda").to(dtype)
    y = rn.group_norm(x, 1, torch.zeros_like(b), b, activation=act)
    (db,) = torch.autograd.grad(y, b, torch.full_like(y, 5.0))
    want = 5.0 * slopes(b.detach(), act)
    off = ((db.double() - want).abs() / want.abs()).max().item()
    assert off <= (2.0 ** -17 if dtype == F32 else 2.0 ** -8 * (1 + 2.0 ** -6)), off
