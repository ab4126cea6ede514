"""GPU parity of the group norm with an activation with its fp64 oracle.

Tolerances. fp32: a statistic is a sum of W terms (in parts of at most 64, then
over lanes), so 2^-24 * (W / 64 + 16) of its value; the remaining operations add
a few roundings: normwise-max 2^-24 * (W / 64 + 64); dweight and dbias are sums
over the rows in addition. bf16: rounded once, 2^-8 of the element at most, and
sigmoids to 2^-21: L2 3e-3 (a uniform rounding is 1.7e-3), normwise-max 2^-8 + 1e-5.
dx = r (dn - mean dn - n mean(dn n)) is a difference: where few channels share a
statistic its terms cancel (one uncentred channel: n^2 = 1 - eps / (var + eps),
dx = r dn eps / (var + eps)), and an error of 2^-24 in n is one of 2^-24 r |dn|
in dx, however small dx is; dx is therefore measured against the largest r |dn|.
A mean that is far above the spread costs |mean| / spread more bits in x - mean
(x itself is exact): the inputs here keep it below 4."""
import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import delta

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def close(got, ref, what, width, rows=1, least=1e-30):
    ref = np.asarray(ref, dtype=np.float64)
    assert tuple(got.shape) == ref.shape, what
    dtype = got.dtype
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), what
    if ref.size == 0:
        return
    worst = np.abs(got - ref).max() / max(np.abs(ref).max(), least)
    if dtype == BF:
        l2 = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), least * 1e-3)
        assert l2 <= 3e-3 and worst <= 2.0 ** -8 + 1e-5, f"{what}: L2 {l2:.3g}, max {worst:.3g}"
    else:
        tol = 2.0 ** -24 * (width / 64 + 64 + rows / 16)
        assert worst <= tol, f"{what}: max {worst:.3g} > {tol:.3g}"


def make(rows, groups, width, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows + width)
    C = groups * width
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(rows, groups, width) + r(groups, 1)) * torch.exp(r(groups, 1))
    return dict(x=x.reshape(rows, C).to(dtype).cuda(), gate=r(rows, C).to(dtype).cuda(), dy=r(rows, C).to(dtype).cuda(),
                w=(1 + 0.3 * r(C)).to(dtype).cuda(), b=(0.3 * r(C)).to(dtype).cuda())


def check(p, groups, act, gate=True, affine=True, centered=True, eps=1e-5):
    names = ["x"] + (["gate"] if gate else []) + (["w", "b"] if affine else [])
    t = {k: p[k].detach().clone().requires_grad_(True) for k in names}
    y = rn.group_norm(t["x"], groups, t.get("w"), t.get("b"), gate=t.get("gate"), activation=act, eps=eps, centered=centered)
    grads = dict(zip(names, torch.autograd.grad(y, [t[k] for k in names], p["dy"])))
    with torch.no_grad():
        assert torch.equal(y, rn.group_norm(t["x"], groups, t.get("w"), t.get("b"), gate=t.get("gate"), activation=act,
                                            eps=eps, centered=centered))
    ref = delta.group_norm(p["x"], groups, t.get("w"), t.get("b"), t.get("gate"), act, eps, centered, p["dy"])
    rows, width = p["x"].shape[0], p["x"].shape[1] // groups
    close(y, ref[0], "y", width)
    for k, r in zip(("x", "gate", "w", "b"), ref[1:5]):
        if k in grads:
            close(grads[k], r, "d" + k, width, rows if k in "wb" else 1, ref[5] if k == "x" else 1e-30)
    return (y, *grads.values())


# (rows, groups, width): one channel; odd widths; part of a warp, whole warps,
# several warps a group, with rows that are whole vectors and that are not; the
# row in shared memory; the widest; more groups than a CTA takes
SHAPES = [(1, 1, 1), (3, 5, 7), (7, 4, 16), (37, 5, 83), (9, 3, 256), (5, 2, 264), (130, 8, 128), (4, 1, 1000), (3, 2, 1001),
          (5, 1, 2049), (9, 3, 382), (2, 1, 2050), (3, 1, 4096), (2, 1, 8192), (2, 1, 14336), (2, 1, 14335), (6, 300, 8), (3, 70, 24), (5000, 3, 40)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "r%dg%dw%d" % s)
def test_parity(shape, dtype):
    p = make(*shape, dtype)
    check(p, shape[1], "silu")
    check(p, shape[1], None, gate=False, centered=False)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("width", [48, 51, 520, 4100])
def test_forms(width, gate, act, dtype):
    p = make(11, 3, width, dtype, seed=2)
    check(p, 3, act, gate)
    check(p, 3, act, gate, affine=False, centered=False, eps=1e-3)
