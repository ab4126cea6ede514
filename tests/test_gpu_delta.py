"""GPU parity of the gated delta rule (forward, backward, single-token step)
with its fp64 oracle, and what its calls promise.

Tolerances. Every product's operands are held to 2^-24 of their values and
summed in fp32. An element of an output is a sum over the earlier steps of a
chain of products; with unit keys and beta in (0, 1) every factor of the
recurrence is a contraction, so the errors of its steps add up without growing,
and the triangular inverse of a chunk doubles them a few times: normwise-max
2^-24 * (64 + T / 4) for fp32 outputs of either storage. dg of bf16 storage is a
sum of up to 8 * 64 row products that cancel where memories are short, 2^-24 *
sqrt(512) = 23 times 2^-24 of a row product each: 2^-24 * (256 + T / 4). bf16
outputs are rounded once on top, by 2^-8 of the element at most: L2 3e-3 (a
uniform rounding is 1.7e-3), normwise-max 2^-8 + the above. dq and dk of bf16
storage are sums of products of two operands that were rounded to bf16 once (dY,
Z, S0, dS1), inside a chunk of three (dY, Z, and M or R): 1.7e-3 each,
independently, sqrt(3 + 1) * 1.7e-3 = 3.4e-3 with the output's own: L2 4e-3; the
normwise maximum four roundings of 2^-8. Those roundings are of the terms, and
dq = scale (D dO + k u.dO) and dk = dS u - D dv (D the decayed state) are sums of
two that can cancel where a head has few channels: the two are measured against
the larger of the sum and its terms."""
import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import delta

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("o", "last", "dq", "dk", "dv", "dg", "dbeta", "dstate")


def close(got, ref, what, T, storage, terms=()):
    ref = np.asarray(ref, dtype=np.float64)
    assert tuple(got.shape) == ref.shape, what
    out = got.dtype
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), what
    if ref.size == 0:
        return
    top = max([np.abs(x).max() for x in (ref, *terms)] + [1e-30])
    worst = np.abs(got - ref).max() / top
    l2 = np.linalg.norm(got - ref) / max([np.linalg.norm(x) for x in (ref, *terms)] + [1e-30])
    inner = 2.0 ** -24 * ((256 if what == "dg" and storage == BF else 64) + T / 4)
    if out == BF:
        rounds = 4 if what in ("dq", "dk") else 1
        assert l2 <= (4e-3 if rounds > 1 else 3e-3) and worst <= rounds * 2.0 ** -8 + inner, f"{what}: L2 {l2:.3g}, max {worst:.3g}"
    else:
        assert worst <= inner, f"{what}: max {worst:.3g} > {inner:.3g}"


def make(B, T, Nk, N, Dk, Dv, dtype, seed=0, lead=None):
    g = torch.Generator().manual_seed(seed + 7 * T + Dk + 3 * Dv)
    lead = (B, T) if lead is None else lead

    def unit(*shape):
        x = torch.randn(*shape, generator=g)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype).cuda()

    p = dict(q=unit(*lead, Nk, Dk), k=unit(*lead, Nk, Dk), v=torch.randn(*lead, N, Dv, generator=g).to(dtype).cuda())
    tau = 2 * torch.exp(torch.rand(N, generator=g) * 6)
    p["g"] = (-torch.nn.functional.softplus(torch.randn(*lead, N, generator=g)) / tau).cuda()
    p["beta"] = torch.sigmoid(torch.randn(*lead, N, generator=g)).cuda()
    p["state"] = (torch.randn(B, 1, N, Dk, Dv, generator=g) / Dk ** 0.5).cuda()
    p["do"] = torch.randn(*lead, N, Dv, generator=g).to(dtype).cuda()
    p["dlast"] = torch.randn(B, 1, N, Dk, Dv, generator=g).cuda()
    return p


LEAVES = ("q", "k", "v", "g", "beta", "state")


def run(p, reset=None, lengths=None, scale=None, grads=True):
    leaves = [p[k].clone().requires_grad_(grads) for k in LEAVES]
    o, last = rn.gated_delta(*leaves, scale=scale, reset=reset, lengths=lengths)
    if not grads:
        return o, last
    return (o, last) + torch.autograd.grad((o, last), leaves, (p["do"], p["dlast"]))


def oracle(p, reset=None, lengths=None, scale=None):
    o, last, trail = delta.fwd(*(p[k] for k in LEAVES), scale, reset, lengths)
    return (o, last) + delta.bwd(*(p[k] for k in LEAVES[:5]), trail, p["do"], p["dlast"], scale)


def check(p, reset=None, lengths=None, scale=None):
    got = run(p, reset, lengths, scale)
    *ref, parts = oracle(p, reset, lengths, scale)
    for name, a, r in zip(NAMES, got, ref):
        terms = parts[:2] if name == "dq" else parts[2:] if name == "dk" else ()
        close(a, r, name, p["q"].shape[1], p["q"].dtype, terms)
    return got


# (B, T, Nk, N, Dk, Dv): one step; one channel; one chunk, one step more and one
# less (64 steps of bf16, 32 of fp32); odd widths; shared heads; widths around
# the tiles of 16, 32, 64 and 128 and the largest; several chunks
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 16, 1, 1, 32, 32), (1, 31, 1, 2, 17, 9), (2, 32, 1, 1, 64, 64), (1, 33, 2, 2, 16, 100),
          (2, 63, 1, 3, 20, 33), (1, 64, 1, 1, 128, 128), (1, 65, 2, 4, 72, 40), (1, 200, 1, 1, 130, 65),
          (1, 130, 1, 1, 256, 256), (1, 129, 1, 1, 192, 192), (1, 100, 1, 1, 208, 7), (1, 700, 1, 2, 48, 64),
          (20, 70, 2, 4, 128, 96)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_parity(shape, dtype):
    check(make(*shape, dtype))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5, 70, 1, 2, 33, 20), (5, 300, 2, 2, 64, 72)], ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_masks(shape, dtype):
    B, T = shape[:2]
    p = make(*shape, dtype, seed=3)
    g = torch.Generator().manual_seed(T)
    reset = torch.rand(B, T, generator=g) < 0.05
    reset[0, 0] = True
    reset[1] = True  # every step its own document
    lengths = torch.tensor([T, T - 1, 0, T // 2, 1], dtype=torch.int32)
    clean = check(p, reset.cuda(), lengths.cuda())
    # whatever stands past a row's length must not matter
    dirty = {k: v.clone() for k, v in p.items()}
    for i in range(B):
        n = int(lengths[i])
        for k in ("q", "k", "v", "g", "beta"):
            dirty[k][i, n:] = float("nan")
        dirty["do"][i, n:] = float("inf")
    again = run(dirty, reset.cuda(), lengths.cuda())
    for a, b in zip(clean, again):
        assert torch.equal(a, b)
    # resets as decays: the same steps with g = -inf, or the type's lowest value
    for low in (float("-inf"), torch.finfo(F32).min):
        as_g = dict(p, g=p["g"].masked_fill(reset.cuda()[..., None], low))
        for a, b in zip(clean, run(as_g, None, lengths.cuda())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_step(dtype):
    for M, P, Nk, N, Dk, Dv in [(1, 1, 1, 1, 1, 1), (5, 9, 2, 6, 40, 33), (3, 3, 1, 1, 256, 256), (7, 8, 1, 2, 128, 64)]:
        p = make(P, 1, Nk, N, Dk, Dv, dtype, lead=(M,))
        pool = p["state"][:, 0].contiguous()
        slots = torch.randperm(P, generator=torch.Generator().manual_seed(M))[:M].to(torch.int32)
        if M > 2:
            slots[1] = -1
        keep, out = pool.clone(), pool.clone()
        args = [p[k] for k in LEAVES[:5]]
        o = rn.gated_delta_step(*args, pool, slots.cuda(), pool_out=out)
        assert torch.equal(pool, keep)
        ref_o, ref_pool = np.zeros((M, N, Dv)), keep.double().cpu().numpy()
        for m in range(M):
            s = int(slots[m])
            if s >= 0:
                r, last, _ = delta.fwd(*(x[m][None, None] for x in args), keep[s][None, None])
                ref_o[m], ref_pool[s] = r[0, 0], last[0, 0]
        close(o, ref_o, "o", 1, dtype if dtype == BF else F32)
        close(out, ref_pool, "pool", 1, F32)
        assert torch.equal(rn.gated_delta_step(*args, pool, slots.cuda()), o) and torch.equal(pool, out)


# few heads and a long axis: the chunks run in segments whose states are joined
# (keys up to 128 channels, and past them), with shorter rows among them
@pytest.mark.parametrize("shape", [(1, 3001, 1, 1, 64, 96), (2, 2500, 1, 2, 144, 40), (1, 2070, 1, 2, 16, 8)],
                         ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_segments(shape):
    p = make(*shape, BF, seed=5)
    check(p)
    B, T = shape[:2]
    lengths = torch.tensor([T // 2 + 3, 70][:B], dtype=torch.int32).cuda()
    reset = (torch.rand(B, T, generator=torch.Generator().manual_seed(1)) < 0.002).cuda()
    check(p, reset, lengths)
