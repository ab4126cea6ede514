"""The delta rule's operators as a model uses them together: projections, unit
keys and queries from the uncentred group norm, the rule, the gated group norm
of its heads, and the projection back; a training step of packed documents, and
the same tokens in a prefill and single steps on a pool of states.

Tolerances. Everything is bf16 between the operators. Along the longest path (x,
projection, norm, rule, norm, projection, and back) some dozen roundings of 1.7e-3
each (L2, uniform) add up independently to 6e-3; the norms' backward passes take
a part out of the gradient that can be most of it, so 3e-2 and cosine 0.999, as
for two stacked layers."""
import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
E, NK, N, DK, DV = 72, 2, 4, 32, 24  # model width; heads of q and k, of v; their channels
PARTS = (NK * DK, NK * DK, N * DV, N * DV)  # q, k, v and the output's gate


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).to(BF).cuda()  # noqa: E731
    return dict(W_in=r(sum(PARTS), E, by=E ** -0.5), W_gates=r(2 * N, E, by=E ** -0.5), w=1 + r(N * DV, by=0.2),
                W_out=r(E, N * DV, by=(N * DV) ** -0.5))


def project(x, p):
    """q, k, v, the output's gate z, g and beta of tokens x [..., E]."""
    q, k, v, z = rn.input_projection(x, p["W_in"]).split(PARTS, -1)
    unit = torch.full((NK * DK,), DK ** -0.5, dtype=BF, device=x.device)
    q, k = (rn.group_norm(t, NK, unit, eps=1e-6, centered=False).unflatten(-1, (NK, DK)) for t in (q, k))
    a, b = (x.float() @ p["W_gates"].float().T).split([N, N], -1)
    return q, k, v.unflatten(-1, (N, DV)), z, -0.1 * torch.nn.functional.softplus(a), torch.sigmoid(b)


def finish(o, z, p):
    o = rn.group_norm(o.flatten(-2), N, p["w"], gate=z, activation="silu")
    return rn.input_projection(o, p["W_out"])


def block(x, p, reset=None, lengths=None):
    q, k, v, z, g, beta = project(x, p)
    o, last = rn.gated_delta(q, k, v, g, beta, reset=reset, lengths=lengths)
    return finish(o, z, p), last


def plain(x, p, reset=None):
    """The block in the inputs' (64-bit) type, step by step."""
    B, T = x.shape[:2]
    q, k, v, z = (x @ p["W_in"].T).split(PARTS, -1)

    def rms(t, heads, eps):
        t = t.unflatten(-1, (heads, -1))
        return t / (t.square().mean(-1, keepdim=True) + eps).sqrt()

    q, k = (rms(t, NK, 1e-6).repeat_interleave(N // NK, 2) * DK ** -0.5 for t in (q, k))
    v = v.unflatten(-1, (N, DV))
    a, b = (x @ p["W_gates"].T).split([N, N], -1)
    decay, beta = torch.exp(-0.1 * torch.nn.functional.softplus(a)), torch.sigmoid(b)
    if reset is not None:
        decay = decay * ~reset[..., None]
    S, out = torch.zeros(B, N, DK, DV, dtype=x.dtype), []
    for t in range(T):
        S = decay[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bnkv,bnk->bnv", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        out.append(DK ** -0.5 * torch.einsum("bnkv,bnk->bnv", S, q[:, t]))
    o = torch.stack(out, 1)
    o = o - o.mean(-1, keepdim=True)
    o = rms(o.flatten(2), N, 1e-5).flatten(2) * p["w"] * torch.nn.functional.silu(z)
    return o @ p["W_out"].T, S[:, None]


def near(got, ref, what):
    got, ref = (np.asarray(t.detach().double().cpu()) for t in (got, ref))
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    l2 = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    cos = (got * ref).sum() / np.linalg.norm(got) / np.linalg.norm(ref)
    assert l2 <= 3e-2 and cos >= 0.999, f"{what}: L2 {l2:.3g}, cosine {cos:.5f}"


def test_training_step():
    p = weights(1)
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(2, 150, E, generator=g).to(BF).cuda() for _ in range(2))
    reset = torch.zeros(2, 150, dtype=torch.bool)
    reset[:, 0] = reset[0, 40] = reset[1, 64] = reset[1, 131] = True
    leaves = [x.requires_grad_(True), *(t.requires_grad_(True) for t in p.values())]
    y, last = block(x, p, reset.cuda())
    got = torch.autograd.grad(y, leaves, dy)
    rx, *rw = (t.detach().double().cpu().requires_grad_(True) for t in leaves)
    ry, rlast = plain(rx, dict(zip(p, rw)), reset)
    ref = torch.autograd.grad(ry, (rx, *rw), dy.double().cpu())
    near(y, ry, "y")
    near(last, rlast, "last")
    for name, a, b in zip(("x", *p), got, ref):
        near(a, b, "d" + name)


@torch.no_grad()
def test_prefill_and_single_tokens():
    """Prompts of several lengths in one padded batch, then tokens by steps in a
    pool of more slots, one row of the batch unused."""
    p = weights(3)
    x = torch.randn(3, 90, E, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    prompt, more = [70, 1, 33], 12
    lengths = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    padded = x.clone()
    for i, n in enumerate(prompt):
        padded[i, n:] = float("nan")
    y, last = block(padded[:, :70], p, lengths=lengths)
    pool = torch.full((6, N, DK, DV), 7.0, device="cuda")
    slots = [4, 0, 5]
    pool[slots] = last[:, 0]
    at = torch.tensor([4, -1, 0, 5], dtype=torch.int32, device="cuda")
    rows = [0, 2, 3]
    steps = []
    for t in range(more):
        tok = torch.zeros(4, E, dtype=BF, device="cuda")
        tok[rows] = torch.stack([x[i, n + t] for i, n in enumerate(prompt)])
        q, k, v, z, g, beta = project(tok, p)
        o = rn.gated_delta_step(q, k, v, g, beta, pool, at)
        steps.append(finish(o, z, p)[rows])
    steps = torch.stack(steps, 1)
    wide = {k: v.double().cpu() for k, v in p.items()}
    for i, n in enumerate(prompt):
        ry, rlast = plain(x[i:i + 1, :n + more].double().cpu(), wide)
        near(torch.cat([y[i, :n], steps[i]]), ry[0], f"row {i}")
        near(pool[slots[i]], rlast[0, 0], f"state {i}")
    assert (pool[1:4] == 7.0).all()
