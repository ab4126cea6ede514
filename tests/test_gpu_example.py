"""The example model: embedding, projection, gated scan, 8-bit checkpoints and
the single-token step together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "gated_lm", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_lm.py"))
gated_lm = importlib.util.module_from_spec(spec)
spec.loader.exec_module(gated_lm)


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_it_learns(checkpoint):
    losses = gated_lm.train(gated_lm.GatedLM(), steps=80, checkpoint=checkpoint)
    assert all(x == x for x in losses)
    # untrained logits are far above log 64 = 4.16; the map from token to token ends far below
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])


def test_eight_bit_gradients_stay_close():
    """int8 with a scale per 32 steps of a channel: an error of at most 1/254 of
    the block's largest value, about 0.4 % of it uniformly distributed, in every
    pre-activation and layer input; the gradients' directions agree to a few
    per cent."""
    model = gated_lm.GatedLM(seed=3)
    tokens = gated_lm.language(8, 200, model.V, seed=1)
    grads = {}
    for ck in (None, "int8"):
        logits, _ = model.forward(tokens, checkpoint=ck)
        grads[ck] = torch.autograd.grad(logits.float().square().mean(), model.parameters())
    for a, b in zip(grads[None], grads["int8"]):
        a, b = a.double().flatten(), b.double().flatten()
        assert torch.dot(a, b) / (a.norm() * b.norm()) > 0.995


def test_steps_follow_the_whole_sequence():
    """Token by token (states in a pool) and at once: the same logits up to the
    bf16 roundings between the layers, which the two paths take in the same
    places; fp32 sums in another order move a rounding by one step at most."""
    model = gated_lm.GatedLM(seed=5)
    tokens = gated_lm.language(3, 40, model.V, seed=2)
    with torch.no_grad():
        whole, states = model.forward(tokens)
    pools = [torch.zeros(5, model.N, model.D, device="cuda") for _ in model.layers]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    steps = torch.stack([model.step(tokens[:, t], pools, slots) for t in range(40)], 1)
    scale = whole.float().abs().max()
    assert (steps.float() - whole.float()).abs().max() <= 2e-2 * scale
    for s, p in zip(states, pools):
        assert (p[slots.long()] - s[:, 0]).abs().max() <= 2e-2 * s.abs().max()


def test_packed_documents_equal_separate_ones():
    model = gated_lm.GatedLM(seed=7)
    a, b = gated_lm.language(1, 37, model.V, 1), gated_lm.language(1, 59, model.V, 2)
    both = torch.cat([a, b], 1)
    reset = torch.zeros(1, 96, dtype=torch.bool, device="cuda")
    reset[0, 0] = reset[0, 37] = True
    with torch.no_grad():
        packed, _ = model.forward(both, reset=reset)
        la, lb = model.forward(a)[0], model.forward(b)[0]
    scale = packed.float().abs().max()
    assert (packed[:, :37].float() - la.float()).abs().max() <= 2e-2 * scale
    assert (packed[:, 37:].float() - lb.float()).abs().max() <= 2e-2 * scale
