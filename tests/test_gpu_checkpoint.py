"""8-bit activation checkpoints: the packed bytes equal the definition's bit
for bit, and the input projection's gradients from a packed input."""
import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import gated, projection
from recurrent_networks_gb300 import _lib

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (31, 3), (32, 130), (33, 64), (200, 37), (97, 66), (64, 520)],
                         ids=lambda s: "%dx%d" % s)
def test_bits(shape, dtype):
    g = torch.Generator().manual_seed(shape[0] * 1000 + shape[1])
    x = torch.randn(shape, generator=g) * torch.exp(4 * torch.randn(shape[1], generator=g))
    x[:, 0] = 0
    if shape[1] > 8:
        x[:, 1] = 127.0          # the largest step holds it exactly
        x[:, 2] = 127.5
        x[:, 3] = torch.finfo(dtype).max
        x[:, 4] = torch.finfo(dtype).tiny / 8   # below the smallest scale's range
        x[:, 5] *= 1e-38
        x[:, 6] = torch.arange(shape[0]) % 2 + 0.5  # halves: ties go to even
        x[0, 6] = 127.0
    x = x.to(dtype)
    q, s = rn.checkpoint_pack(x.cuda())
    rq, rs = gated.pack(x)
    assert np.array_equal(s.cpu().numpy().astype(np.int64), rs)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    for out in (F32, BF):
        y = rn.checkpoint_unpack(q, s, out)
        assert y.dtype == out and np.array_equal(y.double().cpu().numpy(), gated.unpack(rq, rs))
    # half a step of the scale, and 127 / 2 steps fall short of the largest magnitude
    top = np.repeat(gated.f64(x.abs().float()).max(0, keepdims=True), shape[0], 0)
    assert (np.abs(gated.unpack(rq, rs) - gated.f64(x)) <= np.maximum(top / 127, 2.0 ** -127)).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_nonfinite_blocks(dtype):
    x = torch.randn(70, 16)
    x[3, 2], x[40, 5], x[69, 15] = float("inf"), float("nan"), float("-inf")
    q, s = rn.checkpoint_pack(x.to(dtype).cuda())
    y = rn.checkpoint_unpack(q, s, F32).cpu()
    bad = torch.zeros(70, 16, dtype=torch.bool)
    bad[:32, 2] = bad[32:64, 5] = bad[64:, 15] = True
    assert torch.equal(torch.isnan(y), bad)


def test_shapes_strides_and_refusals():
    x = torch.randn(2, 50, 24, device="cuda")
    q, s = rn.checkpoint_pack(x)
    assert q.shape == x.shape and s.shape == (4, 24)
    q2, s2 = rn.checkpoint_pack(x.reshape(100, 24).t().contiguous().t())
    assert torch.equal(q.reshape(100, 24), q2) and torch.equal(s, s2)
    q0, s0 = rn.checkpoint_pack(x[:0])
    assert rn.checkpoint_unpack(q0, s0).shape == (0, 50, 24)
    for call in (lambda: rn.checkpoint_unpack(q, s[:3]), lambda: rn.checkpoint_unpack(q, s.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rn.checkpoint_pack(x.double()), lambda: rn.checkpoint_unpack(x, s),
                 lambda: rn.checkpoint_unpack(q, s, torch.float16)):
        with pytest.raises(TypeError):
            call()
    W = torch.randn(64, 64, device="cuda").to(BF)
    with pytest.raises(ValueError):
        rn.input_projection(W, W, checkpoint="fp8")


def _close(got, ref, what):
    # one rounding to bf16 of an fp32 sum: the projection's own tolerance
    got = got.detach().double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref), what
    assert np.abs(got - ref).max() <= 1e-2 * np.abs(ref).max(), what


@pytest.mark.parametrize("BT,I,C", [(37, 128, 96), (300, 72, 200), (2050, 256, 768)])
def test_projection_with_a_packed_input(BT, I, C):
    g = torch.Generator().manual_seed(BT)
    x = torch.randn(BT, I, generator=g).to(BF).cuda().requires_grad_(True)
    W = (torch.randn(C, I, generator=g) / I ** 0.5).to(BF).cuda().requires_grad_(True)
    bias = torch.randn(C, generator=g).to(BF).cuda().requires_grad_(True)
    dy = torch.randn(BT, C, generator=g).to(BF).cuda()
    y = rn.input_projection(x, W, bias, checkpoint="int8")
    dx, dW, db = torch.autograd.grad(y, (x, W, bias), dy)
    y0 = rn.input_projection(x, W, bias)
    dx0, _, db0 = torch.autograd.grad(y0, (x, W, bias), dy)
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(db, db0)
    _close(dW, projection.bwd(gated.unpacked(x), W, dy)[1], "dW")
    # W frozen: nothing of x is needed
    (dx1,) = torch.autograd.grad(rn.input_projection(x, W.detach(), checkpoint="int8"), x, dy)
    assert torch.equal(dx1, dx)


def test_projection_packs_only_for_a_backward():
    x, W = torch.randn(64, 64, device="cuda").to(torch.bfloat16), torch.randn(64, 64, device="cuda").to(torch.bfloat16)
    ref = rn.input_projection(x, W)

    def launches(checkpoint):
        before = _lib.rnn_kernel_launches()
        y = rn.input_projection(x, W.requires_grad_(True), checkpoint=checkpoint)
        assert torch.equal(y, ref)
        return _lib.rnn_kernel_launches() - before

    assert launches("int8") == launches(None) + 1  # the packing
    with torch.no_grad():
        assert launches("int8") == launches(None)
