"""GPU parity of the token embedding and its gradient with the fp64 oracle.

Tolerances: the forward is one product in fp32 rounded once (bf16: 2^-9
relative, fp32: 2^-24). The gradient sums k terms in fp32: relative to the
sum of their magnitudes k 2^-24, and one rounding to the type. Against the
largest row sum: bf16 1e-2 of the largest element (and 5e-3 in L2), fp32
k 2^-23."""
import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import recurrent_networks_gb300 as rn
from oracle import gated
from recurrent_networks_gb300 import _lib

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(ids, V, E, dtype, scale=1.0, pad=None, id_dtype=torch.int64, seed=0):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, E, generator=g).to(dtype).cuda().requires_grad_(True)
    t = torch.as_tensor(ids).to(id_dtype).cuda()
    out = rn.embedding(t, W, scale=scale, padding_idx=pad)
    assert out.shape == tuple(t.shape) + (E,) and out.dtype == dtype
    flat = np.asarray(ids).reshape(-1)
    ref = gated.embed(flat, W, scale).reshape(out.shape)
    got = out.detach().double().cpu().numpy()
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** (-8 if dtype == BF else -23)).all()
    dout = torch.randn(out.shape, generator=g).to(dtype).cuda()
    (dW,) = torch.autograd.grad(out, W, dout)
    rdW = gated.embed_grad(flat, V, dout.reshape(-1, E), scale, pad)
    got = dW.double().cpu().numpy()
    assert np.isfinite(got).all()
    untouched = np.setdiff1d(np.arange(V), flat if pad is None else flat[flat != pad])
    assert (got[untouched] == 0).all()
    top = max(np.abs(rdW).max(), 1e-30)
    worst = np.abs(got - rdW).max() / top
    if dtype == BF:
        l2 = np.linalg.norm(got - rdW) / max(np.linalg.norm(rdW), 1e-30)
        assert worst <= 1e-2 and l2 <= 5e-3, (worst, l2)
    else:
        k = max(int(np.bincount(flat[(flat >= 0) & (flat < V)], minlength=1).max()) if flat.size else 0, 1)
        assert worst <= 2.0 ** -23 * (k + 1), worst
    (again,) = torch.autograd.grad(rn.embedding(t, W, scale=scale, padding_idx=pad), W, dout)
    assert torch.equal(again, dW)
    return dW


def zipf(n, V, seed=0):
    r = np.random.default_rng(seed)
    p = 1 / (np.arange(V) + 2.7)
    return r.permutation(V)[r.choice(V, size=n, p=p / p.sum())]


# (n, V, E): one token; odd widths (rows of 2-, 4- and 8-byte alignment);
# fewer and more tokens than a single block sorts; more ids than 16 bits hold
SIZES = [(1, 1, 1), (1, 1000, 64), (31, 7, 9), (74, 1003, 200), (700, 300, 130), (4097, 5000, 36), (9000, 70001, 68),
         (20000, 300, 256)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "n%dV%dE%d" % s)
def test_parity(size, dtype):
    n, V, E = size
    check(zipf(n, V, seed=n), V, E, dtype, scale=0.5 + E ** 0.5, id_dtype=torch.int32 if n % 2 else torch.int64)


def test_more_ids_than_two_digits_hold():
    ids = np.random.default_rng(1).integers(0, 5_000_000, 3000)
    ids[:1000] = ids[2000]
    check(ids, 5_000_000, 3, BF)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_one_id_for_every_token(dtype):
    check(np.full(5000, 3), 8, 72, dtype)
    check(np.full(12345, 0), 1, 40, dtype)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_every_id_once_and_in_order(dtype):
    check(np.arange(3000), 3000, 40, dtype)
    check(np.arange(6000)[::-1].copy(), 6000, 40, dtype)


def test_padding():
    ids = zipf(2000, 50)
    ids[::3] = 4
    dW = check(ids.reshape(20, 100), 50, 96, BF, pad=4)
    assert (dW[4] == 0).all()
    check(np.full(300, 4), 50, 96, F32, pad=4)  # nothing else: the gradient is zero


def test_no_tokens():
    W = torch.randn(5, 8, device="cuda", requires_grad=True)
    out = rn.embedding(torch.zeros(0, 3, dtype=torch.int64, device="cuda"), W)
    assert out.shape == (0, 3, 8)
    (dW,) = torch.autograd.grad(out.sum(), W)
    assert (dW == 0).all()


@pytest.mark.parametrize("n", [100, 9001])
def test_ids_out_of_range_are_left_out_and_reported(n):
    V, E = 70, 48
    ids = zipf(n, V)
    bad = ids.copy().astype(np.int64)
    bad[5], bad[50] = V, -1
    bad[7] = 2 ** 40
    W = torch.randn(V, E, device="cuda", requires_grad=True)
    t = torch.as_tensor(bad).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = rn.embedding(t, W, status=status)
    assert (out[[5, 7, 50]] == 0).all()
    with pytest.raises(_lib.RnnError) as err:
        _lib.rnn_check_status(status)
    assert err.value.status == _lib.RNN_ERANGE
    dout = torch.randn(n, E, device="cuda")
    (dW,) = torch.autograd.grad(out, W, dout)
    ref = gated.embed_grad(bad, V, dout, 1.0)
    assert np.abs(dW.double().cpu().numpy() - ref).max() <= np.abs(ref).max() * 2.0 ** -23 * n
    ws = torch.empty(_lib.rnn_embed_bwd_workspace_size(n, V, E), dtype=torch.uint8, device="cuda")
    _lib.rnn_embed_bwd(n, V, E, t, -1, dout, 1.0, torch.empty_like(W), ws)
    with pytest.raises(_lib.RnnError) as err:
        _lib.rnn_check_status(ws)
    assert err.value.status == _lib.RNN_ERANGE


def test_strided_gradient_and_weight():
    V, E, n = 40, 33, 500
    ids = torch.as_tensor(zipf(n, V)).cuda()
    W = torch.randn(E, V, device="cuda").t().requires_grad_(True)
    dout = torch.randn(E, n, device="cuda").t()
    (dW,) = torch.autograd.grad(rn.embedding(ids, W), W, dout)
    W2 = W.detach().contiguous().requires_grad_(True)
    (dW2,) = torch.autograd.grad(rn.embedding(ids, W2), W2, dout.contiguous())
    assert torch.equal(dW, dW2)


def test_gradient_by_differences():
    """sum(out * dout) is linear in W: a difference of two losses is exact up
    to fp32 rounding of the forward (2^-23 of the terms' magnitudes)."""
    ids = torch.as_tensor(zipf(60, 9)).cuda()
    W = torch.randn(9, 12, device="cuda", requires_grad=True)
    dout = torch.randn(60, 12, device="cuda")
    (dW,) = torch.autograd.grad(rn.embedding(ids, W, scale=3.0), W, dout)
    step = torch.zeros_like(W)
    step[2, 5] = 1.0
    d = dout.double()
    hi = (rn.embedding(ids, W + step, scale=3.0).double() * d).sum()
    lo = (rn.embedding(ids, W - step, scale=3.0).double() * d).sum()
    assert abs((hi - lo).item() / 2 - dW[2, 5].item()) < 1e-3


def test_refusals():
    W = torch.randn(5, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    for call in (lambda: rn.embedding(ids, W[0]), lambda: rn.embedding(ids, W, padding_idx=5),
                 lambda: rn.embedding(ids, W, padding_idx=-1), lambda: rn.embedding(ids.cpu(), W)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rn.embedding(ids.float(), W), lambda: rn.embedding(ids, W.double())):
        with pytest.raises(TypeError):
            call()


def test_forward_mode_is_refused():
    W, ids = torch.randn(7, 8, device="cuda"), torch.arange(3, device="cuda")
    for grad in (True, False):
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            with pytest.raises(NotImplementedError):
                rn.embedding(ids, forward_ad.make_dual(W, torch.ones_like(W)))
            rn.embedding(ids, W)
    W.requires_grad_(True)
    with forward_ad.dual_level():
        out = rn.embedding(ids, W)
        with pytest.raises(NotImplementedError):  # forward over reverse
            torch.autograd.grad(out, W, forward_ad.make_dual(torch.ones_like(out), torch.ones_like(out)))
