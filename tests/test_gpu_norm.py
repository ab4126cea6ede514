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
from torch.autograd import forward_ad

import recurrent_networks_gb300 as rn
from oracle import delta
from recurrent_networks_gb300.functional import flashrnn_stack

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
# row in shared memory; the widest; more groups than a CTA takes; many rows a CTA, of one
# warp and of several
SHAPES = [(1, 1, 1), (3, 5, 7), (7, 4, 16), (37, 5, 83), (9, 3, 256), (5, 2, 264), (130, 8, 128), (4, 1, 1000), (3, 2, 1001),
          (5, 1, 2049), (9, 3, 382), (2, 1, 2050), (3, 1, 4096), (2, 1, 8192), (2, 1, 14336), (2, 1, 14335), (6, 300, 8), (3, 70, 24), (5000, 3, 40),
          (4000, 1, 1000)]


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


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_no_rows_constant_rows_and_partial_gradients(dtype):
    p = make(0, 3, 40, dtype)
    x, w, b = (p[k].requires_grad_(True) for k in ("x", "w", "b"))
    y = rn.group_norm(x, 3, w, b)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.zeros_like(y))
    assert y.shape == (0, 120) and dx.shape == (0, 120) and (dw == 0).all() and (db == 0).all()
    # rows without a spread, and zero ones uncentred: n = 0, r = eps^-1/2
    p = make(20, 2, 96, dtype)
    p["x"][3:6] = 2.0
    p["x"][9] = 0.0
    check(p, 2, "silu")
    p["x"][3:6] = 0.0
    check(p, 2, "sigmoid", gate=False, centered=False)
    # each gradient by itself is the one that all of them give
    full = check(p, 2, "silu")
    for i, k in enumerate(("x", "gate", "w", "b")):
        t = {n: p[n].detach().clone().requires_grad_(n == k) for n in ("x", "gate", "w", "b")}
        y = rn.group_norm(t["x"], 2, t["w"], t["b"], t["gate"], "silu")
        (d,) = torch.autograd.grad(y, t[k], p["dy"], retain_graph=True)
        assert torch.equal(d, full[1 + i]) and torch.equal(torch.autograd.grad(y, t[k], p["dy"])[0], d)


def test_a_row_keeps_to_itself():
    """NaN and infinities in one group of one row reach that group's outputs alone."""
    for width in (40, 264, 1000, 4100):
        p = make(9, 2, width, BF)
        clean = rn.group_norm(p["x"], 2, p["w"], p["b"], p["gate"], "silu")
        x = p["x"].clone()
        x[4, width + 3] = float("inf")
        x[7, 0] = float("nan")
        y = rn.group_norm(x, 2, p["w"], p["b"], p["gate"], "silu")
        bad = torch.zeros(9, 2, dtype=torch.bool, device="cuda")
        bad[4, 1] = bad[7, 0] = True
        bad = bad.repeat_interleave(width, 1)
        assert torch.equal(y[~bad], clean[~bad]) and not torch.isfinite(y[4, width:]).any()
        y = rn.group_norm(x, 2, p["w"], p["b"], centered=False)  # the statistic of a group with a NaN is one
        assert y[7, :width].isnan().all() and torch.isfinite(y[7, width:]).all()


def test_leading_axes_strides_and_streams():
    p = make(60, 4, 24, BF)
    w, b = p["w"], p["b"]
    ref = check(p, 4, "silu")
    wide = torch.empty(3, 20, 4, 48, dtype=BF, device="cuda")
    wide[..., :24] = p["x"].view(3, 20, 4, 24)
    raw = torch.empty(97, dtype=BF, device="cuda")
    raw[1:] = w
    x = wide[..., :24].flatten(2).requires_grad_(True)
    gate = p["gate"].view(3, 20, 96).transpose(0, 1).contiguous().transpose(0, 1).requires_grad_(True)
    wt, bt = raw[1:].requires_grad_(True), b.clone().requires_grad_(True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = rn.group_norm(x, 4, wt, bt, gate, "silu")
        got = (y,) + torch.autograd.grad(y, (x, gate, wt, bt), p["dy"].view(3, 20, 96).transpose(0, 1).contiguous().transpose(0, 1))
    torch.cuda.current_stream().wait_stream(st)
    for a, r in zip(got, ref):
        assert torch.equal(a.reshape(r.shape), r)


def test_captured():
    p, other = make(300, 3, 40, BF), make(300, 3, 40, BF, seed=5)

    def work(t):
        leaves = [t[k].detach().requires_grad_(True) for k in ("x", "w", "b", "gate")]
        y = rn.group_norm(leaves[0], 3, *leaves[1:], activation="silu")
        return [y.detach(), *torch.autograd.grad(y, leaves, t["dy"])]

    ref = [t.clone() for t in work(other)]
    static = {k: v.clone() for k, v in p.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        work(static)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(static)
    for k, v in other.items():
        static[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_refusals():
    x = torch.zeros(2, 3, 24, device="cuda")
    w = torch.ones(24, device="cuda")
    for call in (lambda: rn.group_norm(x, 5), lambda: rn.group_norm(x, 0), lambda: rn.group_norm(x[..., :0], 1),
                 lambda: rn.group_norm(x, 4, w[:6]), lambda: rn.group_norm(x, 4, w, w[None]), lambda: rn.group_norm(x, 4, gate=x[0]),
                 lambda: rn.group_norm(x, 4, activation="relu"), lambda: rn.group_norm(x, 4, eps=-1.0),
                 lambda: rn.group_norm(x, 4, eps=float("nan")), lambda: rn.group_norm(x, 4, w.cpu()),
                 lambda: rn.group_norm(torch.zeros(1, 14337, device="cuda"), 1), lambda: rn.group_norm(torch.zeros((), device="cuda"), 1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rn.group_norm(x.double(), 4), lambda: rn.group_norm(x, 4, w.to(BF)), lambda: rn.group_norm(x, 4, gate=x.to(BF))):
        with pytest.raises(TypeError):
            call()
    for i in range(4):
        for grad in (True, False):
            with forward_ad.dual_level(), torch.set_grad_enabled(grad):
                args = [x, w, w, x]
                args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(NotImplementedError):
                    rn.group_norm(args[0], 4, *args[1:])
    t = x.clone().requires_grad_(True)
    y = rn.group_norm(t, 4, activation="silu")
    (d,) = torch.autograd.grad(y, t, torch.ones_like(y).requires_grad_(True), create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_in_a_stack():
    """A layer's `norm` is the group norm of its h, head by head, between the layers and behind the last."""
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: (torch.randn(*s, generator=g) * 0.2).to(BF).cuda()  # noqa: E731
    N, D = 2, 64
    layers = [dict(W_x=bf(4 * N * D, I), R=bf(4, N, D, D), b=bf(4, N, D)) for I in (72, N * D)]
    norms = [dict(weight=1 + bf(N * D), activation="silu"), dict(centered=False, eps=1e-4)]
    x, dh = bf(3, 17, 72), bf(3, 17, N * D)

    def both(run):
        t = x.clone().requires_grad_(True)
        w = norms[0]["weight"].clone().requires_grad_(True)
        h = run(t, [dict(norms[0], weight=w), norms[1]])
        return (h.detach(), *torch.autograd.grad(h, (t, w), dh))

    def whole(t, n):
        return flashrnn_stack(t, [dict(p, norm=m) for p, m in zip(layers, n)])[0]

    def parts(t, n):
        for p, m in zip(layers, n):
            t = rn.group_norm(flashrnn_stack(t, [p])[0], N, **m)
        return t

    for a, b in zip(both(whole), both(parts)):
        assert torch.equal(a, b)
