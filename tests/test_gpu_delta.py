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
uniform rounding is 1.7e-3), normwise-max 2^-8 + the above. dq
and dk of bf16 storage are sums of products of operands in two bf16 planes (2^-17
of a value remain at most; dY, Z, S0, dS1, and M or R, made of two of them),
without the product of two second planes (2^-18): 2^-17 * 4 + 2^-18, below 2^-14
together. They are of the terms, and dq = scale (D dO + k u.dO) and dk = dS u -
D dv (D the decayed state) are sums of two that can cancel where a head has few
channels: the two are measured against the larger of the sum and its terms."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import recurrent_networks_gb300 as rn
from oracle import delta
from recurrent_networks_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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
        inner += 2.0 ** -14 if what in ("dq", "dk") else 0
        assert l2 <= 3e-3 and worst <= 2.0 ** -8 + inner, f"{what}: L2 {l2:.3g}, max {worst:.3g}"
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


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_no_steps_and_optional_arguments(dtype):
    p = make(2, 0, 1, 2, 24, 40, dtype)
    o, last, dq, dk, dv, dg, dbeta, ds = run(p)
    assert o.shape == (2, 0, 2, 40) and torch.equal(last, p["state"]) and torch.equal(ds, p["dlast"])
    assert dq.shape == p["q"].shape and dv.shape == p["v"].shape and dg.shape == p["g"].shape
    assert (rn.gated_delta(*(p[k] for k in LEAVES[:5]))[1] == 0).all()
    p = make(2, 150, 1, 2, 24, 40, dtype, seed=1)
    args = [p[k] for k in LEAVES[:5]]
    for a, b in zip(rn.gated_delta(*args), rn.gated_delta(*args, torch.zeros_like(p["state"]), scale=24 ** -0.5)):
        assert torch.equal(a, b)
    # the gradients of one output alone, with another scale
    o, last, trail = delta.fwd(*args, p["state"], 0.3)
    leaves = [p[k].clone().requires_grad_(True) for k in LEAVES]
    out = rn.gated_delta(*leaves, scale=0.3)
    for i, name in enumerate(("do", "dlast")):
        got = torch.autograd.grad(out[i], leaves, p[name], retain_graph=True)
        *ref, parts = delta.bwd(*args, trail, **{name: p[name]}, scale=0.3)
        for what, a, r in zip(NAMES[2:], got, ref):
            if name == "dlast" and what == "dq":
                assert (a == 0).all()
                continue
            close(a, r, what, 150, dtype, parts[:2] if what == "dq" else parts[2:] if what == "dk" else ())
    # of one input alone, the graph used twice
    v = p["v"].clone().requires_grad_(True)
    o, _ = rn.gated_delta(args[0], args[1], v, args[3], args[4], p["state"], scale=0.3)
    a = torch.autograd.grad(o, v, p["do"], retain_graph=True)
    b = torch.autograd.grad(o, v, p["do"])
    assert torch.equal(a[0], b[0])
    close(a[0], delta.bwd(*args, trail, do=p["do"], scale=0.3)[2], "dv", 150, dtype)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_betas(dtype):
    """beta of 0, below it, and up to 2, where a step's matrix still has norm one."""
    p = make(1, 200, 1, 2, 40, 48, dtype, seed=9)
    p["beta"] = 1.9 * p["beta"]
    p["beta"][:, ::3] = 0
    p["beta"][:, 1::17] *= -0.1
    check(p)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_reset_drops_an_infinite_state(dtype):
    for shape in ((2, 150, 1, 1, 40, 48), (1, 2500, 1, 1, 64, 64)):  # the second in segments
        p = make(*shape, dtype)
        reset = torch.zeros(shape[:2], dtype=torch.bool, device="cuda")
        reset[:, 0] = True
        ref = run(p, reset)
        for bad in (float("inf"), float("nan")):
            got = run(dict(p, state=torch.full_like(p["state"], bad)), reset)
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
            assert (got[-1] == 0).all()
            lengths = torch.zeros(shape[0], dtype=torch.int32, device="cuda")
            o, last = rn.gated_delta(*(p[k] for k in LEAVES[:5]), torch.full_like(p["state"], bad), lengths=lengths)
            assert (o == 0).all() and not torch.isfinite(last).any()


def test_strided_and_misaligned_inputs():
    p = make(2, 140, 2, 4, 24, 40, BF)
    p["g"], p["beta"] = p["g"].to(BF), p["beta"].to(BF)  # gates of the values' type
    plain = [p[k].clone().requires_grad_(True) for k in LEAVES]
    ref = rn.gated_delta(*plain)
    ref = ref + torch.autograd.grad(ref, plain, (p["do"], p["dlast"]))
    # q, k and v as slices of one tensor, gates with their axes swapped, a state
    # that is off the 16-byte grid and a gradient that is not contiguous
    qkv = torch.cat([p[k].flatten(2) for k in ("q", "k", "v")], 2)
    q, k, v = (x.unflatten(2, (n, -1)).requires_grad_(True) for x, n in zip(qkv.split([48, 48, 160], 2), (2, 2, 4)))
    g, beta = (p[x].transpose(1, 2).contiguous().transpose(1, 2).requires_grad_(True) for x in ("g", "beta"))
    raw = torch.empty(p["state"].numel() + 1, device="cuda")
    raw[1:] = p["state"].reshape(-1)
    leaves = [q, k, v, g, beta, raw[1:].view(p["state"].shape).requires_grad_(True)]
    out = rn.gated_delta(*leaves)
    do = p["do"].transpose(2, 3).contiguous().transpose(2, 3)
    got = out + torch.autograd.grad(out, leaves, (do, p["dlast"]))
    assert got[5].dtype == BF
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    state = p["state"].clone()
    args = [x[:, 0] for x in (q, k, v, g, beta)]
    o = rn.gated_delta_step(*args, state[:, 0])
    for i in range(5):
        args[i] = plain[i][:, 0].contiguous()
    again = p["state"][:, 0].clone()
    assert torch.equal(rn.gated_delta_step(*args, again), o) and torch.equal(again, state[:, 0])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_repeatable_and_on_another_stream(dtype):
    for shape in ((3, 300, 2, 6, 64, 72), (1, 2500, 1, 2, 128, 128)):
        p = make(*shape, dtype)
        ref = run(p)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got = run(p)
        torch.cuda.current_stream().wait_stream(st)
        for again in (got, run(p)):
            assert all(torch.equal(a, b) for a, b in zip(again, ref))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_continues_from_its_last_state(dtype):
    """In two calls, and by single tokens: rounded o only where it is bf16."""
    p = make(3, 90, 1, 2, 40, 24, dtype)
    args = [p[k] for k in LEAVES[:5]]
    ref_o, ref_last, _ = delta.fwd(*args, p["state"])
    o1, s = rn.gated_delta(*(x[:, :37] for x in args), p["state"])
    o2, last = rn.gated_delta(*(x[:, 37:] for x in args), s)
    close(torch.cat([o1, o2], 1), ref_o, "o", 90, dtype)
    close(last, ref_last, "last", 90, F32)
    pool = s[:, 0].clone()
    steps = torch.stack([rn.gated_delta_step(*(x[:, t] for x in args), pool) for t in range(37, 90)], 1)
    close(torch.cat([o1, steps], 1), ref_o, "o by steps", 90, dtype)
    close(pool, ref_last[:, 0], "state by steps", 90, F32)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_captured(dtype):
    """Forward, backward and steps in a CUDA graph, replayed on new inputs."""
    shape = (2, 200, 1, 2, 40, 48)
    p, other = make(*shape, dtype), make(*shape, dtype, seed=4)
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")

    def work(x):
        leaves = [x[k].detach().requires_grad_(True) for k in LEAVES]
        out = rn.gated_delta(*leaves)
        grads = torch.autograd.grad(out, leaves, (x["do"], x["dlast"]))
        pool = out[1][:, 0].detach().clone()
        return [t.detach() for t in out] + list(grads) + [rn.gated_delta_step(*(x[k][:, 0] for k in LEAVES[:5]), pool, slots), pool]

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
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


FIRST_CALL = """
import torch, recurrent_networks_gb300 as rn
p = [torch.randn(1, 100, 1, 64, device="cuda").to(torch.bfloat16).requires_grad_(True) for _ in range(3)]
g = -torch.rand(1, 100, 1, device="cuda")
o, _ = rn.gated_delta(p[0], p[1] * 0.1, p[2], g, torch.rand_like(g))
o.backward(torch.ones_like(o))
assert all(torch.isfinite(x.grad).all() for x in p)
"""


def test_backward_in_a_fresh_thread():
    """autograd's thread, in which nothing has used the device before."""
    subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, check=True, timeout=600)


def test_matches_differences():
    """The gradient against differences of the kernel's own loss, along a direction.
    fp32: the loss (order 10) is off by at most 2^-24 * (64 + T/4) of its terms, 3e-5;
    the central difference divides it by 2 h = 0.02 and adds h^2 / 6 of a third
    derivative of order 1 to 10: 2e-3 + 2e-4 of a slope of order 10 or more."""
    p = make(1, 70, 1, 2, 24, 20, F32, seed=2)
    got = run(p)[2:]
    g = torch.Generator().manual_seed(0)
    for name, grad in zip(LEAVES, got):
        way = torch.randn(grad.shape, generator=g).cuda()
        way = way / way.norm() if name in ("q", "k") else way * way.shape[-1] ** -0.5 / 10
        way = way + grad / grad.norm()  # not across the slope

        def loss(h):
            o, last = run(dict(p, **{name: p[name] + h * way}), grads=False)
            return ((o.double() * p["do"]).sum() + (last.double() * p["dlast"]).sum()).item()

        slope = (grad.double() * way).sum().item()
        assert abs((loss(0.01) - loss(-0.01)) / 0.02 - slope) <= 5e-3 * max(abs(slope), 10.0), name


def test_step_reports_a_slot_past_the_pool():
    p = make(2, 1, 1, 1, 16, 16, F32)
    args = [p[k][:, 0] for k in LEAVES[:5]]
    pool = torch.randn(3, 1, 16, 16, device="cuda")
    keep = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = rn.gated_delta_step(*args, pool, torch.tensor([3, 1], dtype=torch.int32, device="cuda"), status=status)
    assert (o[0] == 0).all() and torch.equal(pool[0], keep[0]) and torch.equal(pool[2], keep[2])
    with pytest.raises(_lib.RnnError) as err:
        _lib.rnn_check_status(status)
    assert err.value.status == _lib.RNN_ERANGE
    o = rn.gated_delta_step(*(x[:0] for x in args), pool, torch.zeros(0, dtype=torch.int32, device="cuda"), status=status)
    assert o.shape == (0, 1, 16)
    _lib.rnn_check_status(status)


def test_status_words_are_passed_on():
    """What a kernel records in the tape's first word reaches the caller's, forward and backward."""
    for dtype in (F32, BF):
        p = make(1, 70, 1, 1, 16, 16, dtype)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = p["q"].clone().requires_grad_(True)
        o, _ = rn.gated_delta(q, *(p[k] for k in LEAVES[1:]), status=status)
        torch.autograd.grad(o, q, p["do"], retain_graph=True)
        _lib.rnn_check_status(status)
        tape = o.grad_fn.saved_tensors[-1].data  # autograd is not to see the write
        tape[:4].view(torch.int32).fill_(1)  # a wait that ran out
        torch.autograd.grad(o, q, p["do"])
        with pytest.raises(_lib.RnnError) as err:
            _lib.rnn_check_status(status)
        assert err.value.status == _lib.RNN_ETIMEOUT


def test_step_tells_autograd_that_it_writes_the_pool():
    p = make(2, 1, 1, 1, 8, 8, F32)
    args = [p[k][:, 0] for k in LEAVES[:5]]
    pool, other = torch.randn(3, 1, 8, 8, device="cuda"), torch.zeros(3, 1, 8, 8, device="cuda")
    w = torch.ones_like(pool).requires_grad_(True)
    kept = (w * pool).sum()
    rn.gated_delta_step(*args, pool, pool_out=other)
    kept.backward(retain_graph=True)  # the pool was only read
    rn.gated_delta_step(*args, pool)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()


def test_refusals():
    p = make(2, 3, 1, 2, 8, 12, F32)
    q, k, v, g, beta, s = (p[x] for x in LEAVES)
    call = lambda **kw: rn.gated_delta(**{**dict(q=q, k=k, v=v, g=g, beta=beta, state=s), **kw})  # noqa: E731
    pool = torch.zeros(2, 2, 8, 12, device="cuda")
    step = lambda **kw: rn.gated_delta_step(**{**dict(zip("q k v g beta".split(), (x[:, 0] for x in (q, k, v, g, beta)))),  # noqa: E731
                                               "pool": pool, **kw})
    call(), step()
    i64, wide = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, 3, 1, 257, device="cuda")
    bad = [
        lambda: call(q=q[0]), lambda: call(k=k[:, :2]), lambda: call(v=v[:1]), lambda: call(g=g[..., :1]), lambda: call(beta=beta[0]),
        lambda: call(v=v[:, :, :1].expand(2, 3, 3, 12), q=q.expand(2, 3, 2, 8), k=k.expand(2, 3, 2, 8)), lambda: call(q=wide, k=wide),
        lambda: call(q=q[..., :0], k=k[..., :0]), lambda: call(v=v[:, :, :0]), lambda: call(state=s[:, 0]), lambda: call(state=s.cpu()),
        lambda: call(k=k.cpu()), lambda: call(g=g.cpu()), lambda: call(reset=torch.zeros(2, 4, dtype=torch.bool, device="cuda")),
        lambda: call(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), lambda: step(pool=pool[:1]),
        lambda: step(pool=pool[..., :8]), lambda: step(slots=i64), lambda: step(pool_out=torch.zeros(3, 2, 8, 12, device="cuda")),
        lambda: step(q=q), lambda: step(pool=torch.zeros(49 * 8, device="cuda")[1:385].view(2, 2, 8, 12)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(f"call {i} was not refused")
    for f in (lambda: call(q=q.double(), k=k.double()), lambda: call(k=k.to(BF)), lambda: call(v=v.to(BF)), lambda: call(g=g.to(BF)),
              lambda: call(beta=beta.double()), lambda: call(reset=torch.zeros(2, 3, device="cuda")),
              lambda: call(lengths=torch.zeros(2, device="cuda")), lambda: step(pool=pool.to(BF)), lambda: step(q=q[:, 0].to(BF))):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(_lib.RnnError):
        rn.gated_delta(q[:0], k[:0], v[:0], g[:0], beta[:0])


def test_other_derivatives_are_refused():
    """No forward-mode and no second derivative: both raise instead of giving a wrong one."""
    p = make(1, 5, 1, 1, 8, 8, F32)
    args = [p[k] for k in LEAVES]
    for i in range(6):
        for grad in (True, False):
            with forward_ad.dual_level(), torch.set_grad_enabled(grad):
                duals = list(args)
                duals[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(NotImplementedError):
                    rn.gated_delta(*duals)
    leaves = [x.clone().requires_grad_(True) for x in args]
    o, _ = rn.gated_delta(*leaves)
    dq, = torch.autograd.grad(o, leaves[0], p["do"].requires_grad_(True), create_graph=True)
    with pytest.raises(RuntimeError):
        dq.sum().backward()
