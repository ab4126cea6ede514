"""GPU parity of the gated linear scan (forward, backward, single-token step,
8-bit checkpoint) with its fp64 oracle, and its refusals.

Tolerances. bf16: every output is rounded once (2^-9 relative per element);
the fp32 arithmetic inside is at most 2^-22 a step relative, over at most a
few hundred steps, so L2-normwise 5e-3 and normwise-max 1e-2 as for the other
bf16 outputs. fp32: a step's f carries a relative error of at most about
2^-22 (exponential, sum, division, product), products of up to T of them
T 2^-22: normwise-max 1e-6 + T 2^-22. The carried state and the gradient of
the initial state are fp32 for either dtype; with bf16 inputs the faster
exponential and reciprocal (2^-21 together) take the place: 1e-6 + T 2^-20."""
import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import recurrent_networks_gb300 as rn
from oracle import gated
from recurrent_networks_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def close(got, ref, what, T, fp32, fast=False):
    got = got.detach().double().cpu().numpy()
    ref = np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    top = max(np.abs(ref).max(), 1e-30)
    worst = np.abs(got - ref).max() / top
    if fp32:
        tol = 1e-6 + T * 2.0 ** (-20 if fast else -22)
        assert worst <= tol, f"{what}: max {worst:.3g} > {tol:.3g}"
    else:
        l2 = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
        assert l2 <= 5e-3 and worst <= 1e-2, f"{what}: L2 {l2:.3g}, max {worst:.3g}"


def make(function, B, T, N, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + D)
    G = 4 if function == "linear" else 2
    Wx = torch.randn(B, T, G, N, D, generator=g).to(dtype).cuda()
    b = torch.randn(G, N, D, generator=g)
    b[G // 2 - 1] += 3  # the forget gate: long memories
    return dict(Wx=Wx, b=b.to(dtype).cuda(), state=torch.randn(B, 1, N, D, generator=g).cuda(),
                dh=torch.randn(B, T, N, D, generator=g).to(dtype).cuda(),
                dlast=torch.randn(B, 1, N, D, generator=g).cuda())


def run(p, function, reset=None, lengths=None, checkpoint=None, grads=True):
    leaves = [p[k].clone().requires_grad_(grads) for k in ("Wx", "b", "state")]
    h, last = rn.gated_scan(*leaves, function=function, reset=reset, lengths=lengths, checkpoint=checkpoint)
    if not grads:
        return h, last
    return (h, last) + torch.autograd.grad((h, last), leaves, (p["dh"], p["dlast"]))


def check(p, function, reset=None, lengths=None, checkpoint=None):
    dtype, T = p["Wx"].dtype, p["Wx"].shape[1]
    got = run(p, function, reset, lengths, checkpoint)
    h, last, before = gated.fwd(p["Wx"], p["b"], p["state"], function, reset, lengths)
    ref = (h, last) + gated.bwd(p["Wx"], p["b"], before, function, p["dh"], p["dlast"], reset, lengths,
                                packed=checkpoint is not None)
    for name, a, r in zip(("h", "last", "dWx", "db", "dstate"), got, ref):
        state = name in ("last", "dstate")
        close(a, r, name, T, state or dtype == F32, fast=dtype == BF)
    return got


# (B, T, N, D): one step; one channel; odd widths (no 4-, 8- or 16-byte rows);
# one chunk of 128 steps, one step more and one less; several chunks; several
# 64-channel tiles, a ragged one; enough chunks for the states to pass between
# many blocks
SHAPES = [(1, 1, 1, 1), (2, 16, 1, 32), (3, 5, 2, 17), (1, 127, 1, 9), (2, 128, 1, 64), (2, 129, 3, 22),
          (1, 1000, 1, 130), (2, 515, 1, 200), (1, 5003, 1, 36), (2, 300, 1, 115), (1, 260, 1, 174)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dT%dN%dD%d" % s)
def test_parity(shape, function, dtype):
    check(make(function, *shape, dtype), function)


@pytest.mark.parametrize("checkpoint", [None, "int8"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("shape", [(4, 70, 1, 33), (5, 300, 2, 40), (4, 1100, 1, 64)], ids=lambda s: "B%dT%dN%dD%d" % s)
def test_masks(shape, function, dtype, checkpoint):
    B, T = shape[:2]
    p = make(function, *shape, dtype, seed=3)
    g = torch.Generator().manual_seed(T)
    reset = torch.rand(B, T, generator=g) < 0.05
    reset[0, 0] = True
    reset[1] = True  # every step its own document
    lengths = torch.tensor([T, T - 1, 0, T // 2, 1][:B], dtype=torch.int32)
    clean = check(p, function, reset.cuda(), lengths.cuda(), checkpoint)
    # whatever stands past a row's length must not matter
    dirty = {k: v.clone() for k, v in p.items()}
    for i in range(B):
        n = int(lengths[i])
        dirty["Wx"][i, n:] = float("nan")
        dirty["dh"][i, n:] = float("inf")
    again = run(dirty, function, reset.cuda(), lengths.cuda(), checkpoint)
    for a, b in zip(clean, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 40, 1, 24), (1, 321, 2, 65), (2, 260, 1, 128)], ids=lambda s: "B%dT%dN%dD%d" % s)
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
def test_int8_checkpoint(shape, function, dtype):
    p = make(function, *shape, dtype, seed=5)
    got = check(p, function, checkpoint="int8")
    plain = run(p, function)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])  # the forward is the same


def test_reset_drops_an_infinite_state():
    p = make("linear", 1, 200, 1, 64, F32)
    p["state"].fill_(float("inf"))
    reset = torch.zeros(1, 200, dtype=torch.bool, device="cuda")
    reset[0, 0] = True
    h, last = run(p, "linear", reset=reset, grads=False)
    assert torch.isfinite(h).all() and torch.isfinite(last).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
def test_nan_stays_until_a_reset(function, dtype):
    """A NaN in a gate that is looked at reaches every later step of its channel
    (also through factors that underflow) and no other channel, up to a reset;
    backward it reaches the earlier steps of its document alone."""
    p = make(function, 1, 400, 1, 70, dtype)
    f = 1 if function == "linear" else 0
    p["Wx"][0, :, f] = -12  # f = 6e-6: a few steps' product underflows
    p["Wx"][0, 150, f, 0, 33] = float("nan")
    reset = torch.zeros(1, 400, dtype=torch.bool, device="cuda")
    reset[0, [100, 300]] = True
    h, last, dWx, _, ds = run(p, function, reset=reset)
    bad = torch.isnan(h[0, :, 0])
    want = torch.zeros_like(bad)
    want[150:300, 33] = True
    assert torch.equal(bad, want)
    assert torch.isfinite(last).all() and torch.isfinite(ds).all()
    bad = torch.isnan(dWx[0, :, :, 0]).any(1)
    assert not bad[:100].any() and not bad[300:].any()
    assert bad[100:300, 33].all() and bad.sum() == 200


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("T,nan,resets", [
    (400, 150, [200]), (400, 200, [150]),  # one chunk of 128 steps, different warps of 16
    (400, 148, [155]), (400, 155, [148]),  # one warp
    (400, 10, [60, 300]), (400, 390, [395]), (100, 20, [60]), (100, 60, [20]), (100, 18, [25]), (100, 25, [18])])
def test_nan_keeps_to_its_document(T, nan, resets, function, dtype):
    """As above with the NaN and a reset in the same chunk, in both orders: what
    is NaN is the NaN's channel from its step to the end of its document, and the
    gradients of that document's steps of the channel."""
    g = torch.Generator().manual_seed(T + nan)
    G, C, ch = 4 if function == "linear" else 2, 70, 33
    Wx = torch.randn(2, T, G, 1, C, generator=g)
    Wx[1, nan, G // 2 - 1, 0, ch] = torch.tensor(float("nan")).copysign(torch.tensor(0.5 - nan % 2))  # the forget gate
    leaves = [Wx.to(dtype).cuda(), torch.randn(G, 1, C, generator=g).to(dtype).cuda(),
              torch.randn(2, 1, 1, C, generator=g).cuda()]
    leaves = [x.requires_grad_(True) for x in leaves]
    reset = torch.zeros(2, T, dtype=torch.bool)
    reset[1, resets] = True
    h, last = rn.gated_scan(*leaves, function=function, reset=reset.cuda())
    dWx, _, ds = torch.autograd.grad((h, last), leaves, (torch.ones_like(h), torch.ones_like(last)))
    begin, end = max([0] + [r for r in resets if r <= nan]), min([T] + [r for r in resets if r > nan])

    def only(steps, on=True):
        want = torch.zeros(2, *steps, C, dtype=torch.bool)
        want[1, ..., ch] = on
        return want

    t = torch.arange(T)
    assert torch.equal(torch.isnan(h[:, :, 0]).cpu(), only((T,), (t >= nan) & (t < end)))
    assert torch.equal(torch.isnan(last[:, 0, 0]).cpu(), only((), end == T))
    assert torch.equal(torch.isnan(dWx[:, :, :, 0]).any(2).cpu(), only((T,), (t >= begin) & (t < end)))
    assert torch.equal(torch.isnan(ds[:, 0, 0]).cpu(), only((), begin == 0))


def test_saturated_gates():
    """Logits of +-inf and of the types' lowest value: gates exactly 0 or 1."""
    for dtype in (F32, BF):
        for low in (float("-inf"), torch.finfo(dtype).min):
            Wx = torch.zeros(1, 300, 4, 1, 64, dtype=dtype, device="cuda")
            Wx[:, :, 0] = low   # nothing read
            Wx[:, :, 1] = -low  # everything kept
            Wx[:, :, 2] = 1000
            Wx[:, :, 3] = -low
            s = torch.full((1, 1, 1, 64), 3.0, device="cuda")
            Wx.requires_grad_(True)
            h, last = rn.gated_scan(Wx, None, s)
            assert (h == 3).all() and (last == 3).all()
            (d,) = torch.autograd.grad(h.float().sum(), Wx)
            assert (d == 0).all()


def test_no_steps_and_optional_arguments():
    for dtype in (F32, BF):
        Wx = torch.randn(2, 0, 4, 1, 8, device="cuda").to(dtype).requires_grad_(True)
        b = torch.randn(4, 1, 8, device="cuda").to(dtype).requires_grad_(True)
        s = torch.randn(2, 1, 1, 8, device="cuda", requires_grad=True)
        h, last = rn.gated_scan(Wx, b, s)
        assert h.shape == (2, 0, 1, 8) and torch.equal(last, s)
        dl = torch.randn_like(last)
        dx, db, ds = torch.autograd.grad(last, (Wx, b, s), dl)
        assert dx.shape == Wx.shape and (db == 0).all() and torch.equal(ds, dl)
        h, last = rn.gated_scan(Wx)
        assert (last == 0).all()
    p = make("linear", 2, 150, 1, 40, F32)
    zero_b, zero_s = torch.zeros_like(p["b"]), torch.zeros_like(p["state"])
    h, last = rn.gated_scan(p["Wx"])
    h2, last2 = rn.gated_scan(p["Wx"], zero_b, zero_s)
    assert torch.equal(h, h2) and torch.equal(last, last2)
    # the gradient of one output alone, of one input alone
    x = p["Wx"].clone().requires_grad_(True)
    h, last = rn.gated_scan(x, p["b"], p["state"])
    (d,) = torch.autograd.grad(last, x, p["dlast"])
    _, _, before = gated.fwd(p["Wx"], p["b"], p["state"], "linear")
    close(d, gated.bwd(p["Wx"], p["b"], before, "linear", None, p["dlast"])[0], "dWx of last", 150, True)
    s = p["state"].clone().requires_grad_(True)
    h, last = rn.gated_scan(p["Wx"], p["b"], s)
    (d,) = torch.autograd.grad(h, s, p["dh"])
    close(d, gated.bwd(p["Wx"], p["b"], before, "linear", p["dh"], None)[2], "dstate of h", 150, True)


def test_strided_and_misaligned_inputs():
    p = make("linear", 2, 140, 2, 24, BF)
    ref = run(p, "linear")
    wide = torch.empty(2, 140, 4, 2, 48, dtype=BF, device="cuda")
    wide[..., ::2] = p["Wx"]
    raw = torch.empty(p["b"].numel() + 1, dtype=BF, device="cuda")
    raw[1:] = p["b"].reshape(-1)
    q = dict(p, dh=p["dh"].transpose(2, 3).contiguous().transpose(2, 3))
    leaves = [wide[..., ::2].requires_grad_(True), raw[1:].reshape(p["b"].shape).requires_grad_(True),
              p["state"].clone().requires_grad_(True)]
    h, last = rn.gated_scan(*leaves)
    got = (h, last) + torch.autograd.grad((h, last), leaves, (q["dh"], q["dlast"]))
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_repeatable_and_independent_of_the_batch():
    """The same bits on every run, and for a row whatever rows it runs with."""
    for shape in ((6, 900, 1, 192), (1, 20000, 1, 40)):
        p = make("linear", *shape, BF)
        a, b = run(p, "linear"), run(p, "linear")
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # 32 chunks of 128 steps, in groups that depend on the number of rows
    for dtype, function in ((BF, "linear"), (F32, "linear_coupled")):
        p = make(function, 40, 4000, 1, 192, dtype)
        a = run(p, function)
        for rows in (slice(2, 3), slice(1, 9)):
            part = {k: v[rows].contiguous() if k != "b" else v for k, v in p.items()}
            b = run(part, function)
            for k in (0, 1, 2, 4):  # all but db, which sums over the rows
                assert torch.equal(b[k], a[k][rows])


def test_continues_from_its_last_state():
    p = make("linear", 2, 300, 1, 64, F32)
    h, last = run(p, "linear", grads=False)
    h1, s = rn.gated_scan(p["Wx"][:, :131].contiguous(), p["b"], p["state"])
    h2, l2 = rn.gated_scan(p["Wx"][:, 131:].contiguous(), p["b"], s)
    close(torch.cat([h1, h2], 1), h.double().cpu().numpy(), "h in two calls", 300, True)
    close(l2, last.double().cpu().numpy(), "last in two calls", 300, True)


def test_on_another_stream():
    p = make("linear", 2, 700, 1, 96, BF)
    ref = run(p, "linear")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(p, "linear")
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("M,P,N,D", [(1, 1, 1, 1), (3, 5, 2, 17), (64, 80, 1, 256), (5, 9, 3, 22)])
def test_step(M, P, N, D, function, dtype):
    p = make(function, M, 1, N, D, dtype, seed=11)
    g = torch.Generator().manual_seed(M)
    pool = torch.randn(P, N, D, generator=g).cuda()
    slots = torch.randperm(P, generator=g)[:M].to(torch.int32)
    if M > 2:
        slots[1] = -1
    keep = pool.clone()
    out = keep.clone()
    h = rn.gated_scan_step(p["Wx"][:, 0], p["b"], pool, slots.cuda(), function, pool_out=out)
    assert torch.equal(pool, keep)
    ref_pool = keep.double().cpu().numpy()
    ref_h = np.zeros((M, N, D))
    for m in range(M):
        s = int(slots[m])
        if s >= 0:
            r, last, _ = gated.fwd(p["Wx"][m:m + 1], p["b"], keep[s][None, None], function)
            ref_h[m], ref_pool[s] = r[0, 0], last[0, 0]
    close(h, ref_h, "h", 1, dtype == F32, fast=dtype == BF)
    close(out, ref_pool, "pool", 1, True, fast=dtype == BF)
    h2 = rn.gated_scan_step(p["Wx"][:, 0], p["b"], pool, slots.cuda(), function)  # in place
    assert torch.equal(h, h2) and torch.equal(pool, out)


def test_waits_that_run_out_are_reported():
    """A wait in the pass of the state that nothing ends runs out, forward and
    backward; the status word tells, and everything else went on as it should."""
    for function, dtype, shape in (("linear", BF, (2, 900, 1, 64)), ("linear_coupled", F32, (1, 400, 1, 33))):
        B, T, N, D = shape
        p = make(function, *shape, dtype)
        dims = _lib.make_gated_dims(B, T, N, D, function, dtype)
        ws = [torch.empty(_lib.rnn_gated_workspace_size(dims, k), dtype=torch.uint8, device="cuda")
              for k in (_lib.WS_FWD, _lib.WS_BWD)]

        def passes():
            h, last = torch.empty_like(p["dh"]), torch.empty_like(p["state"])
            tape = torch.empty(_lib.rnn_gated_tape_size(dims), dtype=torch.uint8, device="cuda")
            dWx, db, ds = (torch.empty_like(p[k]) for k in ("Wx", "b", "state"))
            _lib.rnn_gated_fwd(dims, p["Wx"], p["b"], p["state"], None, None, h, last, tape, ws[0])
            _lib.rnn_gated_bwd(dims, p["Wx"], p["b"], None, None, tape, p["dh"], p["dlast"], dWx, db, ds, ws[1])
            return h, last, dWx, db, ds

        ref = passes()
        for w in ws:
            _lib.rnn_check_status(w)
        _lib.rnn_debug_inject_wait(1, 2_000_000)  # 2 ms
        try:
            got = passes()
        finally:
            _lib.rnn_debug_inject_wait(-1)
        for w in ws:
            with pytest.raises(_lib.RnnError) as err:
                _lib.rnn_check_status(w)
            assert err.value.status == _lib.RNN_ETIMEOUT
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(passes(), ref))
        for w in ws:
            _lib.rnn_check_status(w)


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_time_outs_reach_the_callers_status_word(checkpoint):
    p = make("linear", 2, 700, 1, 64, BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def told():
        try:
            _lib.rnn_check_status(status)
        except _lib.RnnError as e:
            return e.status == _lib.RNN_ETIMEOUT
        return False

    def scan(grad, inject):
        x = p["Wx"].clone().requires_grad_(grad)
        _lib.rnn_debug_inject_wait(1 if inject else -1, 2_000_000)
        try:
            return x, rn.gated_scan(x, p["b"], p["state"], checkpoint=checkpoint, status=status)[0]
        finally:
            _lib.rnn_debug_inject_wait(-1)

    for grad in (False, True):
        scan(grad, False)
        assert not told()
        scan(grad, True)
        assert told() and not told()  # read and cleared
    x, h = scan(True, False)
    torch.autograd.grad(h, x, p["dh"], retain_graph=True)
    assert not told()
    _lib.rnn_debug_inject_wait(1, 2_000_000)
    try:
        torch.autograd.grad(h, x, p["dh"])
    finally:
        _lib.rnn_debug_inject_wait(-1)
    assert told()


@pytest.mark.parametrize("checkpoint", [None, "int8"])
@pytest.mark.parametrize("T", [1, 10, 700])
def test_what_a_training_forward_keeps(T, checkpoint):
    """Between forward and backward: the tape, and Wx itself unless its 8-bit copy is in the tape."""
    Wx = torch.randn(16, T, 4, 1, 512, device="cuda").to(BF).requires_grad_(True)
    b = torch.randn(4, 1, 512, device="cuda").to(BF).requires_grad_(True)
    h, _ = rn.gated_scan(Wx, b, checkpoint=checkpoint)
    kept = sum(t.numel() * t.element_size() for t in h.grad_fn.saved_tensors if t is not None and t is not b)
    tape = _lib.rnn_gated_tape_size(_lib.make_gated_dims(16, T, 1, 512, "linear", BF, checkpoint))
    assert kept <= tape + (0 if checkpoint else Wx.numel() * 2) + b.numel() * 2


def test_steps_follow_the_scan():
    p = make("linear", 3, 20, 2, 40, F32)
    h, last = run(p, "linear", grads=False)
    pool = p["state"][:, 0].clone()
    hs = torch.stack([rn.gated_scan_step(p["Wx"][:, t], p["b"], pool) for t in range(20)], 1)
    close(hs, h.double().cpu().numpy(), "h by steps", 20, True)
    close(pool, last[:, 0].double().cpu().numpy(), "state by steps", 20, True)


def test_step_reports_a_slot_past_the_pool():
    p = make("linear", 2, 1, 1, 16, F32)
    pool = torch.randn(3, 1, 16, device="cuda")
    keep = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    h = rn.gated_scan_step(p["Wx"][:, 0], p["b"], pool, slots, status=status)
    assert (h[0] == 0).all() and torch.equal(pool[0], keep[0]) and torch.equal(pool[2], keep[2])
    with pytest.raises(_lib.RnnError) as err:
        _lib.rnn_check_status(status)
    assert err.value.status == _lib.RNN_ERANGE
    _lib.rnn_check_status(status)  # read and cleared


def test_refusals():
    p = make("linear", 2, 3, 1, 8, F32)
    Wx, b, s = p["Wx"], p["b"], p["state"]
    pool = torch.zeros(2, 1, 8, device="cuda")
    bad = [
        lambda: rn.gated_scan(Wx, b, function="lstm"), lambda: rn.gated_scan(Wx, b, function="linear_coupled"),
        lambda: rn.gated_scan(Wx[0], b), lambda: rn.gated_scan(Wx, b[0]), lambda: rn.gated_scan(Wx, b, s[:1]),
        lambda: rn.gated_scan(Wx, b, reset=torch.zeros(2, 4, dtype=torch.bool, device="cuda")),
        lambda: rn.gated_scan(Wx, b, lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: rn.gated_scan(Wx, b, checkpoint="int4"), lambda: rn.gated_scan(Wx, b, s.cpu()),
        lambda: rn.gated_scan_step(Wx[:, 0], b, pool[:1]), lambda: rn.gated_scan_step(Wx[:, 0], b, pool[..., :4]),
        lambda: rn.gated_scan_step(Wx[:, 0], b, pool, torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: rn.gated_scan_step(Wx[:, 0], b, pool, pool_out=torch.zeros(3, 1, 8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rn.gated_scan(Wx.double(), b), lambda: rn.gated_scan(Wx, b.to(BF)),
                 lambda: rn.gated_scan(Wx, b, reset=torch.zeros(2, 3, device="cuda")),
                 lambda: rn.gated_scan(Wx, b, lengths=torch.zeros(2, device="cuda")),
                 lambda: rn.gated_scan_step(Wx[:, 0], b, pool.to(BF))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(_lib.RnnError):
        rn.gated_scan(Wx[:0], b)


def test_forward_mode_is_refused():
    """The operators have no forward-mode derivative: a dual tensor raises, also
    where no gradient is asked for, and does not lose its tangent."""
    args = [torch.randn(1, 5, 4, 1, 8, device="cuda"), torch.randn(4, 1, 8, device="cuda"),
            torch.randn(1, 1, 1, 8, device="cuda")]
    for k in range(3):
        for grad in (True, False):
            with forward_ad.dual_level(), torch.set_grad_enabled(grad):
                duals = list(args)
                duals[k] = forward_ad.make_dual(args[k], torch.ones_like(args[k]))
                with pytest.raises(NotImplementedError):
                    rn.gated_scan(*duals)
                rn.gated_scan(*args)
    # forward over reverse
    x = args[0].clone().requires_grad_(True)
    with forward_ad.dual_level():
        h, last = rn.gated_scan(x, *args[1:])
        for out in (h, last):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(out, x, forward_ad.make_dual(torch.ones_like(out), torch.ones_like(out)),
                                    retain_graph=True)


def test_step_tells_autograd_that_it_writes_the_pool():
    Wx, pool, other = torch.randn(2, 4, 1, 8, device="cuda"), torch.randn(3, 1, 8, device="cuda"), torch.zeros(3, 1, 8, device="cuda")
    w = torch.ones(3, 1, 8, device="cuda", requires_grad=True)
    rn.gated_scan_step(Wx, None, pool)
    kept = (w * pool).sum()  # saves the pool
    rn.gated_scan_step(Wx, None, pool, pool_out=other)
    kept.backward(retain_graph=True)  # the pool was only read
    rn.gated_scan_step(Wx, None, pool)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()
    kept = (w * other).sum()
    rn.gated_scan_step(Wx, None, pool, pool_out=other)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()
    with torch.inference_mode():  # a pool without a version, also outside
        pool = torch.randn(3, 1, 8, device="cuda")
        rn.gated_scan_step(Wx, None, pool)
    rn.gated_scan_step(Wx, None, pool)
