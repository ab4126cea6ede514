"""The fp64 oracle of the gated delta rule and the group norm against central
differences and closed forms, and the host-side refusals of their entry points
(CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import delta
from recurrent_networks_gb300 import _lib


def differences(loss, args, got, tol):
    """Central differences: O(1e-10) truncation, 1e-16 / 1e-5 rounding, on values of order 1-10."""
    for k, grad in enumerate(got):
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[k][i] += 1e-5
            lo[k][i] -= 1e-5
            num[i] = (loss(*hi) - loss(*lo)) / 2e-5
        assert np.abs(num - grad).max() < tol, k


@pytest.mark.parametrize("masked", [False, True])
def test_delta_gradients_match_central_differences(masked):
    r = np.random.default_rng(0)
    B, T, Nk, N, Dk, Dv = 2, 7, 2, 4, 3, 2
    args = [r.normal(size=(B, T, Nk, Dk)) * 0.6, r.normal(size=(B, T, Nk, Dk)) * 0.6, r.normal(size=(B, T, N, Dv)),
            -r.random((B, T, N)), r.random((B, T, N)), r.normal(size=(B, 1, N, Dk, Dv))]
    do, dl = r.normal(size=(B, T, N, Dv)), r.normal(size=(B, 1, N, Dk, Dv))
    reset, lengths = None, None
    if masked:
        reset = np.zeros((B, T), dtype=bool)
        reset[0, [0, 4]] = reset[1, 2] = True
        lengths = [7, 5]

    def loss(*args):
        o, last, _ = delta.fwd(*args, 0.7, reset, lengths)
        return (o * do).sum() + (last * dl).sum()

    trail = delta.fwd(*args, 0.7, reset, lengths)[2]
    *got, parts = delta.bwd(*args[:5], trail, do, dl, 0.7)
    differences(loss, args, got, 1e-8)
    both = (parts[:2].sum(0), parts[2:].sum(0))
    for grad, sums in zip(got, both):  # heads n of q and k head n // 2
        assert np.allclose(sums.reshape(B, T, Nk, 2, Dk).sum(3), grad)


def test_delta_closed_forms():
    # beta = 1, unit keys, no decay: the state answers with the last value written at a key
    k = np.eye(3)[[0, 1, 0, 2]][None, :, None]
    v = np.arange(8.0).reshape(1, 4, 1, 2)
    o, last, _ = delta.fwd(k, k, v, np.zeros((1, 4, 1)), np.ones((1, 4, 1)), scale=1.0)
    assert np.allclose(o, v) and np.allclose(last[0, 0, 0], v[0, [2, 1, 3], 0])
    # beta = 0: the state decays and nothing else
    s = np.ones((1, 1, 1, 3, 2))
    _, last, _ = delta.fwd(k, k, v, np.full((1, 4, 1), -0.5), np.zeros((1, 4, 1)), s)
    assert np.allclose(last, np.exp(-2.0))
    # a reset, or a decay of nothing, drops whatever the state holds
    for g, reset in ((0.0, np.ones((1, 4))), (-np.inf, None)):
        o, last, _ = delta.fwd(k, k, v, np.full((1, 4, 1), g), np.ones((1, 4, 1)), np.full_like(s, np.inf), 1.0, reset)
        assert np.allclose(o, v)


@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_match_central_differences(gated, act, centered):
    r = np.random.default_rng(1)
    x, gate, dy = (r.normal(size=(3, 10)) for _ in range(3))
    w, b = r.normal(size=10), r.normal(size=10)

    def loss(x, gate, w, b):
        return (delta.group_norm(x, 2, w, b, gate if gated else None, act, 1e-2, centered) * dy).sum()

    _, dx, dgate, dw, db, _ = delta.group_norm(x, 2, w, b, gate if gated else None, act, 1e-2, centered, dy)
    differences(loss, [x, gate, w, b], [dx, np.zeros_like(x) if dgate is None else dgate, dw, db], 1e-7)
    t = torch.nn.functional.group_norm(torch.tensor(x), 2, torch.tensor(w), torch.tensor(b), 1e-2).numpy()
    if act is None and not gated and centered:
        assert np.allclose(delta.group_norm(x, 2, w, b, None, None, 1e-2), t)


def dims(B=2, T=70, Nk=1, N=2, Dk=40, Dv=24, dtype=torch.bfloat16):
    return _lib.make_delta_dims(B, T, Nk, N, Dk, Dv, dtype)


def test_sizes():
    assert rn._lib.rnn_delta_tape_size(dims(T=0)) >= 256
    for dtype in (torch.bfloat16, torch.float32):
        ok = dims(dtype=dtype)
        assert _lib.rnn_delta_tape_size(ok) >= _lib.rnn_delta_tape_size(ok, False) > 256
        assert _lib.rnn_delta_bwd_workspace_size(ok) > 256
        for bad in (dict(B=0), dict(T=-1), dict(Nk=0), dict(N=0), dict(N=3, Nk=2), dict(Dk=0), dict(Dk=257), dict(Dv=0), dict(Dv=257),
                    dict(T=2**31 - 1), dict(N=65537), dict(B=2**31 - 1), dict(T=2**32 + 3), dict(B=2**32 + 1), dict(N=2**32 + 2)):
            assert _lib.rnn_delta_tape_size(dims(**{"dtype": dtype, **bad})) == 0, bad
            assert _lib.rnn_delta_bwd_workspace_size(dims(**{"dtype": dtype, **bad})) == 0, bad
    assert _lib.rnn_delta_tape_size(dims(dtype=7)) == 0
    size = _lib.rnn_group_norm_workspace_size
    assert size(1000, 4, 128, torch.float32) >= 256 + 2 * 512 * 4 and size(0, 4, 128, torch.bfloat16) > 0
    for bad in ((-1, 4, 8), (1 << 40, 4, 8), (5, 0, 8), (5, 4, 0), (5, 65536, 8), (5, 1, 14337), (5, 2**32 + 1, 8), (5, 1, 2**32 + 8)):
        assert size(*bad, torch.bfloat16) == 0, bad


def test_refusals_before_any_device_work():
    lib, E, S = _lib.load(), _lib.RNN_EINVAL, _lib.RNN_ENOSPC
    P, big = 4096, 1 << 30  # a pointer that is never followed

    def refused(call, good, changes, code=E):
        for i, bad in changes:
            args = list(good)
            args[i] = bad
            assert call(*args) == code, (i, bad)

    d = ctypes.byref(dims())
    fwd = [d, P, P, P, P, P, P, None, None, 1.0, P, P, 1, P, big, None]
    refused(lib.rnn_delta_fwd, fwd, [(0, ctypes.byref(dims(Dk=300))), (0, None), (1, None), (2, None), (3, None), (4, None), (5, None),
                                     (10, None), (13, None)] + [(i, P + 8) for i in (1, 2, 3, 4, 5, 6, 10, 11, 13)] + [(8, P + 2)])
    refused(lib.rnn_delta_fwd, fwd, [(14, 16), (14, _lib.rnn_delta_tape_size(dims()) - 1)], S)
    bwd = [d, P, P, P, None, 1.0, P, big, P, P, P, P, P, P, P, P, P, big, None]
    refused(lib.rnn_delta_bwd, bwd, [(0, ctypes.byref(dims(N=0)))] + [(i, None) for i in (1, 2, 3, 6, 10, 11, 12, 13, 14, 16)] +
            [(i, P + 8) for i in (1, 2, 3, 6, 8, 9, 10, 11, 12, 13, 14, 15, 16)] + [(4, P + 2)])
    refused(lib.rnn_delta_bwd, bwd, [(7, 16), (7, _lib.rnn_delta_tape_size(dims(), False)), (17, 16),
                                     (17, _lib.rnn_delta_bwd_workspace_size(dims()) - 1)], S)
    step = [3, 4, 1, 2, 8, 8, 1, P, P, P, P, P, None, P, P, 1.0, P, None, None]
    refused(lib.rnn_delta_step, step, [(0, -1), (0, 5), (1, 0), (2, 0), (3, 0), (2, 3), (4, 0), (4, 257), (5, 0), (5, 257), (6, 2)] +
            [(i, None) for i in (7, 8, 9, 10, 11, 13, 14, 16)] + [(i, P + 8) for i in (7, 8, 9, 10, 11, 13, 14, 16)] +
            [(12, P + 2), (17, P + 2)])
    many = list(step)
    many[:4] = [1 << 20, 1 << 20, 1, 4096]  # rows, heads and tiles are counted in 32 bits
    assert lib.rnn_delta_step(*many) == E
    norm = [5, 2, 8, 1, 1, 1, 1e-5, P, P, P, P, P, None]
    refused(lib.rnn_group_norm_fwd, norm, [(0, -1), (1, 0), (2, 0), (2, 14337), (3, 5), (4, -1), (4, 3), (6, -1.0), (6, float("nan")), (7, None),
                                           (11, None)] + [(i, P + 8) for i in (7, 8, 9, 10, 11)])
    back = [5, 2, 8, 1, 1, 1, 1e-5, P, P, P, P, P, P, P, P, P, P, big, None]
    refused(lib.rnn_group_norm_bwd, back, [(0, -1), (2, 14337), (4, 3), (6, -1.0)] + [(i, None) for i in (7, 10, 11, 12, 13, 16)] +
            [(i, P + 8) for i in range(7, 17)])
    refused(lib.rnn_group_norm_bwd, back, [(17, 16)], S)


class There(torch.Tensor):
    """A stand-in for a tensor on cuda:1."""
    is_cuda = True

    def get_device(self):
        return 1


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    t = lambda *s: torch.zeros(*s).as_subclass(There)  # noqa: E731
    args = [t(2, 3, 1, 8), t(2, 3, 1, 8), t(2, 3, 1, 8), t(2, 3, 1), t(2, 3, 1)]
    for call in (lambda: rn.gated_delta(*args), lambda: rn.gated_delta_step(*(x[:, 0] for x in args), t(2, 1, 8, 8)),
                 lambda: rn.group_norm(t(2, 8), 2)):
        with pytest.raises(ValueError, match="cuda:1 and the current device is cuda:0"):
            call()


def test_functions_refuse_cpu_tensors():
    x, g = torch.zeros(1, 2, 1, 8), torch.zeros(1, 2, 1)
    for call in (lambda: rn.gated_delta(x, x, x, g, g), lambda: rn.gated_delta_step(x[0], x[0], x[0], g[0], g[0], torch.zeros(2, 1, 8, 8)),
                 lambda: rn.group_norm(x, 2)):
        with pytest.raises(RuntimeError, match="no CPU path"):
            call()


def test_kept_sizes_belong_to_a_device():
    """The sizes follow from the number of SMs; each device keeps its own."""
    args = (1, 4000, 1, 1, 128, 128, torch.bfloat16)
    try:
        for device, sms in ((0, 8), (1, 148)):
            _lib.load().rnn_plan_set_limits(sms, 227 * 1024, 16)
            d = _lib.make_delta_dims(*args)
            assert _lib.delta_plan(*args, device)[1:] == (_lib.rnn_delta_tape_size(d, False), _lib.rnn_delta_tape_size(d),
                                                          _lib.rnn_delta_bwd_workspace_size(d))
            assert (_lib.rnn_group_norm_workspace_size(4000, 4, 64, torch.float32, device) ==
                    _lib.rnn_group_norm_workspace_size(4000, 4, 64, torch.float32))
        assert _lib.delta_plan(*args, 0)[1:] != _lib.delta_plan(*args, 1)[1:]
    finally:
        _lib.rnn_plan_set_limits(0)
