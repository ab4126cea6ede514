"""The fp64 oracle of the gated linear scan against central differences and
closed forms, and the host-side refusals of the new entry points (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import recurrent_networks_gb300 as rn
from oracle import gated
from recurrent_networks_gb300 import _lib


def _problem(function, B=2, T=9, N=2, D=3, seed=0):
    r = np.random.default_rng(seed)
    G = 4 if function == "linear" else 2
    return (r.normal(size=(B, T, G, N, D)), r.normal(size=(G, N, D)), r.normal(size=(B, 1, N, D)),
            r.normal(size=(B, T, N, D)), r.normal(size=(B, 1, N, D)))


@pytest.mark.parametrize("function", ["linear", "linear_coupled"])
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_match_central_differences(function, masked):
    Wx, b, s0, dh, dl = _problem(function)
    reset = np.zeros(Wx.shape[:2], dtype=bool)
    lengths = None
    if masked:
        reset[0, [0, 4]] = True
        reset[1, 7] = True
        lengths = [9, 5]

    def loss(Wx, b, s0):
        h, last, _ = gated.fwd(Wx, b, s0, function, reset, lengths)
        return (h * dh).sum() + (last * dl).sum()

    _, _, before = gated.fwd(Wx, b, s0, function, reset, lengths)
    got = gated.bwd(Wx, b, before, function, dh, dl, reset, lengths)
    args = [Wx, b, s0]
    for k in range(3):
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[k][i] += 1e-5
            lo[k][i] -= 1e-5
            num[i] = (loss(*hi) - loss(*lo)) / 2e-5
        # central differences: O(1e-10) truncation, 1e-16 / 1e-5 rounding, on values of order 1-10
        assert np.abs(num - got[k]).max() < 1e-8


def test_closed_forms():
    # f = 1/2, coupled: c_t is the running half-half average of the candidates
    Wx = np.zeros((1, 4, 2, 1, 1))
    Wx[0, :, 1, 0, 0] = [1, 2, 3, 4]
    h, last, _ = gated.fwd(Wx, None, None, "linear_coupled")
    assert np.allclose(h[0, :, 0, 0], [0.5, 1.25, 2.125, 3.0625]) and last[0, 0, 0, 0] == 3.0625
    # saturated gates keep the state and read nothing
    Wx = np.zeros((1, 3, 4, 1, 1))
    Wx[0, :, 0], Wx[0, :, 1], Wx[0, :, 2], Wx[0, :, 3] = -1e30, 1e30, 7, 1e30
    h, _, _ = gated.fwd(Wx, None, np.full((1, 1, 1, 1), 5.0), "linear")
    assert (h == 5.0).all()


def test_pack_definition():
    x = np.array([[127.0, 1.0, 0.0], [-127.5, 0.5, 0.0]])
    q, s = gated.pack(x)
    assert s.tolist() == [[128, 121, 1]] and q[:, 0].tolist() == [64, -64] and q[:, 1].tolist() == [64, 32]


def _dims(**kw):
    d = dict(B=2, T=3, N=1, D=8, function="linear", dtype=torch.float32, checkpoint=None)
    d.update(kw)
    return _lib.make_gated_dims(**d)


def test_sizes():
    assert _lib.rnn_gated_tape_size(_dims(T=300, D=40)) == -(-2 * 3 * 40 * 4 // 256) * 256
    q = _lib.rnn_gated_tape_size(_dims(T=300, D=40, checkpoint="int8"))
    assert q >= 2 * 3 * 40 * 4 + 2 * 300 * 160 + 2 * 10 * 160
    for bad in (dict(B=0), dict(T=-1), dict(N=0), dict(D=0), dict(function=2), dict(dtype=5), dict(checkpoint=2)):
        assert _lib.rnn_gated_tape_size(_dims(**bad)) == 0
        assert _lib.rnn_gated_workspace_size(_dims(**bad), _lib.WS_FWD) == 0
    assert _lib.rnn_gated_workspace_size(_dims(), 2) == 0
    assert [_lib.rnn_gated_num_gates(f) for f in ("linear", "linear_coupled", "lstm")] == [4, 2, -1]
    assert _lib.rnn_act_scale_bytes(33, 7) == 14 and _lib.rnn_act_scale_bytes(0, 7) == 0
    assert _lib.rnn_act_scale_bytes(1, 0) == 0
    assert _lib.rnn_embed_bwd_workspace_size(10, 0, 8) == 0 and _lib.rnn_embed_bwd_workspace_size(-1, 5, 8) == 0
    assert _lib.rnn_embed_bwd_workspace_size(1 << 31, 5, 8) == 0


def test_refusals_before_any_device_work():
    lib, E = _lib.load(), _lib.RNN_EINVAL
    d, big = ctypes.byref(_dims()), 1 << 20
    P = 4096  # a pointer that is never followed
    assert lib.rnn_gated_fwd(ctypes.byref(_dims(B=0)), P, P, P, None, None, P, P, P, P, big, None) == E
    assert lib.rnn_gated_fwd(d, None, P, P, None, None, P, P, P, P, big, None) == E
    assert lib.rnn_gated_fwd(d, P, P, P, None, None, None, P, P, P, big, None) == E
    assert lib.rnn_gated_fwd(d, P + 8, P, P, None, None, P, P, P, P, big, None) == E
    assert lib.rnn_gated_fwd(d, P, P, P, None, P + 2, P, P, P, P, big, None) == E
    assert lib.rnn_gated_fwd(d, P, P, P, None, None, P, P, P, None, big, None) == E
    assert lib.rnn_gated_fwd(d, P, P, P, None, None, P, P, P, P, 16, None) == _lib.RNN_ENOSPC
    assert lib.rnn_gated_bwd(d, P, P, None, None, None, P, P, P, P, P, P, big, None) == E  # no tape
    assert lib.rnn_gated_bwd(d, None, P, None, None, P, P, P, P, P, P, P, big, None) == E  # no Wx
    assert lib.rnn_gated_bwd(d, P, P, None, None, P, P, P, P + 4, P, P, P, big, None) == E
    assert lib.rnn_gated_bwd(d, P, P, None, None, P, P, P, P, P, P, P, 16, None) == _lib.RNN_ENOSPC
    step = [3, 4, 1, 8, 0, 0, P, P, P, P, P, P, None, None]

    def with_(**kw):
        v = list(step)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return lib.rnn_gated_step(*v)

    assert with_(a0=-1) == E and with_(a1=0) == E and with_(a4=2) == E and with_(a5=3) == E and with_(a6=None) == E
    assert with_(a9=None) == E and with_(a10=None) == E and with_(a11=P + 4) == E and with_(a8=P + 2) == E
    assert with_(a0=5, a8=None) == E  # more rows than slots, and no slot list
    assert lib.rnn_act_pack(4, 0, 0, P, P, P, None) == E and lib.rnn_act_pack(4, 4, 2, P, P, P, None) == E
    assert lib.rnn_act_pack(4, 4, 0, P, None, P, None) == E and lib.rnn_act_unpack(4, 4, 0, P + 1, P, P, None) == E
    assert lib.rnn_embed_fwd(4, 5, 8, 0, 3, P, P, 1.0, P, None, None) == E
    assert lib.rnn_embed_fwd(4, 5, 8, 0, 8, P + 4, P, 1.0, P, None, None) == E
    assert lib.rnn_embed_fwd(4, 5, 8, 0, 4, None, P, 1.0, P, None, None) == E
    assert lib.rnn_embed_bwd(4, 5, 8, 0, 4, P, -1, P, 1.0, None, P, big, None) == E
    assert lib.rnn_embed_bwd(4, 5, 8, 0, 4, P, -1, P, 1.0, P, P, 16, None) == _lib.RNN_ENOSPC
    assert _lib.rnn_strerror(_lib.RNN_ERANGE) == "a token or slot index is out of range"


def test_functions_refuse_cpu_tensors():
    import recurrent_networks_gb300 as rn
    x = torch.zeros(1, 2, 4, 1, 8)
    for call in (lambda: rn.gated_scan(x), lambda: rn.gated_scan_step(x[0], None, torch.zeros(2, 1, 8)),
                 lambda: rn.checkpoint_pack(x), lambda: rn.checkpoint_unpack(x, x),
                 lambda: rn.embedding(torch.zeros(2, dtype=torch.int64), x[0, 0, 0])):
        with pytest.raises(RuntimeError, match="no CPU path"):
            call()


def test_sizes_past_32_bits_are_refused():
    """Neither the low bits of a longer size nor an overflow on the way to it."""
    for bad in (dict(T=2**32 + 3), dict(B=2**32 + 1), dict(N=2**32 + 1), dict(D=2**32 + 8), dict(B=1, T=2**31 - 1, D=1)):
        assert _lib.rnn_gated_tape_size(_dims(**bad)) == 0
        assert _lib.rnn_gated_workspace_size(_dims(**bad), _lib.WS_FWD) == 0
    assert _lib.rnn_gated_tape_size(_dims(B=1, T=2**31 - 129, D=1)) >= (2**31 - 129) // 128 * 4
    for cols in (2**32 + 8, 2**31 - 1):
        assert _lib.rnn_act_scale_bytes(1, cols) == 0
    assert _lib.rnn_act_scale_bytes(1, 2**31 - 65) == 2**31 - 65
    for V, E in ((2**32 + 5, 8), (5, 2**32 + 8), (5, 2**31 - 1)):
        assert _lib.rnn_embed_bwd_workspace_size(10, V, E) == 0
    assert _lib.rnn_embed_bwd_workspace_size(10, 5, 2**30) > 0
    x = torch.zeros(64)  # refused before it is followed
    for call in (lambda: _lib.rnn_gated_step(2**32 + 1, 4, 1, 8, "linear", torch.float32, x, None, None, x, x, x, stream=0),
                 lambda: _lib.rnn_act_pack(1, 2**32 + 8, x, x, x, stream=0),
                 lambda: _lib.rnn_act_unpack(1, 2**32 + 8, x, x, x, stream=0),
                 lambda: _lib.rnn_embed_fwd(4, 2**32 + 5, 8, x, x, 1.0, x, stream=0),
                 lambda: _lib.rnn_embed_bwd(4, 2**32 + 5, 8, x, -1, x, 1.0, x, x, stream=0)):
        with pytest.raises(_lib.RnnError) as err:
            call()
        assert err.value.status == _lib.RNN_EINVAL


class There(torch.Tensor):
    """A stand-in for a tensor on cuda:1."""
    is_cuda = True

    def get_device(self):
        return 1


def there(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(There)


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """The library launches on the current device; a call on another device's
    tensors must not reach it (the devices are stand-ins: no GPU is needed)."""
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    x, i8, u8, ids = there(2, 3, 4, 1, 8), there(4, 8, dtype=torch.int8), there(1, 8, dtype=torch.uint8), there(3, dtype=torch.int64)
    for call in (lambda: rn.flashrnn(there(2, 3, 4, 1, 8), there(4, 1, 8, 8), there(4, 1, 8)),
                 lambda: rn.input_projection(there(3, 64), there(64, 64)),
                 lambda: rn.gated_scan(x), lambda: rn.gated_scan_step(x[:, 0], None, there(2, 1, 8)),
                 lambda: rn.checkpoint_pack(there(4, 8)), lambda: rn.checkpoint_unpack(i8, u8),
                 lambda: rn.embedding(ids, there(5, 8)),
                 lambda: _lib.rnn_gated_fwd(_dims(), x, None, None, None, None, x, None, None, x),
                 lambda: _lib.rnn_gated_bwd(_dims(), x, None, None, None, x, None, None, None, None, None, x),
                 lambda: _lib.rnn_gated_step(2, 2, 1, 8, "linear", torch.float32, x, None, None, x, x, x),
                 lambda: _lib.rnn_act_pack(1, 8, x, i8, u8), lambda: _lib.rnn_act_unpack(1, 8, i8, u8, x),
                 lambda: _lib.rnn_embed_fwd(3, 5, 8, ids, x, 1.0, x),
                 lambda: _lib.rnn_embed_bwd(3, 5, 8, ids, -1, x, 1.0, x, x)):
        with pytest.raises(ValueError, match="cuda:1 and the current device is cuda:0"):
            call()


def test_kept_sizes_belong_to_a_device(monkeypatch):
    """With the number of SMs that the library plans for changed in between, as
    another current device would change it, each device keeps its own sizes."""
    args = (1, 4000, 1, 64, "linear", torch.float32, None)
    try:
        for device, sms in ((0, 8), (1, 148)):
            _lib.load().rnn_plan_set_limits(sms, 227 * 1024, 16)
            assert _lib.gated_plan(*args, device)[2] == _lib.rnn_gated_workspace_size(_lib.make_gated_dims(*args))
            assert (_lib.rnn_embed_bwd_workspace_size(4000, 50, 64, device) ==
                    _lib.load().rnn_embed_bwd_workspace_size(4000, 50, 64))
        assert _lib.gated_plan(*args, 0)[2] != _lib.gated_plan(*args, 1)[2]
        assert _lib.rnn_embed_bwd_workspace_size(4000, 50, 64, 0) != _lib.rnn_embed_bwd_workspace_size(4000, 50, 64, 1)
    finally:
        _lib.rnn_plan_set_limits(0)


def test_status_words_that_the_kernels_cannot_write_are_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    i32 = torch.int32
    for status, error in ((torch.zeros(1, dtype=i32), ValueError), (there(1), TypeError),
                          (there(1, dtype=torch.int64), TypeError), (there(0, dtype=i32), ValueError)):
        for call in (lambda: rn.gated_scan_step(there(2, 4, 1, 8), None, there(2, 1, 8), status=status),
                     lambda: rn.gated_scan(there(2, 3, 4, 1, 8), status=status),
                     lambda: rn.embedding(there(3, dtype=torch.int64), there(5, 8), status=status)):
            with pytest.raises(error, match="status"):
                call()


def test_calls_give_up_the_interpreter_lock():
    """A launch can wait for the stream's queue, and the queue for a host callback that needs the lock."""
    lib = _lib._quick()
    for name in _lib.EXPORTS:
        assert not getattr(lib, name)._flags_ & ctypes.PyDLL._func_flags_ & ~ctypes.CDLL._func_flags_, name
