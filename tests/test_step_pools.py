"""A step's pool_out is the pool itself or shares no memory with it: states are
read and written in no order. Refused before any device work; CPU."""
import pytest
import torch

from recurrent_networks_gb300 import _lib, functional


def test_entry_points():
    lib, P, slots = _lib.load(), 4096, 4  # a pointer that is never followed
    gated = lambda out, rows: lib.rnn_gated_step(rows, slots, 1, 8, 0, 0, P, P, P, P, out, P, None, None)  # noqa: E731
    delta = lambda out, rows: lib.rnn_delta_step(rows, slots, 1, 2, 8, 8, 1, P, P, P, P, P, None, P, out, 1.0, P, None, None)  # noqa: E731
    for call, size in ((gated, slots * 8 * 4), (delta, slots * 2 * 64 * 4)):
        for off in (16, size // 2, size - 16):
            assert call(P + off, 3) == _lib.RNN_EINVAL and call(P - off, 3) == _lib.RNN_EINVAL
        for out in (P, P + size, P - size):  # no rows: nothing is launched
            assert call(out, 0) == _lib.RNN_OK


def test_functions():
    memory = torch.zeros(7, 2, 8, 8)
    check = lambda a, b: functional._check_pool((a, b), None, 3, (2, 8, 8), "N,Dk,Dv", memory, "q")  # noqa: E731
    for a, b in ((0, 1), (1, 0), (3, 0), (0, 3)):
        with pytest.raises(ValueError, match="memory"):
            check(memory[a:a + 4], memory[b:b + 4])
    assert check(memory[:4], memory[:4]) == 4 and check(memory[:3], memory[3:6]) == 3 and check(memory[4:], memory[:3]) == 3
