"""What stands in a tape, a workspace or an output before a call does not matter:
the delta rule and the group norm on memory filled with 0xFF bytes (a NaN in every
type) give the bits that they give on zeros."""
import pytest
import torch

from recurrent_networks_gb300 import _lib
from test_gpu_delta import BF, F32, LEAVES, make

pytestmark = pytest.mark.gpu


def run(p, fill, lengths, reset, keep=True):
    """Forward (and backward) through the library's entry points, every buffer filled first."""
    B, T, Nk, Dk = p["q"].shape
    N, Dv = p["v"].shape[2:]
    dims = _lib.make_delta_dims(B, T, Nk, N, Dk, Dv, p["q"].dtype)

    def memory(shape, dtype=torch.uint8):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        t.view(-1).view(torch.uint8).fill_(fill)
        return t

    q, k, v, g, beta, state = (p[x] for x in LEAVES)
    o, last = memory(v.shape, v.dtype), memory(state.shape, F32)
    tape = memory((_lib.rnn_delta_tape_size(dims, keep),))
    _lib.rnn_delta_fwd(dims, q, k, v, g, beta, state, reset, lengths, Dk ** -0.5, o, last, keep, tape)
    out = [o, last]
    if keep:
        grads = [memory(p[x].shape, p[x].dtype) for x in LEAVES]
        ws = memory((_lib.rnn_delta_bwd_workspace_size(dims),))
        _lib.rnn_delta_bwd(dims, q, k, v, lengths, Dk ** -0.5, tape, p["do"], p["dlast"], *grads, ws)
        out += grads
    _lib.rnn_check_status(tape)
    return out


# One head of 2500 steps runs in segments. Keys of 16 to 208 channels: the products
# take panels of 64, the segments' maps tiles of 32 or 64, so that between the two
# 16 or 48 columns belong to no tile for some.
SHAPES = [(1, 2500, 1, 1, d, v) for d, v in ((16, 16), (32, 32), (64, 96), (80, 64), (96, 40), (128, 128), (144, 40), (160, 128), (208, 64))]
SHAPES += [(3, 150, 2, 4, 40, 72), (2, 130, 1, 2, 200, 20)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_delta(shape, dtype):
    p = make(*shape, dtype, seed=11)
    B, T = shape[:2]
    short = torch.tensor([T // 2 + 3, T, 0][:B], dtype=torch.int32, device="cuda")
    marks = (torch.rand(B, T, generator=torch.Generator().manual_seed(2)) < 0.004).cuda()
    for lengths, reset, decay in ((None, None, 1), (short, marks, 1), (None, marks, 30)):  # the last: states soon forgotten
        p["g"] = p["g"] * decay
        for keep in (True, False):
            clean, dirty = (run(p, fill, lengths, reset, keep) for fill in (0, 255))
            for name, a, b in zip(("o", "last", *LEAVES), clean, dirty):
                assert torch.isfinite(a).all() and torch.equal(a, b), name


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_norm(dtype):
    for rows, groups, width in ((5000, 3, 40), (7, 2, 1000), (3, 1, 5000)):
        x, z, dy = (torch.randn(rows, groups * width, device="cuda").to(dtype) for _ in range(3))
        w, b = (torch.randn(groups * width, device="cuda").to(dtype) for _ in range(2))
        out = []
        for fill in (0, 255):
            y, dx, dz, dw, db = (torch.empty_like(t) for t in (x, x, x, w, w))
            ws = torch.empty(_lib.rnn_group_norm_workspace_size(rows, groups, width, dtype), dtype=torch.uint8, device="cuda")
            for t in (y, dx, dz, dw, db, ws):
                t.view(-1).view(torch.uint8).fill_(fill)
            _lib.rnn_group_norm_fwd(rows, groups, width, "silu", True, 1e-5, x, w, b, z, y)
            _lib.rnn_group_norm_bwd(rows, groups, width, "silu", True, 1e-5, x, w, b, z, dy, dx, dz, dw, db, ws)
            out.append((y, dx, dz, dw, db))
        for a, c in zip(*out):
            assert torch.isfinite(a).all() and torch.equal(a, c)
