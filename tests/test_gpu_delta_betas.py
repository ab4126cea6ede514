"""Betas near zero (gates that are shut), as small as fp32 has them, of either sign.

Tolerances as in test_gpu_delta.py. bf16 storage takes a |beta| below 2^-60 as
2^-60 where a backward comes, which adds 2^-60 of a row product: far below them."""
import pytest
import torch

from test_gpu_delta import BF, F32, check, close, make, oracle, run

pytestmark = pytest.mark.gpu

SMALL = [0.0, 2.0 ** -59, 2.0 ** -61, 1e-25, 1e-30, 1e-35, 1.2e-38, 1e-40, 3e-43, 1.4e-45]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 200, 1, 2, 40, 48), (1, 130, 1, 1, 128, 128), (1, 2500, 1, 1, 32, 32)],
                         ids=lambda s: "B%dT%dNk%dN%dDk%dDv%d" % s)
def test_small_betas(shape, dtype):
    p = make(*shape, dtype, seed=31)
    for i, small in enumerate(SMALL):
        p["beta"][:, 2 * i::41] = small
        p["beta"][:, 2 * i + 1::41] = -small
    check(p)
    # and one shut step at a time, so that no other's dbeta sets the measure
    got = run(p)[6].double().cpu()
    want = torch.as_tensor(oracle(p)[6])
    for small in SMALL:
        at = (p["beta"].abs() == torch.tensor(small, device="cuda")).cpu()
        assert at.any()
        close(got[at].float(), want[at], "dbeta", shape[1], dtype)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_shut_gates_write_nothing(dtype):
    """Without a backward to come, a beta of zero leaves no trace: steps that keep a state keep its bits."""
    for T in (100, 2500):
        p = make(1, T, 1, 1, 32, 24, dtype, seed=32)
        p["beta"].zero_()
        p["g"].zero_()
        o, last = run(dict(p, state=torch.zeros_like(p["state"])), grads=False)
        assert (o == 0).all() and (last == 0).all()
        assert torch.equal(run(p, grads=False)[1], p["state"])
