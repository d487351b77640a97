"""The group norm on the GPU with the gate in front in every mode, and with more rows than the
workgroups of a launch take at once, against its definition in 64 bits."""

import pytest

from tests import _gnorm as ref
from tests._linattn import assert_within
from tests.test_gpu_gnorm import make, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def check(wk, args, G, how, forward=True, backward=True):
    import torch
    x, gamma, beta, z, dy = args
    rows, W = x.shape[0], x.shape[1] // G
    want = ref.norm(x, G, gamma, beta, z, dy=dy if backward else None, **how)
    K = W + 40
    if forward:
        assert_within(wk.gnorm_forward(x, G, gamma, beta, z=z, **how), want["y"], x.dtype, K, "y")
    if not backward:
        return
    got, again = (wk.gnorm_backward(x, dy, G, gamma, beta, z=z, **how) for _ in range(2))
    for name, g in got._asdict().items():
        given = dict(dx=x, dz=z, dgamma=gamma, dbeta=beta)[name]
        assert (g is None) == (given is None), name
        if g is None:
            continue
        sums = name in ("dgamma", "dbeta")
        assert_within(g, want[name], torch.float32 if sums else x.dtype, 2 * K + (rows if sums else 0), name)
        assert torch.equal(g, getattr(again, name)), name


# every way a group is laid over lanes, as in the other modes' test
SIZES = [(3, 5, 5), (5, 24, 1), (7, 64, 8), (9, 12 * 64, 12), (4, 7 * 143, 7), (2, 1000, 1), (33, 520, 1), (5, 1030, 1),
         (3, 2048, 1), (2, 4096, 1), (2, 8192, 1), (3, 8200, 1), (2, 1027, 1), (1, 16390, 1)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_gate_in_front(wk, size, dtype, center, silu):
    rows, D, G = size
    check(wk, make(31, rows, D, dtype), G, dict(gate_first=True, center=center, silu=silu))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("one", ["gamma", "beta"])
@pytest.mark.parametrize("silu", [False, True])
def test_gate_in_front_with_one_parameter(wk, dtype, one, silu):
    x, gamma, beta, z, dy = make(32, 70, 6 * 128, dtype)
    args = (x, gamma if one == "gamma" else None, beta if one == "beta" else None, z, dy)
    check(wk, args, 6, dict(gate_first=True, silu=silu))


# rows, D, G: a workgroup goes over its rows three times or more, the last time not all of them do
# (which test_norm_plans.py checks)
BACKWARD = [(5003, 2048, 1), (1300, 1027, 1), (1300, 8200, 1), (60001, 64, 4), (7001, 12 * 64, 12), (30001, 15, 5)]
FORWARD = [(17000, 1023, 1), (1050001, 5, 1), (701, 32768, 4096)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", BACKWARD, ids=str)
@pytest.mark.parametrize("how", [dict(gate_first=True), dict(center=False, gate_first=False, silu=True)], ids=str)
def test_gradients_over_many_rows(wk, size, dtype, how):
    rows, D, G = size
    check(wk, make(33, rows, D, dtype), G, how, forward=False)


@pytest.mark.parametrize("size,dtype", [(FORWARD[0], "bf16"), (FORWARD[1], "fp32"), (FORWARD[1], "bf16"), (FORWARD[2], "bf16")],
                         ids=str)
def test_forward_over_many_rows(wk, size, dtype):
    rows, D, G = size
    check(wk, make(34, rows, D, dtype, gate=False), G, dict(), backward=False)
