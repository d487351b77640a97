"""The group norm with an activation on the GPU against its definition in 64 bits."""

import pytest

from tests import _gnorm as ref
from tests._linattn import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rwkv_wkv7_delta_amd as wk
    wk.lib()
    return wk


def make(seed, rows, D, dtype, affine=True, gate=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    normal = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    x = (normal(rows, D) + normal(D)).to(t).cuda()
    z = normal(rows, D).to(t).cuda() if gate else None
    gamma, beta = ((1 + normal(D)).cuda(), normal(D).cuda()) if affine else (None, None)
    return x, gamma, beta, z, normal(rows, D).to(t).cuda()


# rows, D, G: every way a group is laid over lanes (vectors of 8, 2, 1; 4 to 512 lanes; wider)
SIZES = [(1, 1, 1), (3, 5, 5), (5, 24, 1), (7, 64, 8), (3, 128, 2), (9, 12 * 64, 12), (4, 7 * 143, 7), (2, 1000, 1),
         (6, 40 * 64, 40), (33, 520, 1), (5, 1030, 1), (3, 2048, 1), (2, 4096, 1), (2, 8192, 1), (3, 8200, 1),
         (2, 2052, 2), (2, 1027, 1), (2, 3 * 90, 3), (1, 16390, 1)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("mode", [0, 1, 2, 3])
def test_forward_and_gradients(wk, size, dtype, mode):
    import torch
    rows, D, G = size
    how = [dict(center=True, silu=True), dict(center=True, gate_first=False), dict(center=False, gate_first=True),
           dict(center=False, gate_first=False, silu=True)][mode]
    x, gamma, beta, z, dy = make(5 + mode, rows, D, dtype, affine=mode != 2, gate=mode > 0)
    y = wk.gnorm_forward(x, G, gamma, beta, z=z, **how)
    got = wk.gnorm_backward(x, dy, G, gamma, beta, z=z, **how)
    again = wk.gnorm_backward(x, dy, G, gamma, beta, z=z, **how)
    torch.cuda.synchronize()
    want = ref.norm(x, G, gamma, beta, z, dy=dy, **how)
    K = D // G + 40
    assert_within(y, want["y"], x.dtype, K, "y")
    for name, g in got._asdict().items():
        if g is None:
            assert name == "dz" and z is None or name != "dz" and gamma is None
            continue
        sums = name in ("dgamma", "dbeta")
        assert_within(g, want[name], torch.float32 if sums else x.dtype, 2 * K + (rows if sums else 0), name)
        assert torch.equal(g, getattr(again, name))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_rows(wk, dtype):
    """More rows than workgroups: sums over all of them, and one parameter without the other."""
    import torch
    x, gamma, beta, z, dy = make(9, 9001, 96, dtype)
    for ga, be in ((gamma, None), (None, beta)):
        got = wk.gnorm_backward(x, dy, 3, ga, be, z=z)
        want = ref.norm(x, 3, ga, be, z, dy=dy)
        for name in ("dx", "dz", "dgamma" if be is None else "dbeta"):
            sums = name[1] != "x" and name[1] != "z"
            assert_within(getattr(got, name), want[name], torch.float32 if sums else x.dtype,
                          144 + (9001 if sums else 0), name)
        assert (got.dgamma is None) == (ga is None) and (got.dbeta is None) == (be is None)


def test_values_that_are_not_finite(wk):
    """They stay in their row and group."""
    import torch
    x, gamma, beta, z, dy = make(10, 6, 96, "bf16")
    clean = wk.gnorm_forward(x, 3, gamma, beta, z=z), wk.gnorm_backward(x, dy, 3, gamma, beta, z=z)
    for bad in (float("inf"), float("nan")):
        for where in (x, z, dy):
            keep = where.clone()
            where[2, 40] = bad
            y, g = wk.gnorm_forward(x, 3, gamma, beta, z=z), wk.gnorm_backward(x, dy, 3, gamma, beta, z=z)
            where.copy_(keep)
            for a, b in ((y, clean[0]), (g.dx, clean[1].dx), (g.dz, clean[1].dz)):
                same = (a == b) | (a.isnan() & b.isnan())
                same[2, 32:64] = True
                assert bool(same.all())
            for a, b in ((g.dgamma, clean[1].dgamma), (g.dbeta, clean[1].dbeta)):
                assert torch.equal(a[:32], b[:32]) and torch.equal(a[64:], b[64:])


def test_empty(wk):
    import torch
    x = torch.empty(0, 64, device="cuda")
    g = torch.ones(64, device="cuda")
    assert wk.gnorm_forward(x, 2, g, g).shape == (0, 64)
    got = wk.gnorm_backward(x, x, 2, g, None)
    assert got.dx.shape == (0, 64) and torch.equal(got.dgamma, torch.zeros_like(g)) and got.dbeta is None
    got = wk.gnorm_backward(x, x, 2, None, g)
    assert torch.equal(got.dbeta, torch.zeros_like(g)) and got.dgamma is None
    assert wk.gnorm_forward(torch.empty(4, 0, device="cuda"), 1).shape == (4, 0)
