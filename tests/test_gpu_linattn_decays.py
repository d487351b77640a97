"""Log decays that are not finite: they reach what the recurrence takes them to, in every output
and gradient, and the rest is what the definition says."""

import pytest

from tests import _linattn as ref
from tests.test_gpu_linattn import make, rows_kw, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def check(wk, ins, s0, dy, dsT, kw, T):
    import torch
    t = ins[2].dtype
    inner = 1 if t == torch.bfloat16 else 0
    N, P = ins[0].shape[-1], ins[2].shape[-1]
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    torch.cuda.synchronize()
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    K = ref.roundings(T, N, P)
    got = dict(y=(y, t, K, inner), sT=(sT, torch.float32, K, 0), dq=(g.dq, t, 2 * K, inner),
               dk=(g.dk, t, 2 * K, inner), dv=(g.dv, t, 2 * K, inner), ds0=(g.ds0, torch.float32, 2 * K, 0))
    for name, (x, kind, k, more) in got.items():
        value, mag = want[name]
        fine = torch.isfinite(value)
        x = x.double().cpu()
        assert torch.equal(torch.isfinite(x), fine), name
        hide = lambda a: torch.where(fine, a, 0.0)   # noqa: E731
        ref.assert_within(hide(x), (hide(value), hide(mag)), kind, k, name, more)
    if g.dg is not None:
        # also the other tokens of the 64, by the contract
        fine = torch.isfinite(want["dg"][0])
        for i in range(0, T, 64):
            fine[:, i:i + 64] &= fine[:, i:i + 64].all(1, keepdim=True)
        assert torch.isfinite(g.dg.cpu()[fine]).all()


BAD = [float("inf"), float("nan"), 3e38, 2e5]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("at", [[0], [37], [63], [64], [100], [129], [10, 40], [63, 64]], ids=str)
def test_decays_that_are_not_finite(wk, at, bad, dtype):
    ins, s0, dy, dsT, kw = make(61, 2, 130, 4, 2, 32, 64, dtype)
    for t in at:
        ins[3][1, t, 2] = bad
    check(wk, ins, s0, dy, dsT, kw, 130)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", BAD)
def test_beside_decays_of_minus_infinity(wk, bad, dtype):
    """What is forgotten is forgotten (0), what is not finite stays so, in either order."""
    ins, s0, dy, dsT, kw = make(62, 2, 100, 2, 2, 64, 32, dtype)
    ins[3][0, 20, 0], ins[3][0, 30, 0] = bad, float("-inf")
    ins[3][1, 20, 1], ins[3][1, 30, 1] = float("-inf"), bad
    check(wk, ins, s0, dy, dsT, kw, 100)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_time_segments_and_shared_heads(wk, dtype):
    ins, s0, dy, dsT, kw = make(63, 1, 1300, 4, 1, 64, 64, dtype)
    ins[3][0, 700, 1] = float("nan")
    check(wk, ins, s0, dy, dsT, kw, 1300)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", BAD)
def test_constant_decays(wk, bad, dtype):
    ins, s0, dy, dsT, kw = make(64, 3, 70, 2, 1, 32, 32, dtype, fixed=True, rows="padded", lengths=[70, 64, 0])
    ins[3][1] = bad
    check(wk, ins, s0, dy, dsT, kw, 70)
