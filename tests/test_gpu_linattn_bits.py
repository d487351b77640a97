"""How many bits linear attention keeps with bf16 tokens: outputs are the definition's, rounded
once; states and their gradients are exact to 32 bits."""

import pytest

from tests import _linattn as ref
from tests.test_gpu_linattn import CASES, make, rows_kw, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

# A weight, and a state that is read out, loses at most 2^-17 of itself (8 bits, and the rest to 8
# bits: 2^-8 2^-9), in half steps of bf16 (2^-8):
INNER = 2.0 ** -9


@pytest.mark.parametrize("case", CASES, ids=str)
def test_read_outs(wk, case):
    B, T, H, G, N, P, fixed, state, rows, lengths = case
    ins, s0, _, _, kw = make(81, B, T, H, G, N, P, "bf16", fixed, state, rows, lengths)
    y, _, _ = wk.linattn_forward(*ins, s0=s0, **kw)
    want = ref.reference(*ins, s0=s0, **rows_kw(kw))["y"]
    ref.assert_within(y, want, ins[2].dtype, ref.roundings(T, N, P), "y", INNER)


@pytest.mark.parametrize("T", [1, 2, 17, 63, 64])
@pytest.mark.parametrize("H,G,N,P", [(2, 2, 64, 64), (6, 2, 32, 128), (2, 1, 128, 64), (3, 3, 128, 32)])
def test_gradients_within_a_tile(wk, T, H, G, N, P):
    """From states and gradients of states that bf16 holds, so that the checkpoint rounds nothing."""
    ins, s0, dy, dsT, kw = make(82, 3, T, H, G, N, P, "bf16")
    t = ins[2].dtype
    s0, dsT = s0.to(t).float(), dsT.to(t).float()
    _, _, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for name in ("dq", "dk", "dv", "dg"):
        ref.assert_within(getattr(g, name), want[name], t, 4 * ref.roundings(T, N, P), name, INNER)


def off(got, want):
    """How much farther from the definition than its own values rounded once, in 2-norms."""
    import torch
    want = want[0]
    on = ~torch.isnan(want)
    want, got = want[on], got.double().cpu()[on]
    return float((got - want).norm() / (want.to(torch.bfloat16).double() - want).norm())


@pytest.mark.parametrize("B,T,H,G,N,P,state", [(2, 200, 4, 4, 64, 64, True), (1, 130, 3, 1, 128, 128, True),
                                               (2, 300, 4, 2, 32, 32, True), (1, 700, 2, 2, 64, 32, False),
                                               (1, 256, 2, 2, 128, 32, True), (1, 900, 3, 3, 32, 64, False)])
def test_gradients_over_tiles(wk, B, T, H, G, N, P, state):
    """Between tiles the gradients of states keep ten bits, two more than outputs: 1 / 16 of their
    squared error.  dq and dg are from the states of the checkpoints, which hold eight."""
    ins, s0, dy, dsT, kw = make(83, B, T, H, G, N, P, "bf16", state=state)
    y, _, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for name in ("dk", "dv"):
        # 2^-10, and 2^-12 for the two steps of its rounding, in half steps of bf16
        ref.assert_within(getattr(g, name), want[name], ins[2].dtype, 2 * ref.roundings(T, N, P), name, 1.25 / 4 + INNER)
        assert off(getattr(g, name), want[name]) < 1.1, name
    assert off(y, want["y"]) < 1.01


@pytest.mark.parametrize("N,P", [(64, 64), (32, 32), (128, 64), (32, 128)])
def test_gradients_of_states_far_apart(wk, N, P):
    """Neighbours in a row of D that differ by up to 2^28, whole rows by any factor, zeros among them."""
    import torch
    ins, s0, dy, dsT, kw = make(84, 2, 70, 2, 1, N, P, "bf16")
    gen = torch.Generator().manual_seed(1)
    dsT = dsT * torch.exp2(torch.randint(-27, 1, dsT.shape, generator=gen)).cuda()
    dsT = dsT * torch.exp2(torch.randint(-60, 50, dsT.shape[:-1], generator=gen))[..., None].cuda()
    dsT[0, 0, 3], dsT[1, 1, :, 5] = 0.0, 0.0
    ins[3][:] = -1e-3
    dy = torch.zeros_like(dy)
    _, _, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for name in ("dk", "dv"):
        ref.assert_within(getattr(g, name), want[name], ins[2].dtype, 2 * ref.roundings(70, N, P), name, 1.25 / 4 + INNER)


@pytest.mark.parametrize("N,P", [(64, 64), (32, 32), (128, 64)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_gradient_of_a_state_that_is_not_finite(wk, bad, N, P):
    """It stays in its column of dk and its row of dv; beside it bf16's own bits but one are kept."""
    import torch
    ins, s0, dy, dsT, kw = make(85, 1, 64, 2, 2, N, P, "bf16")
    _, _, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    dsT[0, 1, 4, 9] = bad
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for name in ("dk", "dv"):
        value, mag = want[name]
        fine = torch.isfinite(value)
        got = getattr(g, name).double().cpu()
        assert torch.equal(torch.isfinite(got), fine), name
        hide = lambda x: torch.where(fine, x, 0.0)   # noqa: E731
        ref.assert_within(hide(got), (hide(value), hide(mag)), ins[2].dtype, ref.roundings(64, N, P), name, 3)


@pytest.mark.parametrize("power", [-100, -111, -114, -120, -124])
def test_gradients_of_tiny_states(wk, power):
    """Down to where a float's own exponents end, below 2^-112 to bf16's eight bits."""
    import torch
    ins, s0, dy, dsT, kw = make(86, 1, 64, 2, 2, 64, 64, "bf16", state=True)
    ins[2].mul_(2.0 ** 100)
    dsT = torch.ldexp(dsT.clamp(-0.9, 0.9), torch.tensor(power).cuda())
    s0, dy = torch.zeros_like(s0), torch.zeros_like(dy)
    _, _, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    ref.assert_within(g.dk, want["dk"], ins[2].dtype, ref.roundings(64, 64, 64), "dk", 1 + INNER)
    assert off(g.dk, want["dk"]) < (1.1 if power > -111 else 2)
