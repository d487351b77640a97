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
