"""Linear attention's gradients where a launch has more units of work than workgroups (256), so that
each goes from unit to unit: over groups, parts of a group's heads, tiles, rows and padding between
them.  And the bits that states and their gradients keep."""

import pytest

from tests import _linattn as ref
from tests.test_gpu_linattn import check, make, rows_kw, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

# Units: rows x tiles x groups x parts of the heads; parts are made of tiles x groups below 512.
CASES = [
    # B, T, H, G, N, P, fixed, state, rows, lengths
    (5, 700, 14, 7, 32, 32, False, True, "full", None),                                # 385
    (3, 333, 19, 19, 64, 64, False, False, "full", None),                              # 342
    (4, 640, 10, 5, 64, 32, False, True, "full", None),                                # 200 in 2 parts
    (6, 400, 10, 5, 32, 64, False, True, "padded", [400, 3, 0, 130, 64, 257]),         # 210 in 2 parts
    (7, 450, 13, 13, 32, 32, False, True, "padded", [0, 450, 1, 65, 0, 128, 449]),     # 728
    (9, 300, 15, 5, 64, 64, False, True, "packed", [300, 0, 1, 64, 65, 299, 128, 17, 200]),   # 225 in 2 parts
    (3, 300, 22, 22, 128, 128, True, False, "full", None),                             # 330, two or four value blocks
    (2, 200, 80, 40, 32, 128, False, True, "packed", [200, 131]),                      # 320
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_more_units_than_workgroups(wk, case, dtype):
    B, T, H, G, N, P, fixed, state, rows, lengths = case
    check(wk, *make(91, B, T, H, G, N, P, dtype, fixed, state, rows, lengths), T)


def test_decays_of_a_row_beyond_two_to_the_31_elements(wk):
    """dg of its last tokens is that of a row that starts from the state before them."""
    import torch
    T, H, N, P = (1 << 19) + 77, 64, 32, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)   # noqa: E731
    q, k, v, dy = rand(1, T, 1, N), rand(1, T, 1, N), rand(1, T, H, P), rand(1, T, H, P)
    g = -rand(1, T, H).abs()
    cut = T - 128 - T % 64
    _, _, ck = wk.linattn_forward(q, k, v, g, want_ckpt=True)
    all_ = wk.linattn_backward(q, k, v, g, dy, ck).dg[0, cut:].float()
    _, mid, _ = wk.linattn_forward(*[x[:, :cut].clone() for x in (q, k, v, g)])
    tail = [x[:, cut:].clone() for x in (q, k, v, g)]
    _, _, ck2 = wk.linattn_forward(*tail, s0=mid, want_ckpt=True)
    want = wk.linattn_backward(*tail, dy[:, cut:].clone(), ck2).dg[0].float()
    # (states that went through other time segments differ in their last bits, and so may the checkpoints)
    assert torch.allclose(all_, want, rtol=2 ** -6, atol=2 ** -6 * float(want.abs().max()))
    assert float((all_ - want).norm() / want.norm()) < 2 ** -8


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,H,G,N,P", [(3, 1, 2, 2, 64, 64), (2, 64, 3, 1, 128, 64), (1, 1000, 2, 2, 64, 64),
                                         (5, 1000, 4, 2, 32, 128), (2, 640, 2, 2, 128, 128), (2, 500, 4, 4, 32, 32)])
def test_states_keep_32_bits(wk, B, T, H, G, N, P, dtype):
    """Their 2-norm's error: operands are carried to 24 bits, a tile's sums of 64 products round at
    random (8 x 2^-25 of their norm) and so do exponentials (2^-24), decayed from tile to tile as the
    states are: 2^-21 and below.  Two of a value's three bf16 parts would leave 2^-17 / sqrt(3)."""
    ins, s0, dy, dsT, kw = make(92, B, T, H, G, N, P, dtype)
    _, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for name, got in (("sT", sT), ("ds0", g.ds0)):
        value = want[name][0]
        far = float((got.double().cpu() - value).norm() / value.norm())
        assert far < 2.0 ** -20, (name, far)
