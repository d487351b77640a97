"""The convolution's gradients where a row's last inputs or gradients are not finite, or large:
nothing behind the row's last token reaches them, and they reach nothing there."""

import pytest

from tests.test_gpu_conv import make, wk  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [7, 12, 1000])
@pytest.mark.parametrize("silu", [True, False])
def test_convolution_gradients_behind_a_row_are_zero(wk, D, silu, dtype):   # noqa: F811
    T, lengths = 40, [40, 0, 17, 38, 1]
    p, more = make(83, 5, T, D, 4, dtype, lengths=lengths)
    for value in (NAN, INF, -INF):
        for name in ("x", "dy", "dsT"):
            bad = dict(p, **more)
            bad[name] = bad[name].clone()
            for b, n in enumerate(lengths):
                if name == "dsT":
                    bad[name][b, :, 3] = value
                elif n > 0:
                    bad[name][b, n - 1, 3] = value
            dx, dw, db, ds0 = wk.conv_backward(bad["x"], bad["weight"], bad["dy"], bad["bias"], s0=bad["s0"],
                                               dsT=bad["dsT"], lengths=bad["lengths"], silu=silu)
            for b, n in enumerate(lengths):
                assert bool((dx[b, n:] == 0).all()), (name, value, b)


@pytest.mark.parametrize("lengths", [None, [40, 17]])
def test_large_last_inputs(wk, lengths):   # noqa: F811
    """A last input whose product with an earlier tap would leave float32's range: no token sees
    that product, so nothing is infinite."""
    import torch
    B, T, D, big = 2, 40, 8, 2.0 ** 126
    p, more = make(85, B, T, D, 4, "fp32", state=False, lengths=lengths)
    p["weight"][:, 0] = 64.0
    p["weight"][:, 3] = 2.0 ** -30
    for b, n in enumerate(lengths or [T, T]):
        p["x"][b, n - 1] = big
    got = wk.conv_backward(p["x"], p["weight"], more["dy"], p["bias"], lengths=p["lengths"], silu=True)
    assert all(bool(torch.isfinite(g).all()) for g in got if g is not None)
    for b, n in enumerate(lengths or [T, T]):
        # the activation's slope is 1 at 2^96: dx of the last token is its own tap's product,
        # which one rounding of the product leaves exact but for half a step
        want = (more["dy"][b, n - 1].double() * 2.0 ** -30)
        off = (got[0][b, n - 1].double() - want).abs()
        assert bool((off <= 2.0 ** -22 * want.abs()).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [7, 12])
@pytest.mark.parametrize("lengths", [None, [40, 17]])
def test_taps_that_never_meet_the_last_input(wk, lengths, D, dtype):   # noqa: F811
    """Without the activation a last input that is not finite reaches the last tap's gradient alone."""
    import torch
    T = 40
    p, more = make(87, 2, T, D, 4, dtype, lengths=lengths)
    grads = []
    for value in (0.0, NAN, INF):
        x = p["x"].clone()
        for b, n in enumerate(lengths or [T, T]):
            x[b, n - 1, 3] = value
        grads.append(wk.conv_backward(x, p["weight"], more["dy"], p["bias"], s0=p["s0"], dsT=more["dsT"],
                                      lengths=p["lengths"]))
    for dx, dw, db, ds0 in grads[1:]:
        assert torch.equal(dx, grads[0][0]) and torch.equal(db, grads[0][2]) and torch.equal(ds0, grads[0][3])
        assert torch.equal(dw[:, :3], grads[0][1][:, :3]) and not bool(torch.isfinite(dw[3, 3]))
