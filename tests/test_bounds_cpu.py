"""The definition that carries its error bound (tests/_bounds.py): its values are those of the
plain definition, and its bound is as tight as the tests that use it say."""

import numpy as np
import pytest

from tests import _bounds, _mixers as ref


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,lengths", [(1, None), (35, [35, 0]), (33, [-1, 40])])
def test_values_are_the_definition(T, lengths, gate, softplus):
    rng = np.random.default_rng(96)
    B, D, N, G = 2, 6, 8, 2
    a = dict(x=rng.normal(size=(B, T, D)), dt=rng.uniform(-1, 0.5, size=(B, T, D)),
             A=-np.exp(rng.uniform(-3, 0, size=(D, N))), Bm=rng.normal(size=(B, T, G, N)),
             Cm=rng.normal(size=(B, T, G, N)), z=rng.normal(size=(B, T, D)) if gate else None,
             dskip=rng.normal(size=D), dt_bias=rng.uniform(0, 1, size=D), h0=rng.normal(size=(B, D, N)),
             lengths=lengths)
    dy, dhT = rng.normal(size=(B, T, D)), rng.normal(size=(B, D, N))
    s = ref.Scan(softplus_on=softplus, **a)
    want = dict(s.outputs(), ckpt=(s.h[:, 0:T:16], None), **s.grads(dy, dhT))
    got = _bounds.scan(softplus_on=softplus, dy=dy, dhT=dhT, **a)
    for name, f in got.items():
        assert np.allclose(f.v, want[name][0], rtol=1e-12, atol=1e-12 * np.abs(f.m).max()), name
        assert (np.abs(f.v) <= f.m * (1 + 1e-12)).all() and (f.e >= 0).all(), name


def test_the_bound_is_far_below_16_bits():
    """On the CPU: over a long row the allowance stays below an eighth of bfloat16's half step."""
    rng = np.random.default_rng(95)
    B, T, D, N = 1, 1500, 6, 16
    out = _bounds.scan(rng.normal(size=(B, T, D)), rng.uniform(-3, 0.5, size=(B, T, D)),
                       -np.exp(rng.uniform(-3, 0.9, size=(D, N))), rng.normal(size=(B, T, 1, N)),
                       rng.normal(size=(B, T, 1, N)), dt_bias=rng.uniform(-1, 0.5, size=D), segment=80,
                       dy=rng.normal(size=(B, T, D)))
    for name in ("y", "hT", "ckpt", "dh0"):
        m = out[name].m
        assert (1.01 * out[name].e * ref.EPS32 <= 2.0 ** -8 / 8 * m + 1e-300).all(), name
