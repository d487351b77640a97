"""Gradients of the selective scan where a group's channels do not fill a workgroup: the
lanes behind the group take no part, whatever the last channel's bias, decay and incoming
gradient are."""

import numpy as np
import pytest

from tests import _bounds
from tests.test_gpu_ssm import call, host, hosts, make, wk  # noqa: F401

pytestmark = pytest.mark.gpu


def raw_rates(p, bias, low, high, a_min, seed):
    """Rates dt + bias in [low, high] without softplus, decays A from a_min to -0.05."""
    import torch
    rng = np.random.default_rng(seed)
    p["dt_bias"].fill_(bias)
    p["dt"].copy_(torch.from_numpy(rng.uniform(low - bias, high - bias, size=p["dt"].shape)))
    p["A"].copy_(torch.from_numpy(-np.exp(rng.uniform(np.log(0.05), np.log(-a_min), size=p["A"].shape))))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("N,D,G", [(8, 20, 1), (8, 69, 1), (16, 40, 1), (16, 42, 2), (32, 20, 1), (64, 42, 2)])
def test_long_rows_with_a_negative_bias(wk, N, D, G, bits, dtype):   # noqa: F811
    """Every rate is positive and every state decays, while exp(bias A) is above 1."""
    import torch
    B, T = 1, 1100
    p, h0, more = make(71, B, T, D, N, G, dtype)
    raw_rates(p, -0.125, 0.02, 0.5, -16.0, 72)
    args, kw = call(p)
    _, _, ck = wk.ssm_forward(*args, h0=h0, softplus=False, ckpt_bits=bits, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], softplus=False, ckpt_bits=bits, **kw)
    torch.cuda.synchronize()
    entry = None
    if bits == 8:
        codes, scales = wk.ssm_split_ckpt(ck, B, T, D, N)
        entry = host(codes.float()) * host(scales)[..., None]
    want = _bounds.scan(h0=host(h0), softplus_on=False, dy=host(more["dy"]), dhT=host(more["dhT"]), entry=entry,
                        segment=128, **hosts(p))
    _bounds.assert_grads(got, want, p["x"].dtype)


@pytest.mark.parametrize("N,D,G,B", [(8, 20, 1, 2), (8, 21, 1, 2), (16, 40, 1, 2), (16, 14, 2, 2), (32, 20, 1, 2),
                                     (64, 18, 1, 2), (16, 6, 1, 260), (32, 20, 1, 130)])   # the last two: two workgroups a unit
def test_one_step_of_the_bias_alone_overflows(wk, N, D, G, B):   # noqa: F811
    """bias A above 88 without an incoming state gradient: dC and dB stay those of the live channels."""
    p, h0, more = make(73, B, 40, D, N, G, "fp32")
    raw_rates(p, -2.0, 0.02, 0.5, -64.0, 74)
    p["A"][-1].fill_(-64.0)
    args, kw = call(p)
    _, _, ck = wk.ssm_forward(*args, h0=h0, softplus=False, ckpt_bits=32, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, softplus=False, **kw)
    want = _bounds.scan(h0=host(h0), softplus_on=False, dy=host(more["dy"]), **hosts(p))
    _bounds.assert_grads(got, want, p["x"].dtype)


@pytest.mark.parametrize("N,D", [(8, 20), (16, 40), (32, 20), (64, 18)])
def test_growing_states_at_small_rates(wk, N, D):   # noqa: F811
    """A positive last A: its states grow by e over the row at the rates given, by far more at
    the rate of the bias alone."""
    import torch
    T = 640
    p, h0, more = make(75, 1, T, D, N, 1, "fp32")
    p["dt_bias"].fill_(3.0)
    p["dt"].copy_(torch.from_numpy(np.random.default_rng(76).uniform(-10.0, -9.0, size=p["dt"].shape)))
    p["A"][-1].fill_(1.0)
    args, kw = call(p)
    _, _, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=32, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], **kw)
    want = _bounds.scan(h0=host(h0), dy=host(more["dy"]), dhT=host(more["dhT"]), segment=128, **hosts(p))
    _bounds.assert_grads(got, want, p["x"].dtype)


@pytest.mark.parametrize("bits", [32, 8])
def test_no_channels(wk, bits):   # noqa: F811
    """D = 0: nothing depends on B and C, their gradients are 0."""
    import torch
    p, h0, more = make(77, 2, 20, 0, 16, 1, "fp32")
    args, kw = call(p)
    y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=bits, **kw)
    assert y.shape == (2, 20, 0) and hT.shape == (2, 0, 16) and ck.numel() == 0
    dirty = [torch.full_like(p["Bm"], float("nan")) for _ in range(8)]   # what the allocator hands out next
    del dirty
    g = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], ckpt_bits=bits, **kw)
    assert bool((g.dB == 0).all()) and bool((g.dC == 0).all()) and g.dA.shape == (0, 16)
