"""The scan against its definition with the error bound of tests/_bounds.py: groups of many
channel blocks, whose partial sums of dB and dC meet in the second kernel, and long rows in
time segments.  The bound forgets as the states do, so that a state, a segment's map or a
carry held in 16 bits would not pass."""

import ctypes

import numpy as np
import pytest

from tests import _bounds
from tests.test_gpu_ssm import call, host, hosts, make, wk  # noqa: F401

pytestmark = pytest.mark.gpu


def run(wk, p, h0, more, bits=32, softplus=True, segment=0):   # noqa: F811
    """Forward and gradients, every output within its bound."""
    import torch
    B, T, D = p["x"].shape
    N, tok = p["A"].shape[1], p["x"].dtype
    args, kw = call(p)
    y, hT, ck = wk.ssm_forward(*args, h0=h0, softplus=softplus, ckpt_bits=bits, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], softplus=softplus, ckpt_bits=bits, **kw)
    torch.cuda.synchronize()
    inputs = dict(h0=host(h0), softplus_on=softplus, dy=host(more["dy"]), dhT=host(more["dhT"]), segment=segment,
                  **hosts(p))
    want = _bounds.scan(**inputs)
    _bounds.assert_bound(y, want["y"], tok, "y")
    _bounds.assert_bound(hT, want["hT"], torch.float32, "hT")
    if bits == 32:
        _bounds.assert_bound(ck, want["ckpt"], torch.float32, "ckpt")
    else:
        codes, scales = wk.ssm_split_ckpt(ck, B, T, D, N)
        want = _bounds.scan(entry=host(codes.float()) * host(scales)[..., None], **inputs)
    _bounds.assert_grads(got, want, tok)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("D,N,G", [(354, 16, 1),    # 12 blocks of 32 channels, the last of two
                                   (2 * 257, 16, 2),   # 9 blocks a group, odd widths
                                   (581, 8, 1),     # 10 blocks of 64
                                   (137, 32, 1), (275, 64, 1)])   # 9 and 18 blocks of 16
def test_many_channel_blocks(wk, D, N, G, bits, dtype):   # noqa: F811
    p, h0, more = make(91, 2, 20, D, N, G, dtype, lengths=[20, 7] if N == 32 else None)
    run(wk, p, h0, more, bits)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("B,T,D,N,G,lengths", [(1, 1000, 24, 16, 1, None), (2, 700, 10, 8, 2, [700, 300]),
                                               (1, 513, 20, 64, 1, None), (1, 2048, 7, 32, 1, [1999])])
def test_time_segments(wk, B, T, D, N, G, lengths, softplus, dtype):   # noqa: F811
    import torch
    p, h0, more = make(93, B, T, D, N, G, dtype, lengths=lengths)
    if not softplus:   # rates from 0.002 to 0.3, and some of 0 and below
        rates = np.exp(np.random.default_rng(94).uniform(-6, -1.2, size=p["dt"].shape))
        rates[:, ::5] *= -0.01
        p["dt"].copy_(torch.from_numpy(rates) - host_bias(p))
    d = wk.SsmDesc(B, T, D, N, G, wk.WKV7_BF16 if dtype == "bf16" else wk.WKV7_F32, 32)
    assert wk.lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d)) > 0   # segments, of 80 tokens at most here
    run(wk, p, h0, more, softplus=softplus, segment=80)


def host_bias(p):
    import torch
    p["dt_bias"].copy_(torch.round(p["dt_bias"] * 4) / 4)
    return p["dt_bias"].double().cpu()
