"""The short causal convolution on the GPU against its definition in 64 bits.

Rounding: W + 1 products and sums of the pre-activation (6 roundings at most),
the activation's exponential, reciprocal and products (8 more, relative to its
own magnitude with the exponent's factor 1 + |pre| in it): 16.  The gradients'
sums over n tokens add n roundings relative to the sum of magnitudes.
"""

import numpy as np
import pytest

from tests import _mixers as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rwkv_wkv7_delta_amd as wk
    wk.lib()
    return wk


def make(seed, B, T, D, W, dtype, bias=True, state=True, lengths=None):
    import torch
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = lambda a, ty=torch.float32: torch.from_numpy(np.asarray(a)).to(ty).cuda()   # noqa: E731
    p = dict(x=dev(rng.normal(size=(B, T, D)), t), weight=dev(rng.normal(size=(D, W)) / W ** 0.5),
             bias=dev(rng.normal(size=D)) if bias else None,
             s0=dev(rng.normal(size=(B, W - 1, D)), t) if state else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    more = dict(dy=dev(rng.normal(size=(B, T, D)), t), dsT=dev(rng.normal(size=(B, W - 1, D)), t) if state else None)
    return p, more


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


CASES = [
    # B, T, D, W, silu, bias, state, lengths
    (1, 1, 1, 2, False, False, False, None),
    (1, 1, 8, 4, True, True, True, None),
    (2, 2, 24, 4, True, True, False, None),
    (2, 3, 7, 3, False, True, True, None),
    (3, 16, 64, 2, False, False, True, None),
    (2, 17, 65, 4, True, True, True, None),
    (2, 33, 40, 3, True, False, True, [33, 0]),
    (5, 37, 12, 4, True, True, True, [0, 1, 2, 3, 37]),
    (3, 40, 260, 4, False, True, False, [40, -5, 100]),   # clamped to [0, 40]
    (2, 131, 520, 4, True, True, True, None),
    (1, 700, 6, 2, False, False, True, None),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(wk, case, dtype):
    import torch
    B, T, D, W, silu, bias, state, lengths = case
    p, more = make(7, B, T, D, W, dtype, bias, state, lengths)
    y, sT = wk.conv_forward(p["x"], p["weight"], p["bias"], s0=p["s0"], lengths=p["lengths"], silu=silu,
                            want_state=True)
    dx, dw, db, ds0 = wk.conv_backward(p["x"], p["weight"], more["dy"], p["bias"], s0=p["s0"], dsT=more["dsT"],
                                       lengths=p["lengths"], silu=silu)
    torch.cuda.synchronize()
    h = {k: host(v) for k, v in p.items()}
    want = ref.conv(silu=silu, **h)
    ref.assert_within(y, want["y"], p["x"].dtype, 16, "y")
    assert np.array_equal(host(sT), want["sT"][0])   # copies
    grads = ref.conv_grads(dy=host(more["dy"]), dsT=host(more["dsT"]), silu=silu, **h)
    ref.assert_within(dx, grads["dx"], p["x"].dtype, 32, "dx")
    ref.assert_within(ds0, grads["ds0"], p["x"].dtype, 32, "ds0")
    ref.assert_within(dw, grads["dweight"], torch.float32, 32 + B * T, "dweight")
    if bias:
        ref.assert_within(db, grads["dbias"], torch.float32, 32 + B * T, "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 64, 768, 1000])
def test_steps_equal_the_prompt(wk, D, dtype):
    """Token by token from a state gives the prompt form's outputs and last state bit
    for bit (the same sums in the same order)."""
    import torch
    for W, silu in ((2, False), (3, True), (4, True)):
        p, _ = make(11, 3, 9, D, W, dtype)
        y, sT = wk.conv_forward(p["x"], p["weight"], p["bias"], s0=p["s0"], silu=silu, want_state=True)
        state = p["s0"].clone()
        steps = [wk.conv_step(p["x"][:, t].contiguous(), p["weight"], state, p["bias"], silu=silu) for t in range(9)]
        assert torch.equal(torch.stack(steps, 1), y) and torch.equal(state, sT)


def test_token_shift(wk):
    """At two taps (mu, 1 - mu) the convolution is x + mu (previous x - x)."""
    import torch
    p, _ = make(3, 2, 50, 96, 2, "fp32", bias=False, state=False)
    mu = torch.rand(96, device="cuda")
    y, _ = wk.conv_forward(p["x"], torch.stack([mu, 1 - mu], 1))
    x = p["x"].double()
    prev = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1)
    want = x + mu.double() * (prev - x)
    # 1 - mu is rounded once, the two products and their sum once each
    assert float((y.double() - want).abs().max()) <= 4 * ref.EPS32 * float(2 * x.abs().max())


def test_padding_is_not_read(wk):
    """Infinities and NaN behind a row's length change nothing, forward and backward."""
    import torch
    for dtype in ("fp32", "bf16"):
        p, more = make(5, 3, 40, 33, 4, dtype, lengths=[40, 0, 17])
        outs = []
        for fill in (0.0, float("nan"), float("inf")):
            x, dy = p["x"].clone(), more["dy"].clone()
            for b, n in enumerate((40, 0, 17)):
                x[b, n:] = fill
                dy[b, n:] = fill
            f = wk.conv_forward(x, p["weight"], p["bias"], s0=p["s0"], lengths=p["lengths"], silu=True,
                                want_state=True)
            g = wk.conv_backward(x, p["weight"], dy, p["bias"], s0=p["s0"], dsT=more["dsT"], lengths=p["lengths"],
                                 silu=True)
            outs.append(f + g)
        for other in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
        assert float(outs[0][0][1].abs().max()) == 0 and float(outs[0][0][2, 17:].abs().max()) == 0


def test_continued_prompt(wk):
    """A prompt in two parts through the state equals the whole, also with a part shorter
    than the state."""
    import torch
    p, _ = make(13, 2, 30, 48, 4, "bf16")
    kw = dict(silu=True, want_state=True)
    y, sT = wk.conv_forward(p["x"], p["weight"], p["bias"], s0=p["s0"], **kw)
    for cut in (1, 2, 3, 16, 29):
        y1, s1 = wk.conv_forward(p["x"][:, :cut].contiguous(), p["weight"], p["bias"], s0=p["s0"], **kw)
        y2, s2 = wk.conv_forward(p["x"][:, cut:].contiguous(), p["weight"], p["bias"], s0=s1, **kw)
        assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(s2, sT)


def test_empty(wk):
    import torch
    p, more = make(17, 2, 5, 24, 4, "bf16")
    none = p["x"][:, :0].contiguous()
    y, sT = wk.conv_forward(none, p["weight"], p["bias"], s0=p["s0"], want_state=True)
    assert y.shape == (2, 0, 24) and torch.equal(sT, p["s0"])
    dx, dw, db, ds0 = wk.conv_backward(none, p["weight"], none, p["bias"], s0=p["s0"], dsT=more["dsT"])
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0 and torch.equal(ds0, more["dsT"])
    y, sT = wk.conv_forward(p["x"][:0].contiguous(), p["weight"], p["bias"], want_state=True)
    assert y.numel() == 0 and sT.numel() == 0
    _, dw, db, _ = wk.conv_backward(p["x"][:0].contiguous(), p["weight"], p["x"][:0].contiguous(), p["bias"])
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_repeats_agree_and_other_stream(wk):
    import torch
    p, more = make(19, 4, 300, 520, 4, "bf16")
    args = (p["x"], p["weight"], more["dy"], p["bias"])
    first = wk.conv_backward(*args, silu=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = wk.conv_backward(*args, silu=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.parametrize("B,T,D", [(700, 530, 5), (600, 40, 4)])   # gradient runs of 268 and 16 tokens
def test_gradients_of_many_rows(wk, B, T, D):
    import torch
    p, more = make(13, B, T, D, 3, "bf16", lengths=[(7 * b) % (T + 9) for b in range(B)])
    dx, dw, db, ds0 = wk.conv_backward(p["x"], p["weight"], more["dy"], p["bias"], s0=p["s0"], dsT=more["dsT"],
                                       lengths=p["lengths"], silu=True)
    grads = ref.conv_grads(dy=host(more["dy"]), dsT=host(more["dsT"]), silu=True, **{k: host(v) for k, v in p.items()})
    ref.assert_within(dx, grads["dx"], p["x"].dtype, 32, "dx")
    ref.assert_within(ds0, grads["ds0"], p["x"].dtype, 32, "ds0")
    ref.assert_within(dw, grads["dweight"], torch.float32, 32 + B * T, "dweight")
    ref.assert_within(db, grads["dbias"], torch.float32, 32 + B * T, "dbias")
