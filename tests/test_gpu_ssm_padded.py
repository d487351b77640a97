"""The scan's gradients of padded batches whose valid tokens or incoming gradients hold
infinities and NaN: outputs behind a row's length are 0 all the same, and rows without
such values keep theirs."""

import pytest

from tests.test_gpu_ssm import call, make, wk  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def zero_behind(name, t, lengths):
    for b, n in enumerate(lengths):
        assert bool((t[b, n:] == 0).all()), (name, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("N,D,G,T", [(8, 20, 1, 50), (16, 64, 1, 50), (16, 42, 2, 50), (32, 130, 1, 50), (64, 34, 2, 50),
                                     (16, 24, 1, 700)])
def test_scan_gradients_behind_a_row_are_zero(wk, N, D, G, T, gate, dtype):   # noqa: F811
    import torch
    B = 4
    lengths = [T, 0, 17, T - 9]
    p, h0, more = make(81, B, T, D, N, G, dtype, gate=gate, lengths=lengths)
    args, kw = call(p)

    def grads(dhT, **over):
        q = [over.get(k, v) for k, v in zip(("x", "dt", "A", "Bm", "Cm"), args)]
        more_kw = dict(kw, **{k: v for k, v in over.items() if k == "z"})
        for bits in (32, 8):
            y, _, ck = wk.ssm_forward(*q, h0=over.get("h0", h0), ckpt_bits=bits, **more_kw)
            g = wk.ssm_backward(*q, over.get("dy", more["dy"]), ck, dhT=dhT, ckpt_bits=bits, **more_kw)
            yield y, g

    sound = list(grads(more["dhT"]))
    for name in ("x", "dt", "Bm", "Cm", "dy", "h0", "dhT") + (("z",) if gate else ()):
        bad = (h0 if name == "h0" else more[name] if name in more else p[name]).clone()
        for b, n in enumerate(lengths):
            if bad.dim() == 3 and name in ("h0", "dhT"):
                bad[b, 3, 1] = NAN if b < 2 else INF
            elif n > 0 and b > 0:
                bad[b, n - 1].flatten()[3] = NAN if b == 2 else INF
        over = {} if name == "dhT" else {name: bad}
        for (y, g), (y1, g1) in zip(grads(bad if name == "dhT" else more["dhT"], **over), sound):
            zero_behind(f"{name}: y", y, lengths)
            for k in ("dx", "ddt", "dB", "dC", "dz"):
                if getattr(g, k) is not None:
                    zero_behind(f"{name}: {k}", getattr(g, k), lengths)
            if name not in ("h0", "dhT"):   # rows without such values
                assert torch.equal(y[0], y1[0]) and torch.equal(g.dx[:2], g1.dx[:2]) and torch.equal(g.dh0[:2], g1.dh0[:2])
                assert torch.equal(g.dB[:2], g1.dB[:2]) and torch.equal(g.ddt[:2], g1.ddt[:2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,D,T", [(8, 70, 40), (16, 48, 40), (16, 21, 700), (32, 40, 40), (64, 18, 40)])
def test_values_that_are_not_finite_stay_in_their_channel(wk, N, D, T, dtype):   # noqa: F811
    """dB and dC are sums over channels; everything else of the other channels keeps its bits."""
    import torch
    p, h0, more = make(89, 2, T, D, N, 1, dtype)
    args, kw = call(p)

    def grads(x, dy, dhT):
        y, hT, ck = wk.ssm_forward(x, *args[1:], h0=h0, ckpt_bits=8, **kw)
        g = wk.ssm_backward(x, *args[1:], dy, ck, dhT=dhT, ckpt_bits=8, **kw)
        return dict(y=y, hT=hT, dx=g.dx, ddt=g.ddt, dz=g.dz, dA=g.dA[None, None], ddskip=g.ddskip[None, None],
                    ddt_bias=g.ddt_bias[None, None], dh0=g.dh0)

    sound = grads(args[0], more["dy"], more["dhT"])
    others = torch.arange(D, device="cuda") != 7
    for value in (NAN, INF):
        for name in ("x", "dy", "dhT"):
            bad = dict(x=args[0].clone(), dy=more["dy"].clone(), dhT=more["dhT"].clone())
            bad[name][0, 7 if name == "dhT" else 5].flatten()[3 if name == "dhT" else 7] = value
            for k, v in grads(**bad).items():
                dim = 1 if k in ("hT", "dh0") else 2
                pick = lambda t: t.movedim(dim, 0)[others]   # noqa: E731,B023
                assert torch.equal(pick(v), pick(sound[k])), (name, value, k)
