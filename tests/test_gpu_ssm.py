"""The selective scan on the GPU against its definition in 64 bits.

Rounding, relative to the sums of magnitudes: the rate D carries up to 8
roundings (bias, exponential with the exponent's own rounding, logarithm,
reciprocal, products), so exp(D A) carries 10 |D A| + 2 and a step of the state
at most 10 |D A| + 6, T tokens T times that (and 64 for what is added once), the
adjoint as many again; a gradient is a product of both and of a few factors more
(64, 128), its sum over n terms adds n.
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


def make(seed, B, T, D, N, G, dtype, gate=True, skip=True, bias=True, state=True, lengths=None):
    import torch
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = lambda a, ty=torch.float32: torch.from_numpy(np.asarray(a)).to(ty).cuda()   # noqa: E731
    p = dict(x=dev(rng.normal(size=(B, T, D)), t), dt=dev(rng.uniform(-3, 0.5, size=(B, T, D)), t),
             A=dev(-np.exp(rng.uniform(-3, 0.9, size=(D, N)))),
             Bm=dev(rng.normal(size=(B, T, G, N)), t), Cm=dev(rng.normal(size=(B, T, G, N)), t),
             z=dev(rng.normal(size=(B, T, D)), t) if gate else None,
             dskip=dev(rng.normal(size=D)) if skip else None,
             dt_bias=dev(rng.uniform(-1, 0.5, size=D)) if bias else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    h0 = dev(rng.normal(size=(B, D, N))) if state else None
    more = dict(dy=dev(rng.normal(size=(B, T, D)), t), dhT=dev(rng.normal(size=(B, D, N))) if state else None)
    return p, h0, more


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def hosts(p):
    return {k: host(v) for k, v in p.items()}


def call(p):
    return [p[k] for k in ("x", "dt", "A", "Bm", "Cm")], {k: v for k, v in p.items()
                                                           if k in ("z", "dskip", "dt_bias", "lengths")}


def same(a, b):
    import torch
    return torch.allclose(a, b, rtol=0, atol=0, equal_nan=True)


def check_grads(got, s, more, p):
    import torch
    B, T, D, N, G = s.shape
    want, width, K = s.grads(host(more["dy"]), host(more["dhT"])), D // G, 2 * s.roundings()
    tok = p["x"].dtype
    ref.assert_within(got.dx, want["dx"], tok, K + 64, "dx")
    ref.assert_within(got.ddt, want["ddt"], tok, K + 128, "ddt")
    ref.assert_within(got.dB, want["dB"], tok, K + width, "dB")
    ref.assert_within(got.dC, want["dC"], tok, K + width, "dC")
    ref.assert_within(got.dA, want["dA"], torch.float32, K + B * T, "dA")
    ref.assert_within(got.dh0, want["dh0"], torch.float32, K, "dh0")
    for name in ("dz", "ddskip", "ddt_bias"):
        g = getattr(got, name)
        if g is None:
            assert p[dict(dz="z", ddskip="dskip", ddt_bias="dt_bias")[name]] is None
        else:
            ref.assert_within(g, want[name], tok if name == "dz" else torch.float32, K + 128 + B * T, name)


CASES = [
    # B, T, D, N, G, gate, skip, bias, state, lengths, softplus
    (1, 1, 1, 8, 1, False, False, False, False, None, True),
    (1, 1, 16, 64, 1, True, True, True, True, None, True),
    (2, 2, 5, 16, 5, True, True, True, True, None, True),
    (2, 15, 64, 16, 1, True, True, True, True, None, True),
    (2, 16, 65, 16, 1, False, True, False, True, None, True),
    (1, 17, 130, 8, 2, True, False, True, False, None, True),
    (3, 33, 12, 32, 3, True, True, True, True, None, False),
    (2, 40, 34, 64, 2, False, True, True, True, None, True),
    (4, 50, 20, 16, 1, True, True, True, True, [50, 0, 1, 33], True),
    (3, 35, 7, 8, 1, False, False, True, True, [-3, 16, 99], True),   # clamped to [0, 35]
    (1, 100, 300, 16, 3, True, True, True, True, None, True),
    (2, 37, 40, 16, 1, True, True, False, True, None, "positive"),   # no softplus, dt above 0
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(wk, case, dtype):
    import torch
    B, T, D, N, G, gate, skip, bias, state, lengths, sp = case
    p, h0, more = make(23, B, T, D, N, G, dtype, gate, skip, bias, state, lengths)
    if sp == "positive":
        p["dt"].abs_()
        sp = False
    args, kw = call(p)
    y, hT, none = wk.ssm_forward(*args, h0=h0, softplus=sp, **kw)
    assert none is None
    y32, hT32, ck = wk.ssm_forward(*args, h0=h0, softplus=sp, ckpt_bits=32, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], softplus=sp, ckpt_bits=32, **kw)
    torch.cuda.synchronize()
    assert same(y, y32) and same(hT, hT32)
    s = ref.Scan(h0=host(h0), softplus_on=sp, **hosts(p))
    want = s.outputs()
    K = s.roundings()
    ref.assert_within(y, want["y"], p["x"].dtype, K + N, "y")
    ref.assert_within(hT, want["hT"], torch.float32, K, "hT")
    ref.assert_within(ck, (s.h[:, 0:T:16], s.mh[:, 0:T:16]), torch.float32, K, "ckpt")
    check_grads(got, s, more, p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] > 1], ids=str)
def test_checkpoints_in_8_bits(wk, case, dtype):
    """A code is within half a scale of the state (and the code's rounding); the gradients
    are those of the scan whose blocks start from the stored states."""
    import torch
    B, T, D, N, G, gate, skip, bias, state, lengths, sp = case
    p, h0, more = make(29, B, T, D, N, G, dtype, gate, skip, bias, state, lengths)
    grows = not sp
    if sp == "positive":
        p["dt"].abs_()
        sp = False
    args, kw = call(p)
    y, hT, ck = wk.ssm_forward(*args, h0=h0, softplus=sp, ckpt_bits=8, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], softplus=sp, ckpt_bits=8, **kw)
    torch.cuda.synchronize()
    y0, hT0, _ = wk.ssm_forward(*args, h0=h0, softplus=sp, **kw)
    assert same(y, y0) and same(hT, hT0)
    codes, scales = wk.ssm_split_ckpt(ck, B, T, D, N)
    if grows:
        return   # states that grow past float32's range: stored as NaN, tested below
    plain = ref.Scan(h0=host(h0), softplus_on=sp, **hosts(p))
    h, mh = plain.h[:, 0:T:16], plain.mh[:, 0:T:16]
    err = plain.roundings() * ref.EPS32 * mh
    most = np.abs(h).max(-1)
    sc = host(scales)
    assert (np.abs(sc - most / 127) <= (err.max(-1) + 4 * ref.EPS32 * most) / 127).all()
    stored = codes.cpu().numpy().astype(np.float64) * sc[..., None]
    # half a code, the code's argument rounded three times at up to 127 codes, the state's own error
    assert (np.abs(stored - h) <= sc[..., None] * (0.5 + 127 * 3 * ref.EPS32) + err).all()
    s = ref.Scan(h0=host(h0), softplus_on=sp, entry=stored, **hosts(p))
    check_grads(got, s, more, p)


def test_8_bit_checkpoints_of_odd_states(wk):
    """Zero, tiny, infinite and NaN states: zeros, zeros, NaN, NaN."""
    import torch
    p, _, _ = make(31, 1, 16, 4, 16, 1, "fp32")
    args, kw = call(p)
    h0 = torch.ones(1, 4, 16, device="cuda")
    h0[0, 0] = 0
    h0[0, 1] = 1e-38
    h0[0, 2, 5] = float("inf")
    h0[0, 3, 7] = float("nan")
    _, _, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=8, **kw)
    codes, scales = wk.ssm_split_ckpt(ck, 1, 16, 4, 16)
    v = codes[0, 0] * scales[0, 0, :, None]
    assert float(v[:2].abs().max()) == 0 and bool(v[2:].isnan().all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,G,D", [(8, 1, 3), (16, 1, 130), (16, 2, 64), (32, 1, 40), (64, 4, 20)])
def test_steps_follow_the_prompt(wk, N, G, D, dtype):
    import torch
    B, T = 3, 20
    p, h0, _ = make(37, B, T, D, N, G, dtype)
    args, kw = call(p)
    state, ys = h0.clone(), []
    for t in range(T):
        at = lambda v: v[:, t].contiguous()   # noqa: E731
        ys.append(wk.ssm_step(at(p["x"]), at(p["dt"]), p["A"], at(p["Bm"]), at(p["Cm"]), state, z=at(p["z"]),
                              dskip=p["dskip"], dt_bias=p["dt_bias"]))
    torch.cuda.synchronize()
    s = ref.Scan(h0=host(h0), **hosts(p))
    want = s.outputs()
    ref.assert_within(torch.stack(ys, 1), want["y"], p["x"].dtype, s.roundings() + N, "y")
    ref.assert_within(state, want["hT"], torch.float32, s.roundings(), "state")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D,N,G,lengths", [(1, 1000, 24, 16, 1, None), (2, 700, 10, 8, 2, [700, 300]),
                                               (1, 513, 20, 64, 1, None), (1, 2048, 7, 32, 1, [1999])])
def test_few_channels_run_in_time_segments(wk, B, T, D, N, G, lengths, dtype):
    """Long sequences of few channels (several time segments): every output against the definition."""
    import torch
    p, h0, more = make(41, B, T, D, N, G, dtype, lengths=lengths)
    args, kw = call(p)
    d = wk.SsmDesc(B, T, D, N, G, wk.WKV7_BF16 if dtype == "bf16" else wk.WKV7_F32, 32)
    import ctypes
    assert wk.lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d)) > 0   # segments
    y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=32, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], **kw)
    torch.cuda.synchronize()
    s = ref.Scan(h0=host(h0), **hosts(p))
    want = s.outputs()
    K = s.roundings()
    ref.assert_within(y, want["y"], p["x"].dtype, K + N, "y")
    ref.assert_within(hT, want["hT"], torch.float32, K, "hT")
    ref.assert_within(ck, (s.h[:, 0:T:16], s.mh[:, 0:T:16]), torch.float32, K, "ckpt")
    check_grads(got, s, more, p)


def test_padding_is_not_read(wk):
    import torch
    for dtype in ("fp32", "bf16"):
        n = (50, 0, 17)
        p, h0, more = make(43, 3, 50, 33, 16, 1, dtype, lengths=list(n))
        outs = []
        for fill in (0.0, float("nan"), float("inf"), -float("inf")):
            q = dict(p, **{k: p[k].clone() for k in ("x", "dt", "Bm", "Cm", "z")})
            dy = more["dy"].clone()
            for b in range(3):
                for k in ("x", "dt", "Bm", "Cm", "z"):
                    q[k][b, n[b]:] = fill
                dy[b, n[b]:] = fill
            args, kw = call(q)
            for bits in (32, 8):
                y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=bits, **kw)
                g = wk.ssm_backward(*args, dy, ck, dhT=more["dhT"], ckpt_bits=bits, **kw)
                outs.append((y, hT, ck) + tuple(g))
        for k, other in enumerate(outs[2:]):
            assert all(torch.equal(a, b) for a, b in zip(outs[k % 2], other))
        y, hT, ck, dx = outs[0][:4]
        assert float(y[1].abs().max()) == 0 and torch.equal(hT[1], h0[1])
        assert float(y[2, 17:].abs().max()) == 0 and float(dx[2, 17:].abs().max()) == 0


def test_extreme_rates(wk):
    """dt far to either side: a rate of zero keeps the state, a large one forgets it;
    nothing overflows."""
    import torch
    p, h0, more = make(47, 2, 40, 48, 16, 1, "fp32", bias=False)
    p["dt"][:, ::2] = -200.0
    p["dt"][:, 1::2] = 90.0
    p["x"][:, 1::2] *= 1e-2
    args, kw = call(p)
    y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=32, **kw)
    g = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], **kw)
    torch.cuda.synchronize()
    s = ref.Scan(h0=host(h0), **hosts(p))
    # here |D A| reaches 90 * 2.5: 10 |D A| + 6 roundings a step where the exponential is not
    # negligible (it is below 2^-126 from |D A| = 88): at most 886 a token
    ref.assert_within(y, s.outputs()["y"], torch.float32, 886 * 40, "y")
    ref.assert_within(hT, s.outputs()["hT"], torch.float32, 886 * 40, "hT")
    want = s.grads(host(more["dy"]), host(more["dhT"]))
    for name in ("dx", "dB", "dC", "dh0"):
        ref.assert_within(getattr(g, name), want[name], torch.float32, 2 * 886 * 40, name)
    assert bool(torch.isfinite(g.ddt).all()) and bool(torch.isfinite(g.dA).all())


def test_small_rates_keep_their_precision(wk):
    """softplus of a far negative argument is its exponential, to 8 roundings (and the exponent's)."""
    import torch
    D = 256
    dt = torch.linspace(-60, 30, D, device="cuda")[None, None].contiguous()
    one = torch.ones(1, 1, 1, 8, device="cuda")
    A = torch.full((D, 8), -1e-30, device="cuda")
    _, h, _ = wk.ssm_forward(torch.ones_like(dt), dt, A, one, one)
    want = np.logaddexp(host(dt)[0, 0], 0)
    off = np.abs(host(h)[0, :, 0] - want) / want
    assert (off <= (10 + 2 * np.abs(host(dt)[0, 0])) * ref.EPS32).all(), off.max() / ref.EPS32


def test_empty(wk):
    import torch
    p, h0, more = make(53, 2, 5, 24, 16, 2, "bf16")
    q = {k: (v[:, :0].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in p.items()}
    args, kw = call(q)
    for bits in (32, 8):
        y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=bits, **kw)
        assert y.shape == (2, 0, 24) and torch.equal(hT, h0) and ck.numel() == 0
        g = wk.ssm_backward(*args, q["x"], ck, dhT=more["dhT"], ckpt_bits=bits, **kw)
        assert torch.equal(g.dh0, more["dhT"])
        assert all(float(v.abs().max()) == 0 for v in (g.dA, g.ddskip, g.ddt_bias))
    _, hT, _ = wk.ssm_forward(*args, **kw)
    assert float(hT.abs().max()) == 0
    q = {k: (v[:0].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in p.items()}
    args, kw = call(q)
    y, hT, ck = wk.ssm_forward(*args, ckpt_bits=32, **kw)
    g = wk.ssm_backward(*args, q["x"], ck, **kw)
    assert y.numel() == 0 and float(g.dA.abs().max()) == 0


def test_repeats_agree_and_other_stream(wk):
    import torch
    p, h0, more = make(59, 2, 400, 520, 16, 1, "bf16")
    args, kw = call(p)
    def once():
        y, hT, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=8, **kw)
        return (y, hT, ck) + tuple(wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], ckpt_bits=8, **kw))
    first = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = once()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,D,G,gate,lengths", [(16, 32, 16, True, None), (16, 48, 16, False, "some"),
                                                (32, 32, 16, True, "some"), (32, 64, 16, False, None)])
def test_gradients_of_many_workgroups(wk, N, D, G, gate, lengths, dtype):
    """More workgroups than the device has compute units (20 rows of 16 groups): the
    backward's variant for two of them on one unit."""
    B, T = 20, 21
    lengths = [t % 24 for t in range(B)] if lengths else None
    p, h0, more = make(59, B, T, D, N, G, dtype, gate=gate, lengths=lengths)
    args, kw = call(p)
    _, _, ck = wk.ssm_forward(*args, h0=h0, ckpt_bits=32, **kw)
    got = wk.ssm_backward(*args, more["dy"], ck, dhT=more["dhT"], **kw)
    check_grads(got, ref.Scan(h0=host(h0), **hosts(p)), more, p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [8, 64])
def test_single_tokens_of_many_rows(wk, N, dtype):
    """Several rows per lane (4096 workgroups and more of one row each); the last lanes
    have fewer."""
    import torch
    B, D = 4099, 6
    p, h0, _ = make(63, B, 1, D, N, 1, dtype)
    at = lambda v: v[:, 0].contiguous()   # noqa: E731
    state = h0.clone()
    y = wk.ssm_step(at(p["x"]), at(p["dt"]), p["A"], at(p["Bm"]), at(p["Cm"]), state, z=at(p["z"]),
                    dskip=p["dskip"], dt_bias=p["dt_bias"])
    s = ref.Scan(h0=host(h0), **hosts(p))
    want = s.outputs()
    ref.assert_within(y[:, None], want["y"], p["x"].dtype, s.roundings() + N, "y")
    ref.assert_within(state, want["hT"], torch.float32, s.roundings(), "state")
