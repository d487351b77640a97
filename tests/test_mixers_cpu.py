"""The short convolution and the selective scan without a GPU: the 64-bit
definition's gradients against differences, sizes, and every refusal.  The
pointers are made up, so only calls that fail validation or have nothing to do
are made: each refusal names the entry points it is made on."""

import ctypes
import os

import numpy as np
import pytest

import rwkv_wkv7_delta_amd as wk
from tests import _mixers as ref

FAKE = 1 << 20   # aligned, never dereferenced
C = ctypes.byref


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wk.LIB_PATH):
        pytest.skip("libwkv7.so not built")
    return wk.lib()


# ---- the definition ---------------------------------------------------------------------------


def directional(f, args, grads, rng, eps=1e-6):
    """sum <grad, direction> against the central difference of f along random directions."""
    for name, g in grads.items():
        v = args[name]
        d = rng.normal(size=v.shape)
        hi, lo = (f(dict(args, **{name: v + s * eps * d})) for s in (1, -1))
        num, ana = (hi - lo) / (2 * eps), float((g * d).sum())
        # truncation eps^2 and cancellation 2^-53 / eps, relative to the objective's size
        assert abs(num - ana) <= 1e-6 * (abs(ana) + abs(hi) + 1), (name, num, ana)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("W,T,lengths", [(2, 5, None), (4, 2, None), (4, 7, [7, 1]), (3, 6, [0, 4])])
def test_conv_gradients_against_differences(W, T, lengths, silu):
    rng = np.random.default_rng(1)
    B, D = 2, 3
    a = dict(x=rng.normal(size=(B, T, D)), weight=rng.normal(size=(D, W)), bias=rng.normal(size=D),
             s0=rng.normal(size=(B, W - 1, D)))
    dy, dsT = rng.normal(size=(B, T, D)), rng.normal(size=(B, W - 1, D))

    def f(v):
        o = ref.conv(lengths=lengths, silu=silu, **v)
        return float((o["y"][0] * dy).sum() + (o["sT"][0] * dsT).sum())

    g = ref.conv_grads(dy=dy, dsT=dsT, lengths=lengths, silu=silu, **a)
    directional(f, a, dict(x=g["dx"][0], weight=g["dweight"][0], bias=g["dbias"][0], s0=g["ds0"][0]), rng)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("T,lengths", [(1, None), (19, None), (18, [18, 0, 7])])
def test_scan_gradients_against_differences(T, lengths, gate, softplus):
    rng = np.random.default_rng(2)
    B, D, N, G = 3, 4, 5, 2
    a = dict(x=rng.normal(size=(B, T, D)), dt=rng.uniform(-1, 1, size=(B, T, D)), A=-rng.uniform(0.1, 1, size=(D, N)),
             Bm=rng.normal(size=(B, T, G, N)), Cm=rng.normal(size=(B, T, G, N)), dskip=rng.normal(size=D),
             dt_bias=rng.uniform(0, 1, size=D), h0=rng.normal(size=(B, D, N)))
    if gate:
        a["z"] = rng.normal(size=(B, T, D))
    dy, dhT = rng.normal(size=(B, T, D)), rng.normal(size=(B, D, N))

    def f(v):
        o = ref.Scan(lengths=lengths, softplus_on=softplus, **v).outputs()
        return float((o["y"][0] * dy).sum() + (o["hT"][0] * dhT).sum())

    g = ref.Scan(lengths=lengths, softplus_on=softplus, **a).grads(dy, dhT)
    names = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", dskip="ddskip", dt_bias="ddt_bias", h0="dh0")
    if gate:
        names["z"] = "dz"
    directional(f, a, {k: g[n][0] for k, n in names.items()}, rng)


def test_scan_closed_form():
    """A = 0, unit rates and no gate: the state is the running sum of x_t B_t."""
    rng = np.random.default_rng(3)
    x, b, c = rng.normal(size=(1, 6, 2)), rng.normal(size=(1, 6, 1, 8)), rng.normal(size=(1, 6, 1, 8))
    s = ref.Scan(x, np.ones((1, 6, 2)), np.zeros((2, 8)), b, c, softplus_on=False)
    h = np.cumsum(x[..., None] * b, axis=1)
    assert np.allclose(s.h[:, 1:], h) and np.allclose(s.outputs()["y"][0], (h * c).sum(-1))


# ---- sizes ------------------------------------------------------------------------------------


def test_sizes(L):
    d = wk.SsmDesc(2, 33, 5, 16, 1, wk.WKV7_BF16, 32)
    assert wk.ssm_ckpt_bytes(d) == 2 * 3 * 5 * 16 * 4
    d.ckpt_bits = 8
    assert wk.ssm_ckpt_bytes(d) == 2 * 3 * 5 * 16 + 2 * 3 * 5 * 4
    d = wk.SsmDesc(1, 1, 1, 8, 1, wk.WKV7_F32, 8)
    assert wk.ssm_ckpt_bytes(d) == 16 + 4   # the scales start at the next 16-byte boundary
    d.ckpt_bits = 0
    assert wk.ssm_ckpt_bytes(d) == 0
    assert wk.ssm_ckpt_bytes(wk.SsmDesc(1, 0, 4, 8, 1, wk.WKV7_F32, 8)) == 0
    assert wk.ssm_ckpt_bytes(wk.SsmDesc(1, 8, 4, 12, 1, wk.WKV7_F32, 8)) == 0
    assert L.wkv7_ssm_ckpt_bytes(None) == 0 and L.wkv7_ssm_forward_workspace_bytes(None) == 0
    assert L.wkv7_ssm_backward_workspace_bytes(None) == 0 and L.wkv7_conv_backward_workspace_bytes(None) == 0
    # no time segments at many channels
    assert L.wkv7_ssm_forward_workspace_bytes(C(wk.SsmDesc(8, 4096, 2048, 16, 1, wk.WKV7_BF16, 0))) == 0


# ---- refusals at the C ABI ----------------------------------------------------------------------


CONV_OK = dict(B=1, T=8, D=16, W=4, dtype=wk.WKV7_BF16, silu=1)


FORWARD, BACKWARD, STEP = 0, 1, 2
ALL = (FORWARD, BACKWARD, STEP)


def refusals(calls, which):
    return [calls[k]() for k in which]


def conv(L, d, which, **over):
    """Statuses of the named convolution entry points, with valid pointers but for `over`."""
    a = dict(weight=FAKE, bias=FAKE, lengths=None, x=FAKE, s0=None, y=FAKE, sT=None, dy=FAKE, dsT=None, dx=FAKE,
             dweight=FAKE, dbias=FAKE, ds0=None, ws=FAKE, wsb=1 << 30, state=FAKE)
    a.update(over)
    d = d if d is None else C(d)
    return refusals((
        lambda: L.wkv7_conv_forward(d, a["weight"], a["bias"], a["lengths"], a["x"], a["s0"], a["y"], a["sT"], None),
        lambda: L.wkv7_conv_backward(d, a["weight"], a["bias"], a["lengths"], a["x"], a["s0"], a["dy"], a["dsT"],
                                     a["dx"], a["dweight"], a["dbias"], a["ds0"], a["ws"], a["wsb"], None),
        lambda: L.wkv7_conv_step(d, a["weight"], a["bias"], a["x"], a["state"], a["y"], None)), which)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, 1), ("T", -1, 1), ("D", -1, 1), ("silu", 2, 1), ("W", 1, 2), ("W", 5, 2), ("dtype", 2, 2),
    ("T", 2 ** 31 - 1, 2), ("D", 2 ** 31 - 1, 2)])
def test_conv_descriptor(L, field, value, status):
    d = wk.ConvDesc(**dict(CONV_OK, **{field: value}))
    assert conv(L, d, ALL) == [status] * 3
    assert L.wkv7_conv_backward_workspace_bytes(C(d)) == 0


def test_conv_sizes_that_would_wrap(L):
    for over in (dict(B=1 << 20, T=1 << 20, D=1 << 20), dict(B=2 ** 31 - 1, T=2 ** 31 - 100, D=1 << 20),
                 dict(B=1 << 28, T=1, D=8)):
        assert conv(L, wk.ConvDesc(**dict(CONV_OK, **over)), ALL) == [wk.WKV7_ERR_UNSUPPORTED] * 3


def test_conv_pointers(L):
    ok, bad = wk.ConvDesc(**CONV_OK), wk.WKV7_ERR_INVALID_ARG
    assert conv(L, None, ALL) == [bad] * 3
    for name in ("weight", "x", "bias"):
        assert conv(L, ok, ALL, **{name: FAKE + 8}) == [bad] * 3
    for name in ("weight", "x"):
        assert conv(L, ok, ALL, **{name: None}) == [bad] * 3
    for name, which in (("y", FORWARD), ("s0", FORWARD), ("sT", FORWARD), ("dy", BACKWARD), ("dx", BACKWARD),
                        ("dweight", BACKWARD), ("dbias", BACKWARD), ("ds0", BACKWARD), ("dsT", BACKWARD),
                        ("s0", BACKWARD), ("ws", BACKWARD), ("state", STEP), ("y", STEP)):
        assert conv(L, ok, (which,), **{name: FAKE + 4}) == [bad], name
    for name, which in (("y", FORWARD), ("dy", BACKWARD), ("dx", BACKWARD), ("dweight", BACKWARD),
                        ("dbias", BACKWARD), ("state", STEP), ("y", STEP)):
        assert conv(L, ok, (which,), **{name: None}) == [bad], name
    assert conv(L, ok, (FORWARD, BACKWARD), lengths=FAKE + 2) == [bad] * 2
    assert conv(L, ok, (BACKWARD,), bias=None) == [bad]   # a gradient for a bias that is not there
    assert conv(L, ok, (BACKWARD,), ws=None) == [wk.WKV7_ERR_WORKSPACE]
    need = L.wkv7_conv_backward_workspace_bytes(C(ok))
    assert need > 0 and conv(L, ok, (BACKWARD,), wsb=need - 1) == [wk.WKV7_ERR_WORKSPACE]
    # nothing to do
    assert conv(L, wk.ConvDesc(**dict(CONV_OK, D=0)), ALL) == [wk.WKV7_OK] * 3
    assert conv(L, wk.ConvDesc(**dict(CONV_OK, B=0)), (FORWARD, STEP)) == [wk.WKV7_OK] * 2


SSM_OK = dict(B=1, T=8, D=16, N=16, G=2, dtype=wk.WKV7_BF16, ckpt_bits=32)


def ssm(L, d, which, **over):
    """Statuses of the named scan entry points, with valid pointers but for `over`."""
    a = dict(A=FAKE, dskip=FAKE, dt_bias=FAKE, lengths=None, softplus=1, x=FAKE, dt=FAKE, Bm=FAKE, Cm=FAKE, z=FAKE,
             h0=None, y=FAKE, hT=None, ckpt=FAKE, ws=FAKE, wsb=1 << 40, dy=FAKE, dhT=None, state=FAKE, dx=FAKE,
             ddt=FAKE, dBm=FAKE, dCm=FAKE, dz=FAKE, dA=FAKE, ddskip=FAKE, ddt_bias=FAKE, dh0=None, params=True)
    a.update(over)
    p = C(wk.SsmParams(a["A"], a["dskip"], a["dt_bias"], a["lengths"], a["softplus"])) if a["params"] else None
    g = wk.SsmGradPointers(*(a[k] for k in ("dx", "ddt", "dBm", "dCm", "dz", "dA", "ddskip", "ddt_bias", "dh0")))
    d = d if d is None else C(d)
    ins = [a[k] for k in ("x", "dt", "Bm", "Cm", "z")]
    return refusals((
        lambda: L.wkv7_ssm_forward(d, p, *ins, a["h0"], a["y"], a["hT"], a["ckpt"], a["ws"], a["wsb"], None),
        lambda: L.wkv7_ssm_backward(d, p, *ins, a["dy"], a["dhT"], a["ckpt"], C(g), a["ws"], a["wsb"], None),
        lambda: L.wkv7_ssm_step(d, p, *ins, a["state"], a["y"], None)), which)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, 1), ("T", -1, 1), ("D", -16, 1), ("G", 0, 1), ("G", -1, 1), ("G", 3, 1), ("N", 4, 2), ("N", 24, 2),
    ("N", 128, 2), ("N", 0, 2), ("dtype", 5, 2), ("ckpt_bits", 16, 2), ("ckpt_bits", -8, 2), ("T", 2 ** 31 - 1, 2),
    ("D", 1 << 23, 2)])
def test_ssm_descriptor(L, field, value, status):
    d = wk.SsmDesc(**dict(SSM_OK, **{field: value}))
    assert ssm(L, d, ALL) == [status] * 3
    assert wk.ssm_ckpt_bytes(d) == 0 and L.wkv7_ssm_backward_workspace_bytes(C(d)) == 0
    assert L.wkv7_ssm_forward_workspace_bytes(C(d)) == 0


def test_ssm_sizes_that_would_wrap(L):
    for over in (dict(B=1 << 20, T=1 << 20, D=1 << 20), dict(B=2 ** 31 - 1, T=2 ** 31 - 100, D=1 << 22),
                 dict(B=1 << 14, T=1, D=1 << 16), dict(B=1 << 10, T=1 << 25, D=1 << 10, G=1 << 10),
                 dict(D=1 << 20, G=1 << 19)):
        assert ssm(L, wk.SsmDesc(**dict(SSM_OK, **over)), ALL) == [wk.WKV7_ERR_UNSUPPORTED] * 3


def test_ssm_pointers(L):
    ok, bad = wk.SsmDesc(**SSM_OK), wk.WKV7_ERR_INVALID_ARG
    assert ssm(L, None, ALL) == [bad] * 3 and ssm(L, ok, ALL, params=False) == [bad] * 3
    for name in ("A", "x", "dt", "Bm", "Cm"):
        assert ssm(L, ok, ALL, **{name: None}) == [bad] * 3, name
    for name in ("A", "x", "dt", "Bm", "Cm", "z", "dskip", "dt_bias"):
        assert ssm(L, ok, ALL, **{name: FAKE + 8}) == [bad] * 3, name
    assert ssm(L, ok, ALL, softplus=2) == [bad] * 3 and ssm(L, ok, ALL, lengths=FAKE + 1) == [bad] * 3
    assert ssm(L, ok, (STEP,), lengths=FAKE) == [bad]   # a step has no lengths
    for name, which in (("y", FORWARD), ("h0", FORWARD), ("hT", FORWARD), ("ckpt", FORWARD), ("ws", FORWARD),
                        ("dy", BACKWARD), ("dhT", BACKWARD), ("ckpt", BACKWARD), ("dx", BACKWARD),
                        ("ddt", BACKWARD), ("dBm", BACKWARD), ("dCm", BACKWARD), ("dz", BACKWARD),
                        ("dA", BACKWARD), ("ddskip", BACKWARD), ("ddt_bias", BACKWARD), ("dh0", BACKWARD),
                        ("ws", BACKWARD), ("state", STEP), ("y", STEP)):
        assert ssm(L, ok, (which,), **{name: FAKE + 4}) == [bad], name
    for name, which in (("y", FORWARD), ("ckpt", FORWARD), ("dy", BACKWARD), ("ckpt", BACKWARD), ("dx", BACKWARD),
                        ("ddt", BACKWARD), ("dBm", BACKWARD), ("dCm", BACKWARD), ("dz", BACKWARD),
                        ("dA", BACKWARD), ("ddskip", BACKWARD), ("ddt_bias", BACKWARD), ("state", STEP),
                        ("y", STEP)):
        assert ssm(L, ok, (which,), **{name: None}) == [bad], name
    # a gradient for what is not there, a checkpoint that was not asked for
    for name in ("z", "dskip", "dt_bias"):
        assert ssm(L, ok, (BACKWARD,), **{name: None}) == [bad], name
    none = wk.SsmDesc(**dict(SSM_OK, ckpt_bits=0))
    assert ssm(L, none, (FORWARD, BACKWARD)) == [bad, wk.WKV7_ERR_UNSUPPORTED]
    assert ssm(L, ok, (BACKWARD,), ws=None) == [wk.WKV7_ERR_WORKSPACE]
    need = L.wkv7_ssm_backward_workspace_bytes(C(ok))
    assert need > 0 and ssm(L, ok, (BACKWARD,), wsb=need - 1) == [wk.WKV7_ERR_WORKSPACE]
    long = wk.SsmDesc(**dict(SSM_OK, T=4096))
    need = L.wkv7_ssm_forward_workspace_bytes(C(long))
    assert need > 0 and ssm(L, long, (FORWARD,), wsb=need - 1) == [wk.WKV7_ERR_WORKSPACE]
    assert ssm(L, wk.SsmDesc(**dict(SSM_OK, D=0)), ALL) == [wk.WKV7_OK] * 3
    assert ssm(L, wk.SsmDesc(**dict(SSM_OK, B=0)), (FORWARD, STEP)) == [wk.WKV7_OK] * 2


# ---- refusals in the binding --------------------------------------------------------------------


def test_binding_takes_device_tensors_only():
    import torch
    x = torch.zeros(1, 4, 16)
    with pytest.raises(ValueError):
        wk.conv_forward(x, torch.zeros(16, 4))
    with pytest.raises(ValueError):
        wk.conv_backward(x, torch.zeros(16, 4), x)
    with pytest.raises(ValueError):
        wk.conv_step(x[:, 0], torch.zeros(16, 4), x[:, :3])
    b = torch.zeros(1, 4, 1, 16)
    with pytest.raises(ValueError):
        wk.ssm_forward(x, x, torch.zeros(16, 16), b, b)
    with pytest.raises(ValueError):
        wk.ssm_backward(x, x, torch.zeros(16, 16), b, b, x, torch.zeros(1, 1, 16, 16))
    with pytest.raises(ValueError):
        wk.ssm_backward(x, x, torch.zeros(16, 16), b, b, x, x, ckpt_bits=16)
    with pytest.raises(ValueError):
        wk.ssm_step(x[:, 0], x[:, 0], torch.zeros(16, 16), b[:, 0], b[:, 0], torch.zeros(1, 16, 16))
    with pytest.raises(TypeError):
        wk.conv_forward(x.half(), torch.zeros(16, 4))
    with pytest.raises(ValueError):
        wk.conv_forward(x[0], torch.zeros(16, 4))


def test_launches_of_too_many_threads_are_refused():
    """Rows of few channels: small tensors, but a workgroup (512 threads) or a wave each."""
    L = wk.lib()
    for over in (dict(B=1 << 24, D=1, T=1), dict(B=1 << 27, D=1, T=1), dict(B=64, D=1, T=1 << 25)):
        assert conv(L, wk.ConvDesc(**dict(CONV_OK, **over)), ALL) == [wk.WKV7_ERR_UNSUPPORTED] * 3
    for over in (dict(B=1 << 23, D=1, G=1, T=1), dict(B=1 << 12, D=1 << 12, G=1 << 12, T=1),
                 dict(B=1 << 12, D=64, G=1, N=16, T=1 << 17)):   # the last: B T G N of 2^33
        assert ssm(L, wk.SsmDesc(**dict(SSM_OK, **over)), ALL) == [wk.WKV7_ERR_UNSUPPORTED] * 3
