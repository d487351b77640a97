"""The selective scan in 64 bits with a bound on a 32-bit evaluation's error that is
carried through the recurrence: what a decaying state has forgotten is forgotten in
its error too.

A value is an ``F``: what it is (v), the same with every sum over magnitudes (m), and
the error of its 32-bit evaluation in units of 2^-24, half a step of float32 (e).  To
first order in 2^-24, and each with a rounding of its own,

    e(x y) = m(x) e(y) + m(y) e(x) + m(x y),     e(x + y) = e(x) + e(y) + m(x) + m(y),

a sum of n terms in any order n times its magnitudes.  The functions, from their
evaluation by a power of two and a logarithm that are off by a unit in the last
place (two units here):

    exp(x)       the argument's absolute error, and 2
    sigmoid(z)   2 |z| + 6 (z log2 e, rounded twice; the power, the sum, the reciprocal)
    softplus(v)  2 |v| + 10 (the same, then the logarithm's products and sum)
"""

import numpy as np

from tests import _mixers as ref


class F:
    def __init__(self, v, m=None, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.m = np.abs(self.v) if m is None else m
        self.e = np.zeros_like(self.v) + e

    def __mul__(self, o):
        m = self.m * o.m
        return F(self.v * o.v, m, self.m * o.e + o.m * self.e + m)

    def __add__(self, o):
        m = self.m + o.m
        return F(self.v + o.v, m, self.e + o.e + m)

    def __getitem__(self, k):
        return F(self.v[k], self.m[k], self.e[k])

    def sum(self, axis, terms):
        m = self.m.sum(axis)
        return F(self.v.sum(axis), m, self.e.sum(axis) + terms * m)

    def reshape(self, *shape):
        return F(self.v.reshape(shape), self.m.reshape(shape), self.e.reshape(shape))


def stack(parts):
    return F(np.stack([p.v for p in parts], 1), np.stack([p.m for p in parts], 1),
             np.stack([p.e for p in parts], 1))


def sigmoid(z):
    """Of an exact z."""
    s = ref.sigmoid(z)
    return F(s, s, s * (2 * np.abs(z) + 6))


def scan(x, dt, A, Bm, Cm, z=None, dskip=None, dt_bias=None, h0=None, lengths=None, softplus_on=True,
         dy=None, dhT=None, entry=None, segment=0):
    """Every output of the forward, and with dy the gradients, by name.

    entry: the states that the backward's 16-token blocks start from, exact (else the
    forward's own).  segment: tokens of a time segment, whose rates are added up one by
    one (a rounding each) before the exponential of their sum."""
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    width = D // G
    n = ref.row_lengths(lengths, B, T)
    x, Bm, Cm = (ref._masked(v, n) for v in (x, Bm, Cm))
    on = (np.arange(T)[None] < n[:, None])[..., None]      # [B, T, 1]
    v = dt + (0 if dt_bias is None else dt_bias)
    if softplus_on:
        sp, sl = np.logaddexp(v, 0.0), ref.sigmoid(v)
        rate = F(sp * on, e=on * (sp * (2 * np.abs(v) + 10) + sl * np.abs(v)))
        slope = F(sl * on, e=on * sl * (3 * np.abs(v) + 6))
    else:
        rate, slope = F(v * on, e=np.abs(v) * on), F(on * np.ones_like(v))
    skip = F(np.zeros(D) if dskip is None else dskip)
    b = F(np.repeat(Bm, width, axis=2))                    # [B, T, D, N]
    c = F(np.repeat(Cm, width, axis=2))
    u = rate * F(x)
    wide = lambda f: F(f.v[..., None], f.m[..., None], f.e[..., None])   # noqa: E731
    arg = np.abs(rate.v[..., None] * A)
    a = np.exp(rate.v[..., None] * A)
    a = F(a, a, a * (rate.e[..., None] * np.abs(A) + (3 + segment) * arg + 2))
    h = F(np.zeros((B, D, N)) if h0 is None else h0)
    add = wide(u) * b
    before, after = [], []
    for t in range(T):
        if entry is not None and t % 16 == 0:
            h = F(entry[:, t // 16])
        before.append(h)
        h = a[:, t] * h + add[:, t]
        after.append(h)
    out = dict(hT=h)
    if T:
        out["ckpt"] = stack(before[::16])
        after = stack(after)
        y0 = (after * c).sum(3, N) + skip * F(x)
        if z is not None:
            zz = F(z * on)
            s = sigmoid(zz.v)
            gate = zz * s
            y = y0 * gate
        else:
            y = y0
        out["y"] = F(y.v * on, y.m * on, y.e * on)
    if dy is None:
        return out
    dout = F(dy * on if T else dy)
    if z is not None:
        one = F(np.ones_like(s.v))
        out["dz"] = dout * (s * (zz * (one + F(-s.v, s.m, s.e)) + one)) * y0
        back = dout * gate
    else:
        back = dout
    g = F(np.zeros((B, D, N)) if dhT is None else dhT)
    gs, rs = [None] * T, [None] * T
    cdy = wide(back) * c
    for t in reversed(range(T)):
        gs[t] = g + cdy[:, t]
        g = a[:, t] * gs[t]
        rs[t] = g * before[t]
    gs, rs = stack(gs), stack(rs)
    group = lambda f: f.reshape(B, T, G, width, N).sum(3, width)   # noqa: E731
    du = (gs * b).sum(3, N)
    out["dC"], out["dB"] = group(wide(back) * after), group(gs * wide(u))
    out["dx"] = du * rate + back * skip
    ddt = (du * F(x) + (rs * F(A)).sum(3, N)) * slope
    out["ddt"] = ddt
    flat = lambda f: f.reshape(B * T, *f.v.shape[2:]).sum(0, B * T)   # noqa: E731
    out["dA"], out["ddt_bias"] = flat(rs * wide(rate)), flat(ddt)
    out["ddskip"] = flat(back * F(x))
    out["dh0"] = g
    return out


def assert_bound(got, want, dtype, what, tiny=2.0 ** -120):
    """|got - v| <= half a step of dtype at v, and the carried error (1 % on it for the terms of
    second order in 2^-24)."""
    import torch
    half = torch.finfo(dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.v.shape, (what, got.shape, want.v.shape)
    if not got.size:
        return
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} non-finite values"
    inner = 1.01 * want.e * ref.EPS32
    allowed = half * (np.abs(want.v) + inner) + inner + tiny
    far = np.abs(got - want.v) - allowed
    k = far.argmax()
    assert (far <= 0).all(), (f"{what}: off by {np.abs(got - want.v).flat[k]:.3e} at {want.v.flat[k]:.3e}, "
                              f"allowed {allowed.flat[k]:.3e}")


def assert_grads(got, want, dtype):
    import torch
    for name in ("dx", "ddt", "dB", "dC", "dA", "dz", "ddskip", "ddt_bias", "dh0"):
        g = getattr(got, name)
        if g is not None:
            assert_bound(g, want[name], dtype if name in ("dx", "ddt", "dB", "dC", "dz") else torch.float32, name)
