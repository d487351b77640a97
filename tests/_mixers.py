"""The short causal convolution and the selective scan in 64 bits, token by
token (numpy, CPU), with a bound on the rounding error of a 32-bit evaluation.

Every function takes float64 arrays (what the device inputs hold, exactly) and
returns {name: (value, magnitude)}: the magnitude is the same sum with every
term replaced by its absolute value, to which rounding errors are relative.
"""

import numpy as np

EPS32 = 2.0 ** -24   # half a step of float32, relative


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def row_lengths(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


# ---- the convolution --------------------------------------------------------------------------


def conv(x, weight, bias=None, s0=None, lengths=None, silu=False):
    B, T, D = x.shape
    W = weight.shape[1]
    n = row_lengths(lengths, B, T)
    y, mag = np.zeros((B, T, D)), np.zeros((B, T, D))
    sT = np.zeros((B, W - 1, D))
    for b in range(B):
        past = s0[b] if s0 is not None else np.zeros((W - 1, D))
        rows = np.concatenate([past, x[b, :n[b]]])
        sT[b] = rows[n[b]:n[b] + W - 1]
        for t in range(n[b]):
            terms = rows[t:t + W].T * weight
            pre = terms.sum(1) + (0 if bias is None else bias)
            m = np.abs(terms).sum(1) + (0 if bias is None else np.abs(bias))
            # the slope of x sigmoid(x) is at most 1.1, and the sigmoid's own
            # rounding is relative to |pre| <= m (times 1 + |pre| through the exponent)
            y[b, t] = pre * sigmoid(pre) if silu else pre
            mag[b, t] = m * (1.1 + np.abs(y[b, t])) if silu else m
    return dict(y=(y, mag), sT=(sT, np.zeros_like(sT)))


def conv_grads(x, weight, dy, bias=None, s0=None, dsT=None, lengths=None, silu=False):
    B, T, D = x.shape
    W = weight.shape[1]
    n = row_lengths(lengths, B, T)
    out = {k: [np.zeros(s), np.zeros(s)] for k, s in
           dict(dx=(B, T, D), dweight=(D, W), dbias=(D,), ds0=(B, W - 1, D)).items()}
    for b in range(B):
        past = s0[b] if s0 is not None else np.zeros((W - 1, D))
        rows = np.concatenate([past, x[b, :n[b]]])
        drows, mrows = np.zeros_like(rows), np.zeros_like(rows)
        for t in range(n[b]):
            win = rows[t:t + W].T
            e, me = dy[b, t], np.abs(dy[b, t])
            if silu:
                pre = (win * weight).sum(1) + (0 if bias is None else bias)
                m = (np.abs(win * weight)).sum(1) + (0 if bias is None else np.abs(bias))
                s = sigmoid(pre)
                e = e * s * (1 + pre * (1 - s))
                me = me * 1.1 * (1 + m)   # the slope's own slope is below 0.5, its value below 1.1
            drows[t:t + W] += (e[:, None] * weight).T
            mrows[t:t + W] += (me[:, None] * np.abs(weight)).T
            out["dweight"][0] += e[:, None] * win
            out["dweight"][1] += me[:, None] * np.abs(win)
            out["dbias"][0] += e
            out["dbias"][1] += me
        if dsT is not None:
            drows[n[b]:n[b] + W - 1] += dsT[b]
            mrows[n[b]:n[b] + W - 1] += np.abs(dsT[b])
        out["ds0"][0][b], out["ds0"][1][b] = drows[:W - 1], mrows[:W - 1]
        out["dx"][0][b, :n[b]], out["dx"][1][b, :n[b]] = drows[W - 1:], mrows[W - 1:]
    if bias is None:
        del out["dbias"]
    return {k: tuple(v) for k, v in out.items()}


# ---- the scan ---------------------------------------------------------------------------------


def softplus(x):
    return np.logaddexp(x, 0.0)


def _masked(v, n):
    v = np.array(v, dtype=np.float64)
    for b in range(v.shape[0]):
        v[b, n[b]:] = 0
    return v


class Scan:
    """Rates, states (h[:, t] before token t) and read-outs of one call."""

    def __init__(self, x, dt, A, Bm, Cm, z=None, dskip=None, dt_bias=None, h0=None, lengths=None,
                 softplus_on=True, entry=None):
        B, T, D = x.shape
        G, N = Bm.shape[2:]
        self.n = row_lengths(lengths, B, T)
        self.shape, self.A, self.width = (B, T, D, N, G), A, D // G
        self.x, Bm, Cm = (_masked(v, self.n) for v in (x, Bm, Cm))
        self.z = None if z is None else _masked(z, self.n)
        self.v = dt + (0 if dt_bias is None else dt_bias)
        self.rate = _masked(softplus(self.v) if softplus_on else self.v, self.n)
        self.softplus_on, self.dskip = softplus_on, np.zeros(D) if dskip is None else dskip
        self.bm, self.cm = (np.repeat(v, self.width, axis=2) for v in (Bm, Cm))   # [B, T, D, N]
        self.h, self.mh = np.zeros((B, T + 1, D, N)), np.zeros((B, T + 1, D, N))
        if h0 is not None:
            self.h[:, 0], self.mh[:, 0] = h0, np.abs(h0)
        self.a = np.exp(self.rate[..., None] * A)
        u = (self.rate * self.x)[..., None]
        self.before, self.mbefore = np.zeros((B, T, D, N)), np.zeros((B, T, D, N))
        for t in range(T):
            if entry is not None and t % 16 == 0:   # the block starts from a given state
                self.before[:, t], self.mbefore[:, t] = entry[:, t // 16], np.abs(entry[:, t // 16])
            else:
                self.before[:, t], self.mbefore[:, t] = self.h[:, t], self.mh[:, t]
            self.h[:, t + 1] = self.a[:, t] * self.before[:, t] + u[:, t] * self.bm[:, t]
            self.mh[:, t + 1] = self.a[:, t] * self.mbefore[:, t] + np.abs(u[:, t] * self.bm[:, t])
        self.y0 = (self.h[:, 1:] * self.cm).sum(3) + self.dskip * self.x
        self.my0 = (self.mh[:, 1:] * np.abs(self.cm)).sum(3) + np.abs(self.dskip * self.x)

    def roundings(self):
        """Roundings of T steps of the state: 10 |D A| + 6 each, the exponent's among them."""
        T = self.shape[1]
        return T * (10 * float(np.abs(self.rate[..., None] * self.A).max(initial=0)) + 6) + 64

    def outputs(self):
        y, m = self.y0, self.my0
        if self.z is not None:
            g = self.z * sigmoid(self.z)
            y, m = y * g, m * np.abs(g) * (1 + np.abs(self.z))
        return dict(y=(y, m), hT=(self.h[:, -1], self.mh[:, -1]))

    def grads(self, dout, dhT=None):
        B, T, D, N, G = self.shape
        dout = _masked(dout, self.n)
        if self.z is not None:
            s = sigmoid(self.z)
            dy = dout * self.z * s
            mdy = np.abs(dy) * (1 + np.abs(self.z))
            slope = s * (1 + self.z * (1 - s))
            dz = (dout * self.y0 * slope, np.abs(dout) * self.my0 * 1.1 * (1 + np.abs(self.z)))
        else:
            dy, mdy, dz = dout, np.abs(dout), None
        g, mg = np.zeros((B, D, N)), np.zeros((B, D, N))
        if dhT is not None:
            g, mg = dhT.copy(), np.abs(dhT)
        out = {k: [np.zeros(s), np.zeros(s)] for k, s in
               dict(dx=(B, T, D), ddt=(B, T, D), dB=(B, T, G, N), dC=(B, T, G, N), dA=(D, N)).items()}
        absA, absb, absc = np.abs(self.A), np.abs(self.bm), np.abs(self.cm)
        group = lambda v: v.reshape(B, G, self.width, N).sum(2)   # noqa: E731
        slope = sigmoid(self.v) if self.softplus_on else np.ones_like(self.v)
        slope = _masked(slope, self.n)
        for t in reversed(range(T)):
            x = self.x[:, t]
            g, mg = g + dy[:, t, :, None] * self.cm[:, t], mg + mdy[:, t, :, None] * absc[:, t]
            for k, (gg, hh, xx, yy, bb, rr) in enumerate((
                    (g, self.h[:, t + 1], x, dy[:, t], self.bm[:, t], self.rate[:, t]),
                    (mg, self.mh[:, t + 1], np.abs(x), mdy[:, t], absb[:, t], np.abs(self.rate[:, t])))):
                out["dC"][k][:, t] = group(yy[..., None] * hh)
                out["dB"][k][:, t] = group(gg * (rr * xx)[..., None])
                du = (gg * bb).sum(-1)
                r = gg * self.a[:, t] * (self.before[:, t] if k == 0 else self.mbefore[:, t])
                sr = (r * (self.A if k == 0 else absA)).sum(-1)
                out["dx"][k][:, t] = du * rr + yy * (self.dskip if k == 0 else np.abs(self.dskip))
                out["ddt"][k][:, t] = (du * xx + sr) * slope[:, t]
                out["dA"][k] += (r * rr[..., None]).sum(0)
            g, mg = g * self.a[:, t], mg * self.a[:, t]
        out = {k: tuple(v) for k, v in out.items()}
        out["dh0"] = (g, mg)
        out["dz"] = dz
        out["ddskip"] = ((dy * self.x).sum((0, 1)), (mdy * np.abs(self.x)).sum((0, 1)))
        out["ddt_bias"] = tuple(v.sum((0, 1)) for v in out["ddt"])
        return out


def assert_within(got, want, dtype, roundings, what, tiny=2.0 ** -120):
    """|got - value| <= half a step of dtype at the value + roundings 2^-24 magnitude."""
    import torch
    value, mag = want
    half = torch.finfo(dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    # Where the definition itself leaves float32's range (a growing state), nothing is compared:
    # below 2^100 every factor of a sum's terms is in range with the others above 2^-27.
    fits = mag < 2.0 ** 100
    got, value, mag = got[fits], value[fits], mag[fits]
    if not got.size:
        return
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    inner = roundings * EPS32 * mag
    far = np.abs(got - value) - (half * (np.abs(value) + inner) + inner + tiny)
    assert (far <= 0).all(), (f"{what}: off by {np.abs(got - value).flat[far.argmax()]:.3e} at "
                              f"{value.flat[far.argmax()]:.3e}, allowed {(half * np.abs(value) + inner).flat[far.argmax()]:.3e}")
