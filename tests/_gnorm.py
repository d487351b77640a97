"""The group norm with an activation in 64 bits (torch, CPU), its gradients written out from
the formulas, and bounds on the rounding of a 32-bit evaluation.

Every function returns {name: (value, magnitude)}; the error of a 32-bit evaluation is a
number of roundings (2^-24) of the magnitude, which counts how errors of the moments and of
the values under them are passed on:

  n      u carries up to 8 roundings (the gate's sigmoid: 2 |z| + 6, here |z| <= 6), each of up
         to a = max |u| of the group; the mean adds W of them, so a deviation is off by
         (W + 20) 2^-24 a, and n by that times rstd, its own variance error W + 4 relative
"""

import torch


def sig(x):
    return 1 / (1 + torch.exp(-x))


def norm(x, groups, gamma=None, beta=None, z=None, gate_first=False, silu=False, center=True, eps=1e-5, dy=None):
    d = lambda t: None if t is None else t.detach().double().cpu()   # noqa: E731
    x, gamma, beta, z, dy = (d(t) for t in (x, gamma, beta, z, dy))
    D = x.shape[-1]
    W = D // groups
    v = lambda t: t.reshape(-1, groups, W)   # noqa: E731
    shape = x.shape
    x = v(x)
    z = None if z is None else v(z)
    s = None if z is None else z * sig(z)
    g = torch.ones(D, dtype=torch.float64) if gamma is None else gamma
    b = torch.zeros(D, dtype=torch.float64) if beta is None else beta
    g, b = g.view(groups, W), b.view(groups, W)
    u = x * s if gate_first else x
    mean = u.mean(2, keepdim=True) if center else torch.zeros_like(u[..., :1])
    r = 1 / torch.sqrt((u - mean).square().mean(2, keepdim=True) + eps)
    n = (u - mean) * r
    a = u.abs().amax(2, keepdim=True)
    en = n.abs() + a * r                      # times W + 32 roundings
    o = g * n + b
    eo = g.abs() * en + b.abs()
    q = sig(o)
    act = o * q if silu else o
    eact = eo * 1.1 + act.abs() * (1 + o.abs()) if silu else eo
    y = act * s if z is not None and not gate_first else act
    ey = eact * s.abs() * (1 + z.abs()) if z is not None and not gate_first else eact
    out = dict(y=(y, ey))
    if dy is not None:
        e = v(dy)
        ee = e.abs()
        if z is not None and not gate_first:
            dgate, edgate = e * act, ee * eact
            e, ee = e * s, ee * s.abs() * (1 + z.abs())
        if silu:
            slope = q * (1 + o * (1 - q))
            e, ee = e * slope, ee * (slope.abs() + 1.1 + eo)   # the slope's own slope is below 0.5
        out["dgamma"] = (e * n, ee * (n.abs() + en))
        out["dbeta"] = (e, ee)
        f, ef = e * g, ee * g.abs()
        sf = f.mean(2, keepdim=True) if center else 0
        esf = ef.mean(2, keepdim=True) if center else 0
        sfn, esfn = (f * n).mean(2, keepdim=True), (ef * (n.abs() + en)).mean(2, keepdim=True)
        du = r * (f - n * sfn - sf)
        edu = r * (ef + (n.abs() + en) * esfn + esf) * (1 + a * a * r * r)
        if gate_first:
            dgate, edgate = du * x, edu * x.abs()
            du, edu = du * s, edu * s.abs() * (1 + z.abs())
        out["dx"] = (du, edu)
        if z is not None:
            qz = sig(z)
            out["dz"] = (dgate * qz * (1 + z * (1 - qz)), edgate * 1.1 * (1 + z.abs()))
        for k in ("dgamma", "dbeta"):
            out[k] = tuple(t.sum(0).reshape(D) for t in out[k])
    return {k: tuple(t if k in ("dgamma", "dbeta") else t.reshape(shape) for t in p) for k, p in out.items()}
