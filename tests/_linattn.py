"""Linear attention with one decay per head in 64 bits, token by token (torch, CPU), and
bounds on the rounding of the kernels.

The magnitude of an output is the same formula over absolute values; rounding errors are
relative to it.
"""

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def rows_of(v, lengths=None, starts=None):
    """(first token, tokens) of every row of the flattened token tensor."""
    if starts is not None:
        edges = [int(x) for x in starts]
        return [(a, b - a) for a, b in zip(edges, edges[1:])]
    B, T = v.shape[:2]
    n = [T] * B if lengths is None else [max(0, min(T, int(x))) for x in lengths]
    return [(b * T, n[b]) for b in range(B)]


def one_row(q, k, v, decay, s0, scale, dy=None, dsT=None):
    """One row: q, k [n, H, N], v [n, H, P], decay [n, H]; with dy its gradients too."""
    n, H, P = v.shape
    S, states, y = s0, [s0], torch.zeros_like(v)
    for t in range(n):
        S = decay[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
        y[t] = scale * (S * q[t][:, None, :]).sum(-1)
        states.append(S)
    out = dict(y=y, sT=S, states=states)
    if dy is None:
        return out
    D = torch.zeros_like(S) if dsT is None else dsT
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(decay)
    for t in reversed(range(n)):
        D = D + scale * dy[t][:, :, None] * q[t][:, None, :]
        dq[t] = scale * (states[t + 1] * dy[t][:, :, None]).sum(1)
        dk[t] = (D * v[t][:, :, None]).sum(1)
        dv[t] = (D * k[t][:, None, :]).sum(2)
        D = decay[t][:, None, None] * D
        dg[t] = (D * states[t]).sum((1, 2))
    return dict(out, dq=dq, dk=dk, dv=dv, dg=dg, ds0=D)


def reference(q, k, v, g, *, s0=None, lengths=None, starts=None, scale=1.0, dy=None, dsT=None):
    """{name: (value, magnitude)} over the whole call; tokens that no row has are NaN."""
    d = lambda x: None if x is None else x.detach().double().cpu()   # noqa: E731
    q, k, v, g, s0, dy, dsT = (d(x) for x in (q, k, v, g, s0, dy, dsT))
    rows = rows_of(v, lengths, starts)
    lead = v.shape[:-2]
    H, P, (G, N) = v.shape[-2], v.shape[-1], q.shape[-2:]
    flat = lambda x: None if x is None else x.reshape(-1, *x.shape[len(lead):])   # noqa: E731
    rep = lambda x: x.repeat_interleave(H // G, 1)   # noqa: E731
    g = g.expand(*lead, H) if g.dim() == 1 and len(lead) + 1 > 1 and g.shape == (H,) else g
    q, k, v, g, dy = (flat(x) for x in (q, k, v, g, dy))
    size = dict(y=(H, P), dq=(G, N), dk=(G, N), dv=(H, P), dg=(H,))
    keep = 0.0 if starts is None else float("nan")
    out = {}
    for sign in (0, 1):
        a = (lambda x: x) if sign == 0 else (lambda x: None if x is None else x.abs())
        got = {name: torch.full((v.shape[0], *s), keep, dtype=torch.float64) for name, s in size.items()}
        ends = dict(sT=[], ds0=[])
        for b, (i, n) in enumerate(rows):
            j = slice(i, i + n)
            first = torch.zeros(H, P, N, dtype=torch.float64) if s0 is None else s0[b]
            r = one_row(a(rep(q[j])), a(rep(k[j])), a(v[j]), torch.exp(g[j]), a(first), abs(scale) if sign else scale,
                        None if dy is None else a(dy[j]), None if dsT is None else a(dsT[b]))
            got["y"][j] = r["y"]
            ends["sT"].append(r["sT"])
            if dy is None:
                continue
            ends["ds0"].append(r["ds0"])
            for name in ("dq", "dk"):
                got[name][j] = r[name].view(n, G, H // G, N).sum(2)
            got["dv"][j] = r["dv"]
            if sign:
                # a tile's sums for dg pass through all of its pairs, which cancel
                x = (a(rep(q[j])) * r["dq"]).sum(2) + (a(rep(k[j])) * r["dk"]).sum(2)
                for t in range(0, n, 64):
                    r["dg"][t:t + 64] += 2.0 ** -12 * x[t:t + 64].sum(0)
            got["dg"][j] = r["dg"]
        for name, x in list(got.items()) + [(m, torch.stack(e)) for m, e in ends.items() if e]:
            if name in ("y", "sT") or dy is not None:
                x = x.reshape(*lead, *x.shape[1:]) if name in size else x
                out[name] = (x,) if sign == 0 else out[name] + (x,)
    return out


def roundings(T, N, P):
    """Of a 32-bit evaluation: a tile's products add up to 64 terms three times (the parts of a
    32-bit operand) and scale them by exponentials (of arguments up to 16 in what counts: 32
    roundings), a state passes through all tiles, a read-out adds N or P and 64 terms more."""
    return 256 * ((T + 63) // 64) + N + P + 256


def assert_within(got, want, dtype, K, what, inner=0):
    """|got - value| <= half a step of dtype at value, `inner` half steps of the magnitude (weights
    and states that are rounded to dtype inside) and K roundings of 32 bits of it."""
    value, mag = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    on = ~torch.isnan(value)
    got, value, mag = got[on], value[on], mag[on]
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values are not finite"
    half = HALF[dtype]
    e = (inner * half + K * 2.0 ** -24) * mag
    far = (got - value).abs() - (half * (value.abs() + e) + e + 2.0 ** -100)
    k = far.argmax()
    assert far.max() <= 0, (f"{what}: off by {(got - value).abs()[k]:.3e} at {value[k]:.3e} (element {int(k)} of "
                            f"{got.numel()}), allowed {(half * value.abs() + e)[k]:.3e}")
