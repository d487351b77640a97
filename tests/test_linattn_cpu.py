"""Linear attention, the group norm and the slots without a GPU: the 64-bit definitions'
gradients against differences and closed forms, sizes, and every refusal.  The pointers
are made up, so only calls that fail validation or have nothing to do are made."""

import ctypes
import os

import pytest
import torch

import rwkv_wkv7_delta_amd as wk
from tests import _gnorm, _linattn

FAKE = 1 << 20   # aligned, never dereferenced
C = ctypes.byref


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wk.LIB_PATH):
        pytest.skip("libwkv7.so not built")
    return wk.lib()


# ---- the definitions --------------------------------------------------------------------------


def directional(f, args, grads, gen, eps=1e-6):
    """sum <grad, direction> against the central difference of f along random directions."""
    for name, g in grads.items():
        v = args[name]
        d = torch.randn(v.shape, generator=gen, dtype=torch.float64)
        hi, lo = (f(dict(args, **{name: v + s * eps * d})) for s in (1, -1))
        num, ana = (hi - lo) / (2 * eps), float((g * d).sum())
        # truncation eps^2 and cancellation 2^-53 / eps, relative to the objective's size
        assert abs(num - ana) <= 1e-6 * (abs(ana) + abs(hi) + 1), (name, num, ana)


@pytest.mark.parametrize("B,T,H,G,rows", [(1, 1, 1, 1, None), (2, 7, 4, 2, None), (3, 9, 2, 1, [9, 0, 4]),
                                          (2, 70, 2, 2, [70, 66])])
def test_linattn_gradients_against_differences(B, T, H, G, rows):
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)   # noqa: E731
    a = dict(q=n(B, T, G, 3), k=n(B, T, G, 3), v=n(B, T, H, 2), g=-n(B, T, H).abs(), s0=n(B, H, 2, 3))
    dy, dsT = n(B, T, H, 2), n(B, H, 2, 3)

    def f(x):
        o = _linattn.reference(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], lengths=rows, scale=0.7)
        return float((o["y"][0] * dy).sum() + (o["sT"][0] * dsT).sum())

    g = _linattn.reference(a["q"], a["k"], a["v"], a["g"], s0=a["s0"], lengths=rows, scale=0.7, dy=dy, dsT=dsT)
    directional(f, a, dict(q=g["dq"][0], k=g["dk"][0], v=g["dv"][0], g=g["dg"][0], s0=g["ds0"][0]), gen)


def test_linattn_closed_form():
    """Without decay: the running sum of v_s (k_s . q_t)."""
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, 6, 1, 4, generator=gen, dtype=torch.float64) for _ in range(3))
    y = _linattn.reference(q, k, v, torch.zeros(1, 6, 1, dtype=torch.float64), scale=2.0)["y"][0]
    w = torch.tril(torch.einsum("btgn,bsgn->ts", q, k))
    assert torch.allclose(y[0, :, 0], 2 * w @ v[0, :, 0])


def test_linattn_packed_rows_are_padded_rows():
    gen = torch.Generator().manual_seed(3)
    n = [3, 0, 5]
    x = [torch.randn(3, 5, 2, 4, generator=gen, dtype=torch.float64) for _ in range(3)]
    g = -torch.rand(3, 5, 2, generator=gen, dtype=torch.float64)
    pad = _linattn.reference(*x, g, lengths=n)
    flat = lambda t: torch.cat([t[b, :n[b]] for b in range(3)])   # noqa: E731
    packed = _linattn.reference(*[flat(t) for t in x], flat(g), starts=[0, 3, 3, 8])
    assert torch.allclose(packed["y"][0], flat(pad["y"][0])) and torch.allclose(packed["sT"][0], pad["sT"][0])


@pytest.mark.parametrize("how", [dict(), dict(center=False), dict(silu=True), dict(gate_first=True),
                                 dict(center=False, silu=True, gate_first=True)])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients_against_differences(how, gate):
    if how.get("gate_first") and not gate:
        return
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)   # noqa: E731
    a = dict(x=n(3, 12), gamma=n(12), beta=n(12))
    if gate:
        a["z"] = n(3, 12)
    dy = n(3, 12)

    def f(x):
        return float((_gnorm.norm(groups=2, **x, **how)["y"][0] * dy).sum())

    g = _gnorm.norm(groups=2, dy=dy, **a, **how)
    names = dict(x="dx", gamma="dgamma", beta="dbeta", z="dz")
    directional(f, a, {k: g[names[k]][0] for k in a}, gen)


# ---- linear attention at the C ABI ------------------------------------------------------------


LA_OK = dict(B=1, T=8, H=4, G=2, N=64, P=64, dtype=wk.WKV7_BF16, fixed_decay=0, packed=0, tokens=0, scale=1.0)
FORWARD, BACKWARD, STEP = 0, 1, 2
ALL = (FORWARD, BACKWARD, STEP)


def linattn(L, which, desc=None, **over):
    """Statuses of the named entry points, with valid arguments but for `desc` and `over`."""
    d = None if desc is None else C(wk.LinattnDesc(**dict(LA_OK, **desc)))
    a = dict(rows=None, q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, y=FAKE, sT=None, ckpt=FAKE, dy=FAKE, dsT=None,
             dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, ds0=None, ws=FAKE, wsb=1 << 40, slots=None, nslots=1 << 20,
             state=FAKE)
    a.update(over)
    n = lambda *names: [a[x] for x in names]   # noqa: E731
    calls = (lambda: L.wkv7_linattn_forward(d, *n("rows", "q", "k", "v", "g", "s0", "y", "sT", "ckpt", "ws", "wsb"), None),
             lambda: L.wkv7_linattn_backward(d, *n("rows", "q", "k", "v", "g", "dy", "dsT", "ckpt", "dq", "dk", "dv",
                                                   "dg", "ds0", "ws", "wsb"), None),
             lambda: L.wkv7_linattn_step(d, *n("slots", "nslots", "q", "k", "v", "g", "state", "y"), None))
    return {calls[i]() for i in which}


@pytest.mark.parametrize("desc", [dict(B=-1), dict(T=-1), dict(H=-4), dict(G=0), dict(G=3), dict(tokens=-1),
                                  dict(packed=2), dict(fixed_decay=2), dict(scale=float("nan")),
                                  dict(scale=float("inf"))], ids=str)
def test_linattn_invalid(L, desc):
    assert linattn(L, ALL, desc) == {wk.WKV7_ERR_INVALID_ARG}
    d = wk.LinattnDesc(**dict(LA_OK, **desc))
    assert L.wkv7_linattn_ckpt_bytes(C(d)) == 0 and L.wkv7_linattn_backward_workspace_bytes(C(d)) == 0


@pytest.mark.parametrize("desc", [dict(N=16), dict(N=65), dict(P=0), dict(P=256), dict(dtype=2), dict(T=2 ** 31 - 1),
                                  dict(H=1 << 17, G=1 << 17), dict(B=1 << 20, H=4), dict(tokens=2 ** 31 - 1),
                                  dict(B=1 << 19, H=4, T=1 << 20)], ids=str)
def test_linattn_unsupported(L, desc):
    assert linattn(L, ALL, desc) == {wk.WKV7_ERR_UNSUPPORTED}
    assert L.wkv7_linattn_forward_workspace_bytes(C(wk.LinattnDesc(**dict(LA_OK, **desc)))) == 0


def test_linattn_pointers(L):
    bad = {wk.WKV7_ERR_INVALID_ARG}
    assert linattn(L, ALL) == bad and linattn(L, ALL, q=None) == bad
    for name in ("q", "k", "v", "g"):
        for value in (None, FAKE + 4):
            assert linattn(L, ALL, {}, **{name: value}) == bad, name
    for name in ("dy", "ckpt", "dq", "dk", "dv", "dg"):
        for value in (None, FAKE + 8):
            assert linattn(L, (BACKWARD,), {}, **{name: value}) == bad, name
    assert linattn(L, (FORWARD, STEP), {}, y=None) == bad and linattn(L, (STEP,), {}, state=None) == bad
    for name in ("s0", "sT", "ckpt", "ws"):
        assert linattn(L, (FORWARD,), {}, **{name: FAKE + 4}) == bad, name
    for name in ("dsT", "ds0", "ws"):
        assert linattn(L, (BACKWARD,), {}, **{name: FAKE + 4}) == bad, name
    assert linattn(L, (FORWARD, BACKWARD), {}, rows=FAKE + 2) == bad
    assert linattn(L, (FORWARD, BACKWARD), dict(packed=1, tokens=5)) == bad            # no starts
    assert linattn(L, (STEP,), dict(packed=1, tokens=5), rows=FAKE) == bad
    assert linattn(L, (BACKWARD,), dict(fixed_decay=1)) == bad                         # no dg then
    assert linattn(L, (STEP,), {}, nslots=0) == bad and linattn(L, (STEP,), {}, slots=FAKE, nslots=-1) == bad
    assert linattn(L, (STEP,), {}, slots=FAKE + 2) == bad
    assert linattn(L, (STEP,), dict(B=65537), slots=FAKE, nslots=8) == {wk.WKV7_ERR_UNSUPPORTED}


def test_linattn_workspace_and_sizes(L):
    few = dict(B=1, T=16384, H=12, G=12)
    d = wk.LinattnDesc(**dict(LA_OK, **few))
    need = L.wkv7_linattn_forward_workspace_bytes(C(d))
    assert need > 0 and need % (12 * 64 * 64 * 4 + 96) == 0   # segments' states and decays
    assert linattn(L, (FORWARD,), few, wsb=need - 1) == {wk.WKV7_ERR_WORKSPACE}
    assert linattn(L, (FORWARD,), few, ws=None) == {wk.WKV7_ERR_WORKSPACE}
    back = L.wkv7_linattn_backward_workspace_bytes(C(d))
    assert linattn(L, (BACKWARD,), few, wsb=back - 1) == {wk.WKV7_ERR_WORKSPACE}
    many = wk.LinattnDesc(**dict(LA_OK, B=8, T=4096, H=32, G=32))
    assert L.wkv7_linattn_forward_workspace_bytes(C(many)) == 0
    assert L.wkv7_linattn_ckpt_bytes(C(many)) == 8 * 64 * 32 * 64 * 64 * 2
    # the gradient of the state behind every tile, and four parts of a product for each tile and head
    back = L.wkv7_linattn_ckpt_bytes(C(many))
    assert L.wkv7_linattn_backward_workspace_bytes(C(many)) == back + 8 * 64 * 32 * 16
    many.fixed_decay = 1
    assert L.wkv7_linattn_backward_workspace_bytes(C(many)) == back
    packed = wk.LinattnDesc(**dict(LA_OK, B=3, T=100, packed=1, tokens=130, N=32, dtype=wk.WKV7_F32))
    assert L.wkv7_linattn_ckpt_bytes(C(packed)) == (130 // 64 + 3) * 4 * 64 * 32 * 4
    assert wk.linattn_ckpt_shape(3, 100, 4, 64, 32, 130) == (5, 4, 64, 32)
    assert wk.linattn_ckpt_shape(3, 100, 4, 64, 32) == (6, 4, 64, 32)
    assert L.wkv7_linattn_ckpt_bytes(None) == 0 and L.wkv7_linattn_backward_workspace_bytes(None) == 0


def test_linattn_nothing_to_do(L):
    for empty in (dict(B=0), dict(H=0, G=1)):
        assert linattn(L, ALL, empty, q=None, k=None, v=None, g=None, y=None, dy=None, state=None) == {wk.WKV7_OK}
    for none in (dict(T=0), dict(packed=1, tokens=0)):
        assert linattn(L, (FORWARD, BACKWARD), none, rows=FAKE, q=None, k=None, v=None, g=None, y=None, dy=None,
                       ckpt=None, dq=None, dk=None, dv=None, dg=None) == {wk.WKV7_OK}


# ---- the group norm ---------------------------------------------------------------------------


GN_OK = dict(rows=4, D=64, G=2, dtype=wk.WKV7_F32, center=1, silu=0, gate=0, eps=1e-5)


def gnorm(L, which, desc=None, **over):
    d = None if desc is None else C(wk.GnormDesc(**dict(GN_OK, **desc)))
    a = dict(gamma=FAKE, beta=FAKE, x=FAKE, z=None, y=FAKE, dy=FAKE, dx=FAKE, dz=None, dgamma=FAKE, dbeta=FAKE,
             ws=FAKE, wsb=1 << 30)
    a.update(over)
    n = lambda *names: [a[x] for x in names]   # noqa: E731
    calls = (lambda: L.wkv7_gnorm_forward(d, *n("gamma", "beta", "x", "z", "y"), None),
             lambda: L.wkv7_gnorm_backward(d, *n("gamma", "beta", "x", "z", "dy", "dx", "dz", "dgamma", "dbeta", "ws",
                                                 "wsb"), None))
    return {calls[i]() for i in which}


def test_gnorm_refusals(L):
    both, bad, no = (FORWARD, BACKWARD), {wk.WKV7_ERR_INVALID_ARG}, {wk.WKV7_ERR_UNSUPPORTED}
    assert gnorm(L, both) == bad
    for desc in (dict(rows=-1), dict(D=-1), dict(G=0), dict(G=3), dict(center=2), dict(silu=-1), dict(gate=3),
                 dict(gate=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert gnorm(L, both, desc, z=FAKE, dz=FAKE) == bad, desc
    for desc in (dict(dtype=2), dict(D=1 << 23), dict(rows=1 << 40)):
        assert gnorm(L, both, desc) == no, desc
        assert L.wkv7_gnorm_backward_workspace_bytes(C(wk.GnormDesc(**dict(GN_OK, **desc)))) == 0
    assert gnorm(L, both, {}, x=None) == bad and gnorm(L, both, {}, x=FAKE + 4) == bad
    assert gnorm(L, both, {}, gamma=FAKE + 4) == bad and gnorm(L, both, {}, z=FAKE) == bad   # a gate not asked for
    assert gnorm(L, both, dict(gate=1)) == bad                                               # and one not given
    assert gnorm(L, (FORWARD,), {}, y=None) == bad
    for name in ("dy", "dx", "dgamma", "dbeta"):
        assert gnorm(L, (BACKWARD,), {}, **{name: None}) == bad, name
    assert gnorm(L, (BACKWARD,), {}, gamma=None) == bad and gnorm(L, (BACKWARD,), {}, dz=FAKE) == bad
    assert gnorm(L, (BACKWARD,), {}, ws=None) == {wk.WKV7_ERR_WORKSPACE} == gnorm(L, (BACKWARD,), {}, wsb=8)
    none = dict(x=None, y=None, dy=None, dx=None)
    assert gnorm(L, both, dict(D=0), **none) == {wk.WKV7_OK} == gnorm(L, (FORWARD,), dict(rows=0), **none)
    assert gnorm(L, (BACKWARD,), dict(rows=0), gamma=None, beta=None, dgamma=None, dbeta=None, **none) == {wk.WKV7_OK}


# ---- slots ------------------------------------------------------------------------------------


def test_slots_refusals(L):
    def copy(planes=2, slots=8, row=64, n=3, src=FAKE, dst=FAKE, source=FAKE, from_slots=8, pool=FAKE):
        return L.wkv7_slots_copy(planes, slots, row, n, src, dst, source, from_slots, pool, None)

    def compact(planes=2, slots=8, row=64, keep=FAKE, moved=FAKE, count=FAKE, clear=0, pool=FAKE, ws=FAKE, wsb=1 << 20):
        return L.wkv7_slots_compact(planes, slots, row, keep, moved, count, clear, pool, ws, wsb, None)

    bad, no = wk.WKV7_ERR_INVALID_ARG, wk.WKV7_ERR_UNSUPPORTED
    for f in (copy, compact):
        for over in (dict(planes=-1), dict(slots=-1), dict(row=-1), dict(pool=None), dict(pool=FAKE + 8)):
            assert f(**over) == bad, over
        for over in (dict(slots=(1 << 22) + 1), dict(planes=(1 << 20) + 1), dict(row=(1 << 40) + 1)):
            assert f(**over) == no, over
    for over in (dict(n=-1), dict(from_slots=-1), dict(src=None), dict(dst=None), dict(src=FAKE + 2), dict(source=None),
                 dict(source=FAKE + 8), dict(from_slots=7)):   # the pool itself has as many slots as it has
        assert copy(**over) == bad, over
    assert copy(n=65537, row=16) == no == copy(n=65536, row=1 << 24) and copy(source=FAKE * 4, from_slots=(1 << 22) + 1) == no
    for over in (dict(keep=None), dict(moved=None), dict(count=None), dict(moved=FAKE + 2), dict(count=FAKE + 2),
                 dict(clear=2), dict(ws=FAKE + 2)):
        assert compact(**over) == bad, over
    assert compact(slots=1 << 20, row=1 << 24) == no
    need = L.wkv7_slots_compact_workspace_bytes(8)
    assert need == 68 and compact(ws=None) == wk.WKV7_ERR_WORKSPACE == compact(wsb=need - 1)
    assert L.wkv7_slots_compact_workspace_bytes(-1) == 0
    for over in (dict(n=0), dict(planes=0), dict(row=0), dict(slots=0, from_slots=0, source=None)):
        assert copy(**dict(over, src=None, dst=None)) == wk.WKV7_OK, over


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 8, 2, 64)
    with pytest.raises(ValueError):
        wk.linattn_forward(x, x, x, torch.zeros(1, 8, 2))
    with pytest.raises(ValueError):
        wk.gnorm_forward(x, 2)
    with pytest.raises(ValueError):
        wk.slots_copy(x, torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        wk.gnorm_forward(x.half(), 2)
