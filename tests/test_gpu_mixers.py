"""The convolution and the scan as a layer uses them: a run of both in a row for
training and for serving, captured graphs, streams, buffers and other calls that
the interface allows."""

import ctypes

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


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def layer_inputs(seed, B, T, D, N, W, dtype):
    import torch
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = lambda a, ty=torch.float32: torch.from_numpy(np.asarray(a)).to(ty).cuda()   # noqa: E731
    return dict(x=dev(rng.normal(size=(B, T, D)), t), weight=dev(rng.normal(size=(D, W)) / W ** 0.5),
                bias=dev(0.1 * rng.normal(size=D)), dt=dev(rng.uniform(-3, 0.5, size=(B, T, D)), t),
                A=dev(-np.exp(rng.uniform(-3, 0.9, size=(D, N)))), Bm=dev(rng.normal(size=(B, T, 1, N)), t),
                Cm=dev(rng.normal(size=(B, T, 1, N)), t), z=dev(rng.normal(size=(B, T, D)), t),
                dskip=dev(rng.normal(size=D)), dt_bias=dev(rng.uniform(-1, 0.5, size=D)),
                dy=dev(rng.normal(size=(B, T, D)), t))


def layer(wk, p, bits=0, s0=None, h0=None, lengths=None):
    """Convolution, then the scan of its outputs."""
    u, sT = wk.conv_forward(p["x"], p["weight"], p["bias"], s0=s0, lengths=lengths, silu=True, want_state=True)
    y, hT, ck = wk.ssm_forward(u, p["dt"], p["A"], p["Bm"], p["Cm"], z=p["z"], dskip=p["dskip"],
                               dt_bias=p["dt_bias"], h0=h0, lengths=lengths, ckpt_bits=bits)
    return u, sT, y, hT, ck


def layer_backward(wk, p, u, ck, bits, lengths=None):
    g = wk.ssm_backward(u, p["dt"], p["A"], p["Bm"], p["Cm"], p["dy"], ck, z=p["z"], dskip=p["dskip"],
                        dt_bias=p["dt_bias"], lengths=lengths, ckpt_bits=bits)
    return g, wk.conv_backward(p["x"], p["weight"], g.dx, p["bias"], lengths=lengths, silu=True)


def test_training_run(wk):
    """Forward and backward of the pair in fp32, every gradient against the definition's
    (the convolution's outputs and the scan's dx are rounded to fp32 in between)."""
    import torch
    B, T, D, N, W, lengths = 3, 45, 40, 16, 4, [45, 17, 0]
    p = layer_inputs(61, B, T, D, N, W, "fp32")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    u, sT, y, hT, ck = layer(wk, p, 32, lengths=n)
    g, (dx, dw, db, ds0) = layer_backward(wk, p, u, ck, 32, lengths=n)
    torch.cuda.synchronize()
    h = {k: host(v) for k, v in p.items()}
    s = ref.Scan(host(u), h["dt"], h["A"], h["Bm"], h["Cm"], z=h["z"], dskip=h["dskip"], dt_bias=h["dt_bias"],
                 lengths=lengths)
    ref.assert_within(y, s.outputs()["y"], torch.float32, s.roundings() + N, "y")
    want = s.grads(h["dy"])
    ref.assert_within(g.dx, want["dx"], torch.float32, 2 * s.roundings() + 64, "du")
    cw = ref.conv_grads(h["x"], h["weight"], host(g.dx), h["bias"], lengths=lengths, silu=True)
    ref.assert_within(dx, cw["dx"], torch.float32, 32, "dx")
    ref.assert_within(dw, cw["dweight"], torch.float32, 32 + B * T, "dweight")
    ref.assert_within(db, cw["dbias"], torch.float32, 32 + B * T, "dbias")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompt_then_tokens(wk, dtype):
    """A padded prompt batch and then single tokens from its states: each row's outputs
    are those of the whole row run at once."""
    import torch
    B, T, D, N, W, more = 3, 37, 72, 16, 4, 5
    p = layer_inputs(67, B, T + more, D, N, W, dtype)
    lengths = [37, 1, 20]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pre = {k: (v[:, :T].contiguous() if v.dim() >= 3 else v) for k, v in p.items()}
    _, state, y, h, _ = layer(wk, pre, lengths=n)
    rows = torch.arange(B, device="cuda")
    outs = []
    for k in range(more):   # row b's token lengths[b] + k
        at = lambda v: v[rows, n.long() + k].contiguous()   # noqa: E731
        u = wk.conv_step(at(p["x"]), p["weight"], state, p["bias"], silu=True)
        outs.append(wk.ssm_step(u, at(p["dt"]), p["A"], at(p["Bm"]), at(p["Cm"]), h, z=at(p["z"]),
                                dskip=p["dskip"], dt_bias=p["dt_bias"]))
    torch.cuda.synchronize()
    for b in range(B):
        end = lengths[b] + more
        one = {k: (v[b:b + 1, :end].clone() if v.dim() >= 3 else v) for k, v in p.items()}
        _, _, yb, hb, _ = layer(wk, one)
        s = ref.Scan(host(wk.conv_forward(one["x"], one["weight"], one["bias"], silu=True)[0]),
                     *(host(one[k]) for k in ("dt", "A", "Bm", "Cm")), z=host(one["z"]), dskip=host(one["dskip"]),
                     dt_bias=host(one["dt_bias"]))
        want, mag = s.outputs()["y"]
        K = s.roundings() + N
        ref.assert_within(yb, (want, mag), p["x"].dtype, K, "whole row")
        got = torch.cat([y[b:b + 1, :lengths[b]]] + [o[b:b + 1, None] for o in outs], 1)
        ref.assert_within(got, (want, mag), p["x"].dtype, K, "prompt, then tokens")
        ref.assert_within(h[b:b + 1], s.outputs()["hT"], torch.float32, s.roundings(), "state")


def test_token_shift_in_front_of_the_recurrence(wk):
    """The convolution at two taps feeds the WKV7 recurrence's inputs, as the token shift
    does: its output is a token tensor of forward()."""
    import torch
    from rwkv_wkv7_delta_amd import synth
    import oracle
    inp = synth.generate(2, 50, 3, 64, dtype="fp32", seed=3)
    d = [torch.from_numpy(x).cuda() for x in inp.tensors()]
    r = d[0]
    mu = torch.rand(192, device="cuda")
    rr, _ = wk.conv_forward(r.reshape(2, 50, 192), torch.stack([mu, 1 - mu], 1))
    y, _, _ = wk.forward(rr.view(2, 50, 3, 64), *d[1:])
    want, _ = oracle.forward(rr.double().cpu().numpy().reshape(2, 50, 3, 64), *inp.tensors()[1:])
    assert np.abs(host(y) - want).max() <= 1e-4 * np.abs(want).max()


@pytest.mark.parametrize("T,D", [(40, 48), (700, 24)])   # without and with time segments
def test_graph_capture(wk, T, D):
    """The run captured in a graph, replayed with new inputs between eager calls: every
    replay equals the eager result bit for bit."""
    import torch
    p = layer_inputs(71, 2, T, D, 16, 4, "bf16")

    def once():
        u, sT, y, hT, ck = layer(wk, p, 8)
        g, c = layer_backward(wk, p, u, ck, 8)
        return (u, sT, y, hT, ck) + tuple(g) + tuple(c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for seed in (1, 2, 3):
        new = layer_inputs(seed, 2, T, D, 16, 4, "bf16")
        for k in p:
            p[k].copy_(new[k])
        eager = [o.clone() for o in once()]
        for o in outs:
            o.view(torch.uint8).fill_(0xFF) if o.dtype != torch.uint8 else o.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs))


def test_step_captured_in_place(wk):
    import torch
    p = layer_inputs(73, 4, 8, 64, 16, 4, "bf16")
    one = {k: (v[:, 0].contiguous() if v.dim() >= 3 else v) for k, v in p.items()}
    state = torch.zeros(4, 3, 64, device="cuda", dtype=torch.bfloat16)
    h = torch.zeros(4, 64, 16, device="cuda")

    def once():
        u = wk.conv_step(one["x"], one["weight"], state, one["bias"], silu=True)
        return wk.ssm_step(u, one["dt"], one["A"], one["Bm"], one["Cm"], h, z=one["z"], dskip=one["dskip"],
                           dt_bias=one["dt_bias"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    graph_states, eager_states = [], []
    for keep in (graph_states, eager_states):
        state.zero_(), h.zero_()
        for t in range(4):
            for k in ("x", "dt", "Bm", "Cm", "z"):
                one[k].copy_(p[k][:, t])
            if keep is graph_states:
                graph.replay()
                y = out
            else:
                y = once()
            keep.append((y.clone(), state.clone(), h.clone()))
    for a, b in zip(graph_states, eager_states):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_two_calls_at_once(wk):
    """Two streams, each with its own workspace and different inputs."""
    import torch
    sets = [layer_inputs(79 + k, 2, 600, 40, 16, 4, "bf16") for k in range(2)]

    def once(p):
        u, sT, y, hT, ck = layer(wk, p, 32)
        g, c = layer_backward(wk, p, u, ck, 32)
        return (y, hT) + tuple(g) + tuple(c)

    alone = [once(p) for p in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = once(sets[k])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_callers_buffers(wk):
    """`out` and `workspace`: used, and refused where they do not fit or overlap an input;
    what lies behind the workspace's need is left alone."""
    import torch
    p = layer_inputs(83, 1, 300, 24, 16, 4, "bf16")
    args = (p["x"], p["dt"], p["A"], p["Bm"], p["Cm"])
    out = torch.full_like(p["x"], 7.0)
    d = wk.SsmDesc(1, 300, 24, 16, 1, wk.WKV7_BF16, 32)
    need = wk.lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d))
    assert need > 0
    ws = torch.full((need + 64,), 0xA5, device="cuda", dtype=torch.uint8)
    y, hT, ck = wk.ssm_forward(*args, out=out, workspace=ws, ckpt_bits=32)
    y2, _, _ = wk.ssm_forward(*args)
    assert y is out and torch.equal(y, y2) and bool((ws[need:] == 0xA5).all())
    with pytest.raises(wk.WKV7Error):
        wk.ssm_forward(*args, workspace=ws[:need // 2].clone())
    for bad in (p["x"], p["dt"]):
        with pytest.raises(ValueError):
            wk.ssm_forward(*args, out=bad)
    with pytest.raises(ValueError):
        wk.conv_forward(p["x"], p["weight"], out=p["x"])
    with pytest.raises(ValueError):
        wk.ssm_forward(*args, out=out[:, :-1])
    need = wk.lib().wkv7_ssm_backward_workspace_bytes(ctypes.byref(d))
    ws = torch.full((need + 64,), 0xA5, device="cuda", dtype=torch.uint8)
    g = wk.ssm_backward(*args, p["dy"], ck, workspace=ws)
    g2 = wk.ssm_backward(*args, p["dy"], ck)
    assert bool((ws[need:] == 0xA5).all()) and all(a is b is None or torch.equal(a, b) for a, b in zip(g, g2))
    c = wk.ConvDesc(1, 300, 24, 4, wk.WKV7_BF16, 0)
    need = wk.lib().wkv7_conv_backward_workspace_bytes(ctypes.byref(c))
    ws = torch.full((need + 64,), 0xA5, device="cuda", dtype=torch.uint8)
    a = wk.conv_backward(p["x"], p["weight"], p["dy"], workspace=ws)
    b = wk.conv_backward(p["x"], p["weight"], p["dy"])
    assert bool((ws[need:] == 0xA5).all()) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refusals(wk):
    import torch
    p = layer_inputs(89, 2, 20, 24, 16, 4, "bf16")
    args = [p["x"], p["dt"], p["A"], p["Bm"], p["Cm"]]
    wide = torch.zeros(2, 20, 48, device="cuda", dtype=torch.bfloat16)
    for k, bad in ((0, wide[..., :24]), (1, p["dt"].float()), (2, p["A"].bfloat16()), (2, p["A"][:, :12].contiguous()),
                   (3, p["Bm"][..., :8].contiguous()), (3, p["Bm"][:, :, 0]), (4, p["Cm"][:1].contiguous()),
                   (4, p["Cm"].cpu())):
        with pytest.raises((ValueError, wk.WKV7Error)):
            wk.ssm_forward(*(args[:k] + [bad] + args[k + 1:]))
    with pytest.raises(ValueError):
        wk.ssm_forward(*args, lengths=torch.zeros(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        wk.ssm_forward(*args, h0=torch.zeros(2, 24, 8, device="cuda"))
    with pytest.raises(wk.WKV7Error):
        wk.ssm_forward(*args, ckpt_bits=16)
    _, _, ck = wk.ssm_forward(*args, ckpt_bits=8)
    with pytest.raises(ValueError):
        wk.ssm_backward(*args, p["dy"], ck, ckpt_bits=32)
    with pytest.raises(ValueError):
        wk.ssm_backward(*args, p["dy"], ck[:-1].clone(), ckpt_bits=8)
    three = torch.zeros(2, 20, 3, 16, device="cuda", dtype=torch.bfloat16)
    groups = torch.zeros(2, 20, 5, 16, device="cuda", dtype=torch.bfloat16)   # 24 channels in 5 groups
    with pytest.raises(wk.WKV7Error):
        wk.ssm_forward(*args[:3], groups, groups)
    assert wk.ssm_forward(*args[:3], three, three)[0].shape == p["x"].shape
    with pytest.raises(wk.WKV7Error):
        wk.conv_forward(p["x"], torch.zeros(24, 5, device="cuda"))
    with pytest.raises(ValueError):
        wk.conv_forward(p["x"], p["weight"][:12].contiguous())
    # a row of an odd width starts between 16-byte boundaries
    odd = torch.zeros(2, 3, 7, device="cuda")
    with pytest.raises(wk.WKV7Error):
        wk.conv_forward(odd[1:], torch.zeros(7, 4, device="cuda"))


def test_long_rows_past_31_bits(wk):
    """A batch row of more than 2^31 bytes: token offsets and segment buffers.  Channels
    do not meet (but in B and C), so a few of them are checked on their own."""
    import torch
    T, D, N = 70000, 16384, 8
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(1, T, D, device="cuda", dtype=torch.bfloat16, generator=g)
    assert x.numel() * 2 > 1 << 31
    dt = torch.randn(1, T, D, device="cuda", dtype=torch.bfloat16, generator=g) * 0.5 - 3
    A = -torch.rand(D, N, device="cuda", generator=g) - 0.5
    Bm = torch.randn(1, T, 1, N, device="cuda", dtype=torch.bfloat16, generator=g)
    Cm = torch.randn(1, T, 1, N, device="cuda", dtype=torch.bfloat16, generator=g)
    y, hT, ck = wk.ssm_forward(x, dt, A, Bm, Cm, ckpt_bits=8)
    grads = wk.ssm_backward(x, dt, A, Bm, Cm, x, ck, ckpt_bits=8)
    w = torch.randn(D, 4, device="cuda", generator=g)
    c, _ = wk.conv_forward(x, w, silu=True)
    cg = wk.conv_backward(x, w, x, silu=True)
    torch.cuda.synchronize()
    some = torch.tensor([0, 1, 8191, 16382, 16383], device="cuda")
    pick = lambda v: v.index_select(-1, some).contiguous()   # noqa: E731
    xs, ds = pick(x), pick(dt)
    ys, hs, cks = wk.ssm_forward(xs, ds, A[some].contiguous(), Bm, Cm, ckpt_bits=8)
    gs = wk.ssm_backward(xs, ds, A[some].contiguous(), Bm, Cm, xs, cks, ckpt_bits=8)
    near = lambda a, b, tol: float((a.float() - b.float()).norm()) <= tol * float(b.float().norm())   # noqa: E731
    # other segments round differently by a few 2^-24, which moves a bf16 result by a step
    # (2^-8) only where it lies at a border, and an 8-bit state by one code (0.8 % of the
    # largest) likewise: far below 1e-3 in the norm
    assert near(pick(y), ys, 1e-3) and near(hT[:, some], hs, 1e-5)
    assert near(pick(grads.dx), gs.dx, 2e-3) and near(pick(grads.ddt), gs.ddt, 2e-3)
    assert near(grads.dA[some], gs.dA, 2e-3)
    cs, _ = wk.conv_forward(xs, w[some].contiguous(), silu=True)
    cgs = wk.conv_backward(xs, w[some].contiguous(), xs, silu=True)
    assert torch.equal(pick(c), cs) and near(pick(cg[0]), cgs[0], 1e-3) and near(cg[1][some], cgs[1], 1e-5)


def test_wide_segments_are_forced(wk):
    """Where a row's buffers would pass 2^31 bytes, the plan has time segments whatever the
    number of channels."""
    d = wk.SsmDesc(1, 70000, 16384, 8, 1, wk.WKV7_BF16, 8)
    assert wk.lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d)) > 0
    d = wk.SsmDesc(8, 4096, 16384, 8, 1, wk.WKV7_BF16, 8)
    assert wk.lib().wkv7_ssm_forward_workspace_bytes(ctypes.byref(d)) == 0


def test_no_negative_infinity_surprises(wk):
    """dt of -infinity is a rate of 0 (the token changes nothing); an infinity or a NaN in one
    batch row or channel stays there."""
    import torch
    p = layer_inputs(97, 2, 20, 24, 16, 4, "fp32")
    args = [p["x"], p["dt"].clone(), p["A"], p["Bm"], p["Cm"]]
    args[1][0, 3] = -float("inf")
    y, hT, _ = wk.ssm_forward(*args)
    s = ref.Scan(*(host(a) for a in args))
    ref.assert_within(y, s.outputs()["y"], torch.float32, s.roundings() + 16, "y")
    clean = wk.ssm_forward(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"])[0]
    x = p["x"].clone()
    x[0, 5, 7] = float("nan")
    y = wk.ssm_forward(x, *[p[k] for k in ("dt", "A", "Bm", "Cm")])[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 5:, 7] = True
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], clean[~bad])
