"""Linear attention at its edges: values that are not finite, decays of -infinity, rows that
lie anywhere in a packed tensor, slots named twice, long tensors, streams, graphs, refusals."""

import pytest

from tests import _linattn as ref
from tests.test_gpu_linattn import check, make, rows_kw, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def same(a, b):
    import torch
    return torch.equal(torch.nan_to_num(a.float(), nan=1e30), torch.nan_to_num(b.float(), nan=1e30))


def finite_as(got, want, what):
    """Finite where the definition is."""
    import torch
    value = want[0]
    assert torch.equal(torch.isfinite(got.double().cpu()), torch.isfinite(value)), what


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("at", [0, 37, 64, 100])
def test_values_that_are_not_finite(wk, name, bad, at, dtype):
    """They reach what the recurrence takes them to, and nothing else: not the tokens before,
    though those share a tile's products, nor the other heads and rows."""
    import torch
    B, T, H, G, N, P = 2, 130, 4, 2, 32, 64
    ins, s0, dy, dsT, kw = make(21, B, T, H, G, N, P, dtype)
    clean_y, clean_s, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    clean = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    dict(q=ins[0], k=ins[1], v=ins[2], dy=dy)[name][1, at, 1, 5] = bad
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    grads = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    torch.cuda.synchronize()
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    finite_as(y, want["y"], "y")
    finite_as(sT, want["sT"], "sT")
    for n in ("dq", "dk", "dv", "ds0"):
        finite_as(getattr(grads, n), want[n], n)
    # dg: also the other tokens of the tile, by the definition's leave
    fine = torch.isfinite(want["dg"][0])
    for t in range(0, T, 64):
        fine[:, t:t + 64] &= fine[:, t:t + 64].all(1, keepdim=True)
    assert torch.isfinite(grads.dg.cpu()[fine]).all()
    # Tokens before it read out what they did (its tile's sums run in another order).
    half = ref.HALF[ins[2].dtype]
    was, got = clean_y[1, :at].float(), y[1, :at].float()
    assert bool(((got - was).abs() <= 4 * half * (was.abs() + clean_y.float().abs().max())).all())
    assert same(y[0], clean_y[0]) and same(sT[0], clean_s[0]) and same(grads.ds0[0], clean.ds0[0])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_states_that_are_not_finite(wk, dtype):
    import torch
    ins, s0, dy, dsT, kw = make(22, 3, 70, 2, 2, 64, 32, dtype, rows="padded", lengths=[70, 65, 3])
    s0[1, 0, 3, 4] = float("inf")
    dsT[2, 1, 0, 7] = float("nan")
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    grads = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    for n, got in (("y", y), ("sT", sT), ("dq", grads.dq), ("dk", grads.dk), ("dv", grads.dv), ("ds0", grads.ds0)):
        finite_as(got, want[n], n)
    for x in (y, grads.dq, grads.dk, grads.dv, grads.dg):
        assert bool((x[1, 65:] == 0).all()) and bool((x[2, 3:] == 0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_padding_is_not_used(wk, dtype):
    import torch
    ins, s0, dy, dsT, kw = make(23, 3, 150, 4, 2, 64, 64, dtype, rows="padded", lengths=[150, 0, 66])
    want = check(wk, ins, s0, dy, dsT, kw, 150)
    for x in (*ins, dy):
        x[1, :] = float("nan")
        x[2, 66:] = float("inf")
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    grads = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    assert torch.equal(y, want[0]) and torch.equal(sT, want[1])
    for a, b in zip(grads, want[3]):
        assert torch.equal(a, b)
    assert torch.equal(sT[1], s0[1]) and torch.equal(grads.ds0[1], dsT[1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("low", [float("-inf"), -3e38, -1e4, -60.0])
def test_strong_decays(wk, dtype, low):
    """What is forgotten entirely, at a tile's edges and inside, beside ordinary decays."""
    ins, s0, dy, dsT, kw = make(24, 2, 200, 2, 1, 64, 64, dtype)
    for t in (0, 5, 63, 64, 127, 199):
        ins[3][0, t] = low
    ins[3][1, 20:90] = low
    check(wk, ins, s0, dy, dsT, kw, 200)


def test_growth(wk):
    """Log decays above 0, as long as the sums stay in range."""
    ins, s0, dy, dsT, kw = make(25, 1, 100, 2, 2, 32, 32, "fp32")
    ins[3][:, ::7] = 0.3
    check(wk, ins, s0, dy, dsT, kw, 100)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_anywhere_in_a_packed_tensor(wk, dtype):
    """Rows that begin behind the first token, leave some behind the last, are longer than the
    call says (also with time segments and with no length at all): tokens of no row stay."""
    import torch
    total = 1700
    ins, _, dy, _, kw = make(26, 1, total, 2, 1, 64, 64, dtype)
    ins, dy = [x[0] for x in ins], dy[0]
    starts = [5, 5, 70, 1500, 1650]
    B = len(starts) - 1
    dev = torch.tensor(starts, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(1)
    s0, dsT = (torch.randn(B, 2, 64, 64, generator=gen).cuda() for _ in range(2))
    want = ref.reference(*ins, s0=s0, starts=starts, scale=kw["scale"], dy=dy, dsT=dsT)
    K, t = ref.roundings(1500, 64, 64), ins[2].dtype
    inner = 1 if t == torch.bfloat16 else 0
    for max_len in (1430, 2000, 64, 1, 0):
        out = torch.full_like(ins[2], 7.0)
        y, sT, ck = wk.linattn_forward(*ins, s0=s0, starts=dev, max_len=max_len, scale=kw["scale"], want_ckpt=True, out=out)
        g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, starts=dev, max_len=max_len, scale=kw["scale"])
        torch.cuda.synchronize()
        assert bool((y[:5] == 7).all()) and bool((y[1650:] == 7).all())
        ref.assert_within(y, want["y"], t, K, "y", inner)
        ref.assert_within(sT, want["sT"], torch.float32, K, "sT")
        for n in ("dq", "dk", "dv"):
            ref.assert_within(getattr(g, n), want[n], t, 2 * K, n, inner)
        ref.assert_within(g.ds0, want["ds0"], torch.float32, 2 * K, "ds0")
        ref.assert_within(g.dg, want["dg"], t, 4 * K, "dg", 2 * inner)


def test_starts_out_of_range_touch_nothing_else(wk):
    import torch
    ins, _, _, _, kw = make(27, 1, 100, 2, 2, 64, 64, "bf16")
    ins = [x[0] for x in ins]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    y0, s, _ = wk.linattn_forward(*ins, starts=dev([0, 100]), max_len=100)
    y1, s1, _ = wk.linattn_forward(*ins, starts=dev([-7, 100000]), max_len=100)
    assert torch.equal(y0, y1) and torch.equal(s, s1)
    out = torch.full_like(ins[2], 3.0)
    y2, s2, _ = wk.linattn_forward(*ins, starts=dev([90, 20]), max_len=100, out=out)   # falling: no tokens
    assert bool((y2 == 3).all()) and bool((s2 == 0).all())


def test_empty(wk):
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)   # noqa: E731
    s0 = torch.randn(2, 4, 64, 32, device="cuda")
    y, sT, ck = wk.linattn_forward(z(2, 0, 2, 32), z(2, 0, 2, 32), z(2, 0, 4, 64), z(2, 0, 4), s0=s0, want_ckpt=True)
    assert y.shape == (2, 0, 4, 64) and torch.equal(sT, s0) and ck.shape[0] == 0
    g = wk.linattn_backward(z(2, 0, 2, 32), z(2, 0, 2, 32), z(2, 0, 4, 64), z(2, 0, 4), y, ck, dsT=s0)
    assert torch.equal(g.ds0, s0)
    y, sT, _ = wk.linattn_forward(z(0, 5, 2, 32), z(0, 5, 2, 32), z(0, 5, 4, 64), z(0, 5, 4))
    assert y.shape[0] == 0 and sT.shape[0] == 0
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, sT, _ = wk.linattn_forward(z(7, 2, 32), z(7, 2, 32), z(7, 4, 64), z(7, 4), starts=one, max_len=7)   # no rows
    assert sT.shape[0] == 0
    assert wk.linattn_step(z(0, 2, 32), z(0, 2, 32), z(0, 4, 64), z(0, 4), s0[:0].contiguous()).shape == (0, 4, 64)


def test_slots_named_twice_or_not_there(wk):
    import torch
    B, H, N, P = 70, 2, 64, 64
    ins, _, _, _, kw = make(28, B, 1, H, H, N, P, "bf16")
    ins = [x[:, 0].contiguous() for x in ins]
    pool = torch.randn(40, H, P, N, generator=torch.Generator().manual_seed(4)).cuda()
    at = torch.arange(B, dtype=torch.int32) % 30
    at[3], at[4], at[5] = -1, 40, 2 ** 31 - 1
    at[0] = 31
    seen, live = set(), []
    for b, s in enumerate(at.tolist()):
        live.append(0 <= s < 40 and s not in seen)
        seen.add(s)
    before = pool.clone()
    y = wk.linattn_step(*ins, pool, slots=at.cuda(), scale=kw["scale"])
    keep = torch.tensor(live)
    sub = [x[keep.cuda()] for x in ins]
    states = before[at[keep].long().cuda()].contiguous()
    y1 = wk.linattn_step(*sub, states, scale=kw["scale"])
    assert torch.equal(y[keep.cuda()], y1) and bool((y[~keep.cuda()] == 0).all())
    want = before.clone()
    want[at[keep].long().cuda()] = states
    assert torch.equal(pool, want)


@pytest.mark.parametrize("case", [(2, 300, 4, 4, 64, 64, "full", None), (3, 500, 8, 1, 64, 32, "padded", [500, 40, 0]),
                                  (2, 900, 2, 1, 128, 128, "packed", [900, 129])], ids=str)
def test_calls_agree_bit_for_bit(wk, case):
    """Also with a workspace of the caller's that holds anything, and on another stream."""
    import torch
    B, T, H, G, N, P, rows, lengths = case
    ins, s0, dy, dsT, kw = make(29, B, T, H, G, N, P, "bf16", rows=rows, lengths=lengths)
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.full((1 << 26,), 0xff, dtype=torch.uint8, device="cuda")
        y2, sT2, _ = wk.linattn_forward(*ins, s0=s0, workspace=ws, **kw)
        g2 = wk.linattn_backward(*ins, dy, ck, dsT=dsT, workspace=ws, **kw)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(sT, sT2)
    for a, b in zip(g, g2):
        assert torch.equal(a, b)


def test_a_row_beyond_two_to_the_31_elements(wk):
    """Its last tokens are those of a row that starts from the state before them."""
    import torch
    T, H, N, P = (1 << 19) + 77, 64, 32, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)   # noqa: E731
    q, k, v, dy = rand(1, T, 1, N), rand(1, T, 1, N), rand(1, T, H, P), rand(1, T, H, P)
    g = -rand(1, T, H).abs()
    cut = T - 64 - T % 64
    y, sT, ck = wk.linattn_forward(q, k, v, g, want_ckpt=True)
    head = [x[:, :cut].contiguous() for x in (q, k, v, g)]
    tail = [x[:, cut:].contiguous() for x in (q, k, v, g)]
    _, mid, _ = wk.linattn_forward(*head)
    del head
    y2, sT2, ck2 = wk.linattn_forward(*tail, s0=mid, want_ckpt=True)
    # (a state that went through other time segments differs in its last bits)
    assert torch.allclose(sT, sT2, rtol=1e-4, atol=1e-4) and torch.allclose(y[:, cut:].float(), y2.float(), rtol=2 ** -7, atol=0.05)
    grads = wk.linattn_backward(q, k, v, g, dy, ck)
    g2 = wk.linattn_backward(*tail, dy[:, cut:].contiguous(), ck2)
    for n in ("dq", "dk", "dv"):
        a, b = getattr(grads, n)[:, cut:].float(), getattr(g2, n).float()
        assert torch.allclose(a, b, rtol=2 ** -6, atol=2 ** -6 * float(b.abs().max())), n


def test_captured_and_replayed(wk):
    """Forward, backward and a step in one graph, replayed with eager work in between."""
    import torch
    ins, s0, dy, dsT, kw = make(30, 2, 640, 2, 1, 64, 64, "bf16")
    one = [x[:, 0].clone() for x in ins]
    pool = torch.randn(6, 2, 64, 64, device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")

    def work(state):
        y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
        g = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
        return (y, sT, *g, wk.linattn_step(*one, state, slots=slots))

    state = pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(state)
    eager = pool.clone()
    state.copy_(pool)
    for i in range(4):
        ins[2].copy_(torch.randn_like(ins[2]))
        want = work(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
        assert torch.equal(state, eager)


def test_refusals(wk):
    import torch
    ins, s0, dy, dsT, kw = make(31, 2, 64, 2, 1, 64, 64, "bf16")
    q, k, v, g = ins
    bad = pytest.raises(ValueError)
    with bad:
        wk.linattn_forward(q, k, v.transpose(1, 2), g)
    with bad:
        wk.linattn_forward(q, k[:, :-1].contiguous(), v, g)
    with bad:
        wk.linattn_forward(q, k, v, g.float())
    with bad:
        wk.linattn_forward(q, k, v, g, s0=s0[:1])
    with bad:
        wk.linattn_forward(q, k, v, g, lengths=torch.ones(2, device="cuda"))
    with bad:
        wk.linattn_forward(q, k, v, g, max_len=3)
    with bad:
        wk.linattn_forward(q, k, v, g, out=v)
    with bad:
        wk.linattn_forward(q[0], k[0], v[0], g[0], starts=torch.tensor([0, 64], device="cuda", dtype=torch.int32))
    with bad:
        wk.linattn_backward(q, k, v, g, dy, torch.empty(1, 2, 64, 64, device="cuda", dtype=torch.bfloat16))
    with bad:
        wk.linattn_step(q[:, 0].clone(), k[:, 0].clone(), v[:, 0].clone(), g[:, 0].clone(), s0.bfloat16())
    with pytest.raises(wk.WKV7Error):
        wk.linattn_forward(q[..., :48].contiguous(), k[..., :48].contiguous(), v, g)
    with pytest.raises(wk.WKV7Error):
        wk.linattn_forward(q, k, v, g, scale=float("nan"))
    few = make(31, 1, 16384, 1, 1, 64, 64, "bf16")[0]
    with pytest.raises(wk.WKV7Error):
        wk.linattn_forward(*few, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
