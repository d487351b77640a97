"""Linear attention, the norm behind it and the slots in a row, as a layer's training step and
as a server's loop, against the definitions in 64 bits."""

import pytest

from tests import _gnorm, _linattn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rwkv_wkv7_delta_amd as wk
    wk.lib()
    return wk


def test_training_step(wk):
    """y = norm(attention(q, k, v, g)) gated by z, and every gradient, against the definitions
    in a row (fp32 tokens: what one passes on to the next is not rounded)."""
    import torch
    B, T, H, G, N, P = 2, 150, 4, 2, 32, 32
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()   # noqa: E731
    q, k, v, g = n(B, T, G, N), n(B, T, G, N), n(B, T, H, P), -n(B, T, H).abs()
    z, gamma, beta, dout = n(B, T, H * P), 1 + 0.1 * n(H * P), n(H * P), n(B, T, H * P)
    y, sT, ck = wk.linattn_forward(q, k, v, g, scale=N ** -0.5, want_ckpt=True)
    flat = y.view(B, T, H * P)
    out = wk.gnorm_forward(flat, H, gamma, beta, z=z)
    gn = wk.gnorm_backward(flat, dout, H, gamma, beta, z=z)
    la = wk.linattn_backward(q, k, v, g, gn.dx.view_as(y), ck, scale=N ** -0.5)
    torch.cuda.synchronize()
    r = _linattn.reference(q, k, v, g, scale=N ** -0.5)
    y64 = r["y"][0].view(B, T, H * P)
    m = _gnorm.norm(y64, H, gamma, beta, z, dy=dout)
    r = _linattn.reference(q, k, v, g, scale=N ** -0.5, dy=m["dx"][0].view(B, T, H, P))

    def near(got, want, what):
        # errors of one step pass through the next: 2-norms, 2^-24 times the terms of a row's sums
        # (T of them, both ways, through a norm of slope up to 10)
        d = (got.double().cpu() - want).norm() / want.norm()
        assert d <= 10 * 2 * T * 2.0 ** -24, (what, float(d))

    near(out, m["y"][0], "out")
    for name in ("dgamma", "dbeta", "dz"):
        near(getattr(gn, name), m[name][0], name)
    for name in ("dq", "dk", "dv", "dg", "ds0"):
        near(getattr(la, name), r[name][0], name)


def test_serving_loop(wk):
    """Prompts of different lengths one behind the other; their states go to slots of a cache of
    three layers, a sequence is forked, tokens are decoded, sequences end, the cache is compacted
    and decoding goes on: every read-out is the one of the whole sequence from the start."""
    import torch
    layers, S, H, N, P = 3, 8, 2, 64, 64
    n = [70, 1, 130]
    gen = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()   # noqa: E731
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    total = sum(n)
    cache = torch.zeros(layers, S, H, P, N, device="cuda")
    home = [5, 0, 3]                                     # slots of the three sequences
    history = {}                                         # (layer, slot): tokens so far, 64-bit
    starts = [0, 70, 71, 201]
    for layer in range(layers):
        q, k, v, g = rand(total, H, N), rand(total, H, N), rand(total, H, P), -rand(total, H).abs()
        _, sT, _ = wk.linattn_forward(q, k, v, g, starts=dev(starts), max_len=130)
        wk.slots_copy(cache[layer:layer + 1], dev([0, 1, 2]), dev(home), source=sT[None])
        for i, s in enumerate(home):
            history[layer, s] = [x[starts[i]:starts[i + 1]].double().cpu() for x in (q, k, v, g)]

    def decode(slots):
        for layer in range(layers):
            B = len(slots)
            q, k, v, g = rand(B, H, N), rand(B, H, N), rand(B, H, P), -rand(B, H).abs()
            y = wk.linattn_step(q, k, v, g, cache[layer], slots=dev(slots))
            for i, s in enumerate(slots):
                new = [x[i:i + 1].double().cpu() for x in (q, k, v, g)]
                history[layer, s] = [torch.cat(p) for p in zip(history[layer, s], new)]
                h = [x[None] for x in history[layer, s]]
                want = _linattn.reference(*h)["y"]
                _linattn.assert_within(y[i], tuple(x[0, -1] for x in want), torch.float32,
                                       _linattn.roundings(h[0].shape[1], N, P) + 8 * 4, f"layer {layer} slot {s}")

    decode(home)
    wk.slots_copy(cache, dev([3, 3]), dev([6, 7]))       # sequence 2 twice more
    for layer in range(layers):
        for s in (6, 7):
            history[layer, s] = history[layer, 3]
    decode([5, 0, 3, 6, 7])
    keep = torch.zeros(S, dtype=torch.bool, device="cuda")
    keep[[0, 5, 7]] = True                               # 3 and 6 have ended
    moved, count = wk.slots_compact(cache, keep, clear=True)
    assert int(count) == 3 and moved.tolist() == [0, -1, -1, -1, -1, 1, -1, 2]
    assert bool((cache[:, 3:] == 0).all())
    history = {(layer, int(moved[s])): h for (layer, s), h in history.items() if int(moved[s]) >= 0}
    decode([2, 0, 1])


def test_captured_and_replayed(wk):
    """A step, the norm with its gradients, copies and a compaction in one graph, replayed with
    other values, lists and eager work in between; first on a stream of their own."""
    import torch
    L, S, B, H, N, P = 2, 6, 3, 2, 32, 64
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()   # noqa: E731
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    q, k, v, g, z = rand(B, H, N), rand(B, H, N), rand(B, H, P), -rand(B, H).abs(), rand(B, H * P)
    gamma, beta, dy = rand(H * P), rand(H * P), rand(B, H * P)
    slots, src, dst = dev([4, 0, 2]), dev([4, -1]), dev([5, 1])
    keep = torch.tensor([True, False, True, False, True, True], device="cuda")

    def work(cache):
        o = [wk.linattn_step(q, k, v, g, cache[i], slots=slots).view(B, H * P) for i in range(L)]
        y = wk.gnorm_forward(o[1], H, gamma, beta, z=z, silu=True)
        grads = wk.gnorm_backward(o[1], dy, H, gamma, beta, z=z, silu=True)
        wk.slots_copy(cache, src, dst)
        return (*o, y, *grads, *wk.slots_compact(cache, keep, clear=True))

    pool = rand(L, S, H, P, N)
    cache, eager = pool.clone(), pool.clone()
    want = work(pool.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(cache)
    cache.copy_(pool)
    for i in range(4):
        v.copy_(rand(B, H, P))
        src[0] = i % 3
        keep[i] = not bool(keep[i])
        want = work(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
        assert torch.equal(cache, eager), i
