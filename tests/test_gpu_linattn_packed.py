"""Packed rows of linear attention: what a call's own outputs hold where no row has tokens, and
lengths that the call overstates."""

import pytest

from tests import _linattn as ref
from tests.test_gpu_linattn import make, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def stale(*like):
    """Leaves NaN in memory that the next tensors of these sizes are made of."""
    import torch
    held = [torch.full_like(x, float("nan")) for x in like for _ in range(3)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,G,N,P", [(2, 1, 64, 64), (3, 3, 32, 128), (1, 1, 32, 32), (7, 1, 128, 32)])
@pytest.mark.parametrize("starts", [[5, 5, 70, 200, 211], [0, 100], [37, 300], [0, 0], [300, 300], [150], [299, 300]])
def test_tokens_of_no_row_are_zero(wk, H, G, N, P, starts, dtype):
    """In every tensor that the binding makes; the tokens of rows are what a call gives whose
    tensors hold nothing else."""
    import torch
    total = 300
    ins, _, dy, _, kw = make(41, 1, total, H, G, N, P, dtype)
    ins, dy = [x[0] for x in ins], dy[0]
    dev = torch.tensor(starts, dtype=torch.int32, device="cuda")
    rows = dict(starts=dev, max_len=64, scale=kw["scale"])   # (one plan for both)
    stale(*ins)
    y, _, ck = wk.linattn_forward(*ins, want_ckpt=True, **rows)
    stale(*ins)
    g = wk.linattn_backward(*ins, dy, ck, **rows)
    a, b = starts[0], starts[-1]
    for x in (y, g.dq, g.dk, g.dv, g.dg):
        assert bool((x[:a] == 0).all()) and bool((x[b:] == 0).all())
    if b > a:
        cut = dict(rows, starts=dev - a)
        ins2, dy2 = [x[a:b].clone() for x in ins], dy[a:b].clone()   # (aligned)
        y2, _, ck2 = wk.linattn_forward(*ins2, want_ckpt=True, **cut)
        g2 = wk.linattn_backward(*ins2, dy2, ck2, **cut)
        for x, x2 in zip((y, g.dq, g.dk, g.dv, g.dg), (y2, g2.dq, g2.dk, g2.dv, g2.dg)):
            assert torch.equal(x[a:b], x2)


def test_constant_decays_and_a_captured_graph(wk):
    """No gradient of g; and starts that change between the replays of a graph."""
    import torch
    total = 260
    ins, _, dy, _, kw = make(42, 1, total, 4, 2, 64, 64, "bf16", fixed=True)
    ins, dy = [*[x[0] for x in ins[:3]], ins[3]], dy[0]
    dev = torch.tensor([10, 100, 200], dtype=torch.int32, device="cuda")

    def work():
        y, sT, ck = wk.linattn_forward(*ins, starts=dev, max_len=total, want_ckpt=True)
        g = wk.linattn_backward(*ins, dy, ck, starts=dev, max_len=total)
        assert g.dg is None
        return y, sT, g.dq, g.dk, g.dv, g.ds0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for starts in ([10, 100, 200], [0, 130, 260], [255, 255, 256], [0, 0, 0]):
        dev.copy_(torch.tensor(starts, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for a, b in zip(got, work()):
            assert torch.equal(a, b), starts
        for x in (got[0], *got[2:5]):
            assert bool((x[:starts[0]] == 0).all()) and bool((x[starts[-1]:] == 0).all())


@pytest.mark.parametrize("max_len", [1 << 17, (1 << 29) - 64])
def test_a_length_that_is_overstated(wk, max_len):
    """A model's whole context, or the longest there is: the same results as the rows' own length."""
    import torch
    ins, _, dy, _, kw = make(43, 1, 63, 512, 1, 32, 32, "bf16")
    ins, dy = [x[0] for x in ins], dy[0]
    starts = torch.tensor([0, 63], dtype=torch.int32, device="cuda")
    want = got = None
    for n in (63, max_len):
        rows = dict(starts=starts, max_len=n, scale=kw["scale"])
        y, sT, ck = wk.linattn_forward(*ins, want_ckpt=True, **rows)
        want, got = got, (y, sT, *wk.linattn_backward(*ins, dy, ck, **rows))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_starts_that_fall(wk):
    """What the rows' tokens get is not touched, also where starts fall, which they may not."""
    import torch
    ins, _, _, _, kw = make(44, 1, 128, 2, 2, 32, 32, "fp32")
    ins = [x[0] for x in ins]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    want, _, _ = wk.linattn_forward(*ins, starts=dev([0, 100]), max_len=100)
    y, _, _ = wk.linattn_forward(*ins, starts=dev([0, 100, 50]), max_len=100)
    assert torch.equal(y[:100], want[:100]) and bool((y[100:] == 0).all())
