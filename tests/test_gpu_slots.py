"""Copies between the slots of a cache, and its compaction, on the GPU against indexing."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rwkv_wkv7_delta_amd as wk
    wk.lib()
    return wk


def in_order(pool, src, dst, source=None):
    pool = pool.clone()
    read_slots = (pool if source is None else source).shape[1]
    for s, d in zip(src, dst):
        if not (0 <= d < pool.shape[1] and -1 <= s < read_slots):
            continue
        pool[:, d] = 0 if s < 0 else (pool if source is None else source)[:, s]
    return pool


LISTS = [
    ([0], [3]),
    ([2, 4, -1], [1, 3, 6]),                    # targets that do not touch
    ([0, 0, 0], [1, 2, 3]),                     # one source for several
    ([0, 1, 2, 3], [1, 2, 3, 4]),               # a chain: each reads what the one before wrote
    ([3, 2, 1, 0], [4, 3, 2, 1]),
    ([0, 1], [1, 0]),                           # one target is the other's source
    ([5, 6, -1], [2, 2, 2]),                    # one target, the last stays
    ([4, 4, 1], [4, 0, 4]),                     # onto itself
    ([-2, 7, 1, 99, 0], [1, -1, 7, 2, 8]),      # slots that do not exist
]


@pytest.mark.parametrize("row", [1, 3, 8, 34, 1024, 5000, 70001])
@pytest.mark.parametrize("kind", ["float32", "bfloat16", "uint8"])
def test_copy(wk, row, kind):
    import torch
    t = getattr(torch, kind)
    base = torch.randint(0, 200, (3, 7, row), generator=torch.Generator().manual_seed(row)).to(t)
    other = torch.randint(0, 200, (3, 9, row), generator=torch.Generator().manual_seed(row + 1)).to(t)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    for src, dst in LISTS:
        pool = base.cuda()
        wk.slots_copy(pool, dev(src), dev(dst))
        assert torch.equal(pool.cpu(), in_order(base, src, dst)), (src, dst)
        pool = base.cuda()
        wk.slots_copy(pool, dev(src), dev(dst), source=other.cuda())
        assert torch.equal(pool.cpu(), in_order(base, src, dst, other)), (src, dst)


def test_copy_many(wk):
    """More slots than the table of targets has bits, and lists longer than a workgroup."""
    import torch
    gen = torch.Generator().manual_seed(3)
    S = 20000
    base = torch.randn(2, S, 6, generator=gen)
    order = torch.randperm(S, generator=gen).to(torch.int32)
    for src, dst in ((order[:700], order[700:1400]), (order[:9000], order[9000:18000]), (order, order.flip(0))):
        pool = base.cuda()
        wk.slots_copy(pool, src.cuda(), dst.cuda())
        assert torch.equal(pool.cpu(), in_order(base, src.tolist(), dst.tolist()))


def compacted(pool, keep, clear):
    pool, S = pool.clone(), len(keep)
    count = sum(keep)
    moved = [i if k else -1 for i, k in enumerate(keep)]
    holes = [i for i in range(count) if not keep[i]]
    late = [i for i in range(count, S) if keep[i]]
    for h, i in zip(holes, late):
        pool[:, h] = pool[:, i]
        moved[i] = h
    if clear:
        pool[:, count:] = 0
    return pool, moved, count


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("S,row,share", [(1, 4, 1.0), (1, 4, 0.0), (2, 7, 0.5), (37, 130, 0.5), (64, 16, 0.0),
                                         (65, 16, 1.0), (300, 2000, 0.2), (1500, 33, 0.8), (3001, 8, 0.5)])
def test_compact(wk, S, row, share, clear):
    import torch
    gen = torch.Generator().manual_seed(S)
    base = torch.randn(2, S, row, generator=gen)
    keep = torch.rand(S, generator=gen) < share
    pool = base.cuda()
    moved, count = wk.slots_compact(pool, keep.cuda(), clear=clear)
    want, places, n = compacted(base, keep.tolist(), clear)
    assert int(count) == n and moved.tolist() == places
    assert torch.equal(pool.cpu(), want)
    again, _ = wk.slots_compact(pool, (torch.arange(S) < n).cuda(), clear=clear)
    assert torch.equal(pool.cpu(), want) and again.tolist() == list(range(n)) + [-1] * (S - n)


def test_empty(wk):
    import torch
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    pool = torch.ones(2, 3, 4, device="cuda")
    wk.slots_copy(pool, none, none)
    assert bool((pool == 1).all())
    moved, count = wk.slots_compact(torch.empty(2, 0, 4, device="cuda"), torch.empty(0, dtype=torch.bool, device="cuda"))
    assert moved.numel() == 0 and int(count) == 0
    moved, count = wk.slots_compact(torch.empty(0, 3, 4, device="cuda"), torch.tensor([False, True, True], device="cuda"))
    assert moved.tolist() == [-1, 1, 0] and int(count) == 2
