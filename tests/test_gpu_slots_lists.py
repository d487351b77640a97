"""Lists of copies between the slots of a large cache: every pair that touches another is found,
wherever its slots lie, and pairs that do not touch are copied at once."""

import pytest

from tests.test_gpu_slots import in_order, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def dev(x):
    import torch
    return torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("S", [31, 33, 8192, 8193, 40000, 1 << 18, (1 << 18) + 1, 700001])
def test_pairs_that_touch(wk, S):
    """At the first and last slots, either side of a multiple of what a table may hold, and far apart."""
    import torch
    gen = torch.Generator().manual_seed(S)
    base = torch.randn(1, S, 4, generator=gen)
    far = sorted({0, 1, 30, S // 2, S - 2, S - 1} | {x for x in (8191, 8192, (1 << 18) - 1, 1 << 18) if x < S})
    lists = [([5, 6], [far[-1], far[-1]]), ([far[-1], 7], [2, far[-1]]), ([7, far[-1]], [far[-1], 2]),
             ([far[0], far[-1], -1], [far[-1], 9, far[0]]), (far, far[::-1]), (far[::-1], far[1:] + far[:1]),
             ([3] * len(far), far), (far + [4], [8] * len(far) + [far[-1]])]
    for src, dst in lists:
        pool = base.cuda()
        wk.slots_copy(pool, dev(src), dev(dst))
        assert torch.equal(pool.cpu(), in_order(base, src, dst)), (src, dst)


def test_the_longest_list(wk):
    import torch
    gen = torch.Generator().manual_seed(2)
    S = 140000
    base = torch.randn(1, S, 4, generator=gen)
    order = torch.randperm(S, generator=gen)
    src, dst = order[:65536], order[65536:131072]
    want = base.clone()
    want[:, dst] = base[:, src]
    pool = base.cuda()
    wk.slots_copy(pool, dev(src), dev(dst))
    assert torch.equal(pool.cpu(), want)
    dst[-1] = src[0]                       # the last pair's target is the first one's source
    want = in_order(base, src.tolist(), dst.tolist())
    pool = base.cuda()
    wk.slots_copy(pool, dev(src), dev(dst))
    assert torch.equal(pool.cpu(), want)


def test_pairs_that_do_not_touch_are_copied_at_once(wk):
    """Whatever their distance: targets a power of two apart take no longer than neighbours do.
    (One row after the other takes twenty times as long.)"""
    import torch
    pool = torch.zeros(1, 60 * 4096, 256, device="cuda")

    def time(dst):
        src, dst = dev([5 + 2 * i for i in range(len(dst))]), dev(dst)
        best = float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                wk.slots_copy(pool, src, dst)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    # (sources up to 483)
    near = time([1000 + i for i in range(239)])
    assert time([1000 + 1024 * i for i in range(239)]) < 6 * near
