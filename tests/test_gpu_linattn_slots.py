"""Single tokens of linear attention on caches at the ends of their sizes."""

import pytest

from tests.test_gpu_linattn import make, wk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_a_cache_without_slots(wk):
    """No row's slot exists, so every y is 0."""
    import torch
    ins, _, _, _, kw = make(71, 5, 1, 4, 2, 32, 64, "bf16")
    ins = [x[:, 0].clone() for x in ins]
    cache = torch.empty(0, 4, 64, 32, device="cuda")
    for slots in ([0, 1, 2, 3, 4], [-1, 0, 2 ** 31 - 1, 0, 0]):
        out = torch.full((5, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        at = torch.tensor(slots, dtype=torch.int32, device="cuda")
        y = wk.linattn_step(*ins, cache, slots=at, scale=kw["scale"], out=out)
        assert y is out and bool((y == 0).all())
