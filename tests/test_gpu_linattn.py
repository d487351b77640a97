"""Linear attention with one decay per head on the GPU against its definition in 64 bits."""

import pytest

from tests import _linattn as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rwkv_wkv7_delta_amd as wk
    wk.lib()
    return wk


def make(seed, B, T, H, G, N, P, dtype, fixed=False, state=True, rows="full", lengths=None):
    """Inputs of one call, their rows, and the gradients that come in."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    normal = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    tokens, kw = (B, T), {}
    if rows == "packed":
        n = torch.tensor(lengths, dtype=torch.int32)
        kw["starts"] = torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)]).cuda()
        kw["max_len"] = T
        tokens = (int(n.sum()),)
    elif rows == "padded":
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32).cuda()
    rate = torch.exp(torch.empty(H).uniform_(-7, 0.5, generator=gen))
    g = -rate if fixed else (-rate * torch.exp(normal(*tokens, H))).to(t)
    ins = [x.cuda() for x in (normal(*tokens, G, N).to(t), normal(*tokens, G, N).to(t), normal(*tokens, H, P).to(t), g)]
    s0 = normal(B, H, P, N).cuda() if state else None
    dy = normal(*tokens, H, P).to(t).cuda()
    dsT = normal(B, H, P, N).cuda() if state else None
    return ins, s0, dy, dsT, dict(kw, scale=N ** -0.5)


def rows_kw(kw):
    return {k: v for k, v in kw.items() if k != "max_len"}


def check(wk, ins, s0, dy, dsT, kw, T, names=None):
    import torch
    t = ins[2].dtype
    inner = 1 if t == torch.bfloat16 else 0
    N, P = ins[0].shape[-1], ins[2].shape[-1]
    y, sT, ck = wk.linattn_forward(*ins, s0=s0, want_ckpt=True, **kw)
    grads = wk.linattn_backward(*ins, dy, ck, dsT=dsT, **kw)
    torch.cuda.synchronize()
    want = ref.reference(*ins, s0=s0, dy=dy, dsT=dsT, **rows_kw(kw))
    K = ref.roundings(T, N, P)
    ref.assert_within(y, want["y"], t, K, "y", inner)
    ref.assert_within(sT, want["sT"], torch.float32, K, "sT")
    for name in ("dq", "dk", "dv"):
        ref.assert_within(getattr(grads, name), want[name], t, 2 * K, name, inner)
    ref.assert_within(grads.ds0, want["ds0"], torch.float32, 2 * K, "ds0")
    if grads.dg is not None:
        # both the state and its gradient are rounded
        ref.assert_within(grads.dg, want["dg"], t, 4 * K, "dg", 2 * inner)
    return y, sT, ck, grads


CASES = [
    # B, T, H, G, N, P, fixed, state, rows, lengths
    (1, 1, 1, 1, 32, 32, False, False, "full", None),
    (2, 1, 2, 1, 64, 64, False, True, "full", None),
    (1, 2, 3, 3, 64, 32, True, True, "full", None),
    (2, 17, 2, 2, 32, 64, False, True, "full", None),
    (1, 63, 4, 2, 64, 64, False, True, "full", None),
    (1, 64, 2, 1, 128, 64, False, False, "full", None),
    (2, 65, 6, 2, 32, 128, True, True, "full", None),
    (1, 130, 3, 1, 128, 128, False, True, "full", None),
    (3, 200, 2, 2, 64, 128, False, True, "padded", [200, 0, 77]),
    (3, 70, 4, 1, 128, 32, False, True, "padded", [-5, 64, 99]),
    (4, 129, 2, 1, 64, 64, False, True, "packed", [1, 0, 129, 64]),
    (2, 300, 5, 5, 32, 32, True, False, "packed", [300, 11]),
    (1, 700, 2, 2, 64, 64, False, True, "full", None),     # time segments
    (2, 900, 2, 1, 128, 64, False, True, "padded", [900, 333]),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(wk, case, dtype):
    B, T, H, G, N, P, fixed, state, rows, lengths = case
    check(wk, *make(11, B, T, H, G, N, P, dtype, fixed, state, rows, lengths), T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,G,N,P", [(1, 1, 1, 32, 32), (3, 4, 2, 64, 64), (2, 3, 1, 128, 128), (5, 2, 2, 64, 32),
                                       (2, 2, 2, 32, 128)])
@pytest.mark.parametrize("slots", [False, True])
def test_single_tokens(wk, B, H, G, N, P, slots, dtype):
    import torch
    ins, _, _, _, kw = make(12, B, 6, H, G, N, P, dtype)
    n = B + 3 if slots else B
    pool = torch.randn(n, H, P, N, generator=torch.Generator().manual_seed(1)).cuda()
    at = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32).cuda() if slots else None
    before = pool.clone()
    s0 = pool[at.long()] if slots else pool.clone()
    ys = [wk.linattn_step(*[x[:, t].clone() for x in ins], pool, slots=at, scale=kw["scale"]) for t in range(6)]
    torch.cuda.synchronize()
    want = ref.reference(*ins, s0=s0, scale=kw["scale"])
    K = 6 * 8 + N
    ref.assert_within(torch.stack(ys, 1), want["y"], ins[2].dtype, K, "y")
    ref.assert_within(pool[at.long()] if slots else pool, want["sT"], torch.float32, K, "state")
    if slots:
        others = [i for i in range(n) if i not in at.tolist()]
        assert torch.equal(pool[others], before[others])
