"""Measured cases of linear attention with one decay per head (prompts, gradients, single
tokens), the group norm with an activation over channels last, and the copies between the
slots of a cache of states.

Linear attention, per head h with a state of P value rows and N key columns; the H heads
share G sets of queries and keys:
    S_t = exp(g_t) S_{t-1} + v_t k_t^T,   y_t = scale S_t q_t
g is a log decay for every token and head, or one constant per head.  A training forward
keeps the state entering every 64 tokens in the tokens' type; the backward starts each
block of 64 tokens from it.

Group norm, per row of D channels in G groups of neighbouring channels:
    x' = x, or x z sigmoid(z)        n = (x' - mean) / sqrt(var + eps), or x' / sqrt(mean x'^2 + eps)
    o = gamma n + beta,   y = o, or o sigmoid(o),   and then perhaps times z sigmoid(z)

Slots: a cache [planes, slots, row]; a copy gives slot dst[i] of every plane what slot src[i]
holds (zeros where src[i] is -1), a compaction moves the kept slots to the front.
"""

import math

import torch

own = False

CHUNK = 64   # tokens per state checkpoint


def listed():
    return [
        # Prompts of a training or serving batch at the 1.5B width (32 heads of 64).
        dict(name="prompt_2048", op="la", B=8, T=4096, H=32, G=32, N=64, P=64, dtype="bf16", fixed=False,
             state=False, rows="full"),
        # One long prompt at the 0.19B width (12 heads of 64) that continues a state, with
        # constant decays: few heads, many tokens.
        dict(name="prompt_long", op="la", B=1, T=16384, H=12, G=12, N=64, P=64, dtype="bf16", fixed=True,
             state=True, rows="full"),
        # Prompts of different lengths one behind the other, in fp32, two heads to a key.
        dict(name="prompt_packed", op="la", B=6, T=1021, H=10, G=5, N=32, P=128, dtype="fp32", fixed=False,
             state=True, rows="packed"),
        # One training step (forward with checkpoints, then every gradient) at the 0.19B shape.
        dict(name="step_768", op="la_train", B=4, T=1024, H=12, G=12, N=64, P=64, dtype="bf16", fixed=False,
             state=True, rows="full"),
        # The gradients of a training step at the 2.9B shape (40 heads of 64).
        dict(name="grads_2560", op="la_bwd", B=8, T=4096, H=40, G=40, N=64, P=64, dtype="bf16", fixed=False,
             state=False, rows="full"),
        # Gradients of a padded batch whose 32 heads share one wide key.
        dict(name="grads_shared", op="la_bwd", B=3, T=1500, H=32, G=1, N=128, P=64, dtype="bf16", fixed=False,
             state=True, rows="padded"),
        # One token of one sequence: the smallest call, where latency counts.
        dict(name="token_1", op="la_step", B=1, S=0, H=12, G=12, N=64, P=64, dtype="bf16", fixed=False),
        # One token of every sequence that a serving batch decodes at the 2.9B width, their
        # states in slots of a larger cache.
        dict(name="token_256", op="la_step", B=256, S=320, H=40, G=40, N=64, P=64, dtype="bf16", fixed=False),
        # Per-head norm and gate behind the read-out, 2.9B training shape.
        dict(name="norm_2560", op="gn", rows=32768, D=2560, G=40, dtype="bf16", gate="after", silu=False,
             center=True, affine=True),
        # Gradients of a whole-row norm of gated values at the 1.5B width.
        dict(name="norm_grads", op="gn_bwd", rows=16384, D=2048, G=1, dtype="bf16", gate="before", silu=False,
             center=False, affine=True),
        # Forked sequences: 48 slots of twelve layers' states (12 heads of 64) copied.
        dict(name="fork", op="copy", planes=12, S=128, n=48, row=12 * 64 * 64, dtype="fp32"),
        # The slots of the sequences that go on, moved to the front; an odd row of 16-bit values.
        dict(name="compact", op="compact", planes=7, S=200, row=30001, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["la", "la", "la_train", "la_bwd", "la_bwd", "la_step", "gn", "gn_bwd", "copy", "compact"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("copy", "compact"):
        S, row, planes = _spread(rng, 2, 400), _spread(rng, 100, 100000), _spread(rng, 1, 24)
        planes = max(1, min(planes, (1 << 26) // (S * row)))
        c = dict(op=op, planes=planes, S=S, row=row, dtype=dtype)
        return dict(c, n=rng.randint(1, S // 2)) if op == "copy" else c
    if op in ("gn", "gn_bwd"):
        G = rng.choice([1, 1, 4, 7, 12, 40])
        D = G * _spread(rng, max(8, 64 // G), 8192 // G)
        return dict(op=op, rows=_spread(rng, 1, min(40000, (1 << 25) // D)), D=D, G=G, dtype=dtype,
                    gate=rng.choice([None, "before", "after"]), silu=rng.random() < 0.3,
                    center=rng.random() < 0.6, affine=rng.random() < 0.8)
    G = rng.choice([1, 2, 3, 5, 8, 16])
    c = dict(op=op, G=G, H=G * rng.choice([1, 1, 2, 4]), N=rng.choice([32, 64, 64, 128]),
             P=rng.choice([32, 64, 64, 128]), dtype=dtype, fixed=rng.random() < 0.3)
    size = c["H"] * max(c["N"], c["P"])
    if op == "la_step":
        B = _spread(rng, 1, min(256, (1 << 25) // (c["H"] * c["N"] * c["P"])))
        return dict(c, B=B, S=rng.choice([0, B + rng.randint(0, 20)]))
    B = _spread(rng, 1, 16)
    most = max(1, min(8192, (1 << 25) // (B * size)))
    return dict(c, B=B, T=_spread(rng, 1, most), state=rng.random() < 0.5,
                rows=rng.choice(["full", "padded", "packed"]))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dtype, op = _type(case), case["op"]
    s = dict(case=case)
    if op in ("copy", "compact"):
        S = case["S"]
        s["pool"] = normal(case["planes"], S, case["row"]).to(dtype)
        order = torch.randperm(S, generator=gen, device="cuda")
        if op == "compact":
            s["keep"] = uniform(S) < 0.5
        else:
            # Free slots take copies of the others (one of them perhaps several times) or zeros.
            n = case["n"]
            src = order[n:][torch.randint(0, S - n, (n,), generator=gen, device="cuda")]
            s["src"] = torch.where(uniform(n) < 0.1, -1, src).to(torch.int32)
            s["dst"] = order[:n].to(torch.int32)
        return s
    if op in ("gn", "gn_bwd"):
        rows, D = case["rows"], case["D"]
        s["x"] = (normal(rows, D) + normal(D, scale=0.5)).to(dtype)
        s["z"] = normal(rows, D).to(dtype) if case["gate"] else None
        s["gamma"] = 1 + normal(D, scale=0.2) if case["affine"] else None
        s["beta"] = normal(D, scale=0.2) if case["affine"] else None
        s["dy"] = normal(rows, D).to(dtype) if op == "gn_bwd" else None
        return s
    B, H, G, N, P = (case[k] for k in "BHGNP")
    s["scale"] = N ** -0.5
    s["lengths"] = s["starts"] = None
    if op == "la_step":
        tokens = (B,)
        states = case["S"] or B
        s["s0"] = normal(states, H, P, N)
        s["slots"] = None
        if case["S"]:
            s["slots"] = torch.randperm(states, generator=gen, device="cuda")[:B].to(torch.int32)
    else:
        T = case["T"]
        tokens = (B, T)
        if case["rows"] == "padded":
            # From none to all of the tokens; the last row fills the batch.
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            s["lengths"][B - 1] = T
        elif case["rows"] == "packed":
            # Evenly from none to all, in any order: as many tokens for every seed.
            n = (torch.arange(B, device="cuda") + (B == 1)) * T // max(1, B - 1)
            n = n[torch.randperm(B, generator=gen, device="cuda")].to(torch.int32)
            s["starts"] = torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)])
            tokens = (int(s["starts"][-1]),)
        s["s0"] = normal(B, H, P, N) if case["state"] else None
    s["q"], s["k"] = (normal(*tokens, G, N).to(dtype) for _ in range(2))
    s["v"] = normal(*tokens, H, P).to(dtype)
    # Rates from 1/1000 to 1/2 of the state per token, over the heads; around them over the tokens.
    rate = torch.exp(math.log(1e-3) + uniform(H) * math.log(500.0))
    s["g"] = -rate if case["fixed"] else (-rate * torch.exp(normal(*tokens, H, scale=0.5))).to(dtype)
    if op in ("la_train", "la_bwd"):
        s["dy"] = normal(*tokens, H, P).to(dtype)
        s["dsT"] = normal(B, H, P, N) if case["state"] else None
    if op == "la_bwd":
        entering = _forward(s)[2]
        at, used = _blocks(s)
        s["ckpt"] = torch.zeros(_ckpt_rows(s), H, P, N, device="cuda", dtype=dtype)
        s["ckpt"][at[used]] = entering[used].to(dtype)
    return s


# ---- the plain form -------------------------------------------------------------------------


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _places(s):
    """Index of token t of sequence b among all tokens [B, T up to whole blocks], and whether it is one."""
    B, T = s["case"]["B"], s["case"]["T"]
    t = torch.arange((T + CHUNK - 1) // CHUNK * CHUNK, device="cuda")
    if s["starts"] is not None:
        first, n = s["starts"][:-1].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    else:
        first = torch.arange(B, device="cuda") * T
        n = torch.full_like(first, T) if s["lengths"] is None else s["lengths"].long()
    on = t < n[:, None]
    return torch.where(on, first[:, None] + t, 0), on


def _blocks(s):
    """Row of the checkpoint tensor for each block of each sequence [B, blocks], and whether it holds tokens."""
    B, T = s["case"]["B"], s["case"]["T"]
    blocks = torch.arange((T + CHUNK - 1) // CHUNK, device="cuda")
    b = torch.arange(B, device="cuda")[:, None]
    if s["starts"] is None:
        at = b * len(blocks) + blocks
    else:
        at = s["starts"][:-1, None].long() // CHUNK + b + blocks
    used = _places(s)[1][:, ::CHUNK]
    return torch.where(used, at, 0), used


def _ckpt_rows(s):
    B, T = s["case"]["B"], s["case"]["T"]
    return B * ((T + CHUNK - 1) // CHUNK) if s["starts"] is None else s["v"].shape[0] // CHUNK + B


def _blocked(s, name):
    """A token tensor in 32 bits as [B, blocks, heads, CHUNK, size], zero where there is no token."""
    x, H = s[name], s["case"]["H"]
    at, on = _places(s)
    flat = x.reshape(-1, *x.shape[1 if s["starts"] is not None else 2:]).float()
    if not flat.numel():
        flat = flat.new_zeros(1, *flat.shape[1:])
    v = torch.where(on.view(*on.shape, 1, 1), flat[at], 0.0)
    v = v.repeat_interleave(H // v.shape[2], dim=2)
    B, T = at.shape
    return v.view(B, T // CHUNK, CHUNK, H, -1).transpose(2, 3).contiguous()


def _decays(s):
    """Running sums of the log decays inside each block, in 64 bits, [B, blocks, H, CHUNK]."""
    at, on = _places(s)
    B, T = at.shape
    H, g = s["case"]["H"], s["g"]
    if s["case"]["fixed"]:
        g = g.double().expand(B, T, H)
    else:
        flat = g.reshape(-1, H).double()
        g = flat[at] if flat.numel() else flat.new_zeros(B, T, H)
    g = torch.where(on[..., None], g, 0.0)
    return g.view(B, T // CHUNK, CHUNK, H).transpose(2, 3).cumsum(3)


def _along(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dimension 1, by doubling spans."""
    a, b, span = a.clone(), b.clone(), 1
    while span < a.shape[1]:
        b[:, span:] = b[:, span:] + a[:, span:] * b[:, :-span]
        a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    return b


def _pairs(c):
    """exp(G_t - G_s) for s <= t, else 0: [B, blocks, H, t, s]."""
    d = c[..., :, None] - c[..., None, :]
    keep = torch.ones(CHUNK, CHUNK, device=c.device, dtype=torch.bool).tril()
    return torch.where(keep, torch.exp(torch.where(keep, d, 0.0)), 0.0).float()


def _behind(s, x):
    """[B, blocks, H, CHUNK, size] as the token tensor that the call returns, zero behind each row's end."""
    B, T, H = s["case"]["B"], s["case"]["T"], s["case"]["H"]
    x = x.transpose(2, 3).reshape(B, -1, H, x.shape[-1])
    if s["starts"] is None:
        return x[:, :T]
    return x[_places(s)[1]]


def _shared(s, x):
    """The sum over the heads of a group of [..., H, size]."""
    G = s["case"]["G"]
    return x.unflatten(-2, (G, -1)).sum(-2)


def _forward(s):
    """y, the last state, and the state entering every block."""
    q, k, v, c = _blocked(s, "q"), _blocked(s, "k"), _blocked(s, "v"), _decays(s)
    last = torch.exp(c[..., -1:] - c).float()
    whole = torch.exp(c[..., -1]).float()[..., None, None]
    add = torch.matmul((v * last[..., None]).transpose(3, 4).contiguous(), k)   # [B, blocks, H, P, N]
    if s["s0"] is not None:
        add[:, 0] += whole[:, 0] * s["s0"]
    after = _along(whole, add)
    first = s["s0"] if s["s0"] is not None else torch.zeros_like(after[:, 0])
    entering = torch.cat([first[:, None], after[:, :-1]], 1)
    y = torch.matmul(torch.matmul(q, k.transpose(3, 4).contiguous()) * _pairs(c), v)
    y += torch.exp(c).float()[..., None] * torch.matmul(q, entering.transpose(3, 4).contiguous())
    return _behind(s, s["scale"] * y), after[:, -1].clone(), entering


def _la(s):
    y, sT, _ = _forward(s)
    return y.to(s["v"].dtype), sT


def _grads(s, entering):
    dtype = s["v"].dtype
    q, k, v, dy, c = (_blocked(s, "q"), _blocked(s, "k"), _blocked(s, "v"), _blocked(s, "dy"), _decays(s))
    dy = dy * s["scale"]
    first, last = torch.exp(c).float()[..., None], torch.exp(c[..., -1:] - c).float()[..., None]
    whole = torch.exp(c[..., -1]).float()[..., None, None]
    add = torch.matmul((dy * first).transpose(3, 4).contiguous(), q)
    if s["dsT"] is not None:
        # the last state's gradient, as what a block behind the last one would add
        add = torch.cat([add, s["dsT"][:, None]], 1)
        behind = torch.cat([whole, torch.ones_like(whole[:, :1])], 1)
    else:
        add, behind = torch.cat([add, torch.zeros_like(add[:, :1])], 1), torch.cat([whole, whole[:, :1]], 1)
    before = _along(behind.flip(1), add.flip(1)).flip(1)   # the gradient of the state entering each block
    ds = before[:, 1:]                                     # and of the state behind it
    pairs = _pairs(c)
    kq = torch.matmul(q, k.transpose(3, 4).contiguous()) * pairs
    vy = torch.matmul(dy, v.transpose(3, 4).contiguous())
    both = kq * vy
    vy = vy * pairs
    dq0 = first * torch.matmul(dy, entering)
    dk0 = last * torch.matmul(v, ds)
    dv = torch.matmul(kq.transpose(3, 4).contiguous(), dy) + last * torch.matmul(k, ds.transpose(3, 4).contiguous())
    dq = dq0 + torch.matmul(vy, k)
    dk = dk0 + torch.matmul(vy.transpose(3, 4).contiguous(), q)
    dg = None
    if not s["case"]["fixed"]:
        # pairs on both sides of t, tokens from t on with the state before, tokens before t with the
        # state behind, and the two states
        a, b = (q * dq0).sum(4), (k * dk0).sum(4)
        across = (both.sum(4) - both.sum(3) + a).double()
        across = across.flip(3).cumsum(3).flip(3)
        early = b.double().cumsum(3) - b
        dg = across + early + (whole * (entering * ds)).double().sum((3, 4))[..., None]
        dg = _behind(s, dg.float()[..., None])[..., 0].to(dtype)
    return dict(dq=_shared(s, _behind(s, dq)).to(dtype), dk=_shared(s, _behind(s, dk)).to(dtype),
                dv=_behind(s, dv).to(dtype), dg=dg if dg is None else _zeroed(s, dg), ds0=before[:, 0].clone())


def _zeroed(s, dg):
    """What the sums leave behind a padded row's end is 0."""
    if s["lengths"] is None:
        return dg
    return torch.where(_places(s)[1][:, :dg.shape[1], None], dg, 0.0)


def _la_train(s):
    y, sT, entering = _forward(s)
    return dict(_grads(s, entering), y=y.to(s["v"].dtype), sT=sT)


def _la_bwd(s):
    at, used = _blocks(s)
    return _grads(s, torch.where(used[..., None, None, None], s["ckpt"][at].float(), 0.0))


def _la_step(s):
    H = s["case"]["H"]
    at = slice(None) if s["slots"] is None else s["slots"].long()
    q, k = (s[n].float().repeat_interleave(H // s["case"]["G"], dim=1) for n in "qk")
    h = torch.exp(s["g"].float())[..., None, None] * s["s0"][at] + s["v"].float()[..., None] * k[..., None, :]
    s["s0"][at] = h
    return (s["scale"] * (h * q[..., None, :]).sum(3)).to(s["v"].dtype), s["s0"]


def _normed(s, wide):
    c = s["case"]
    x = s["x"].to(wide).view(c["rows"], c["G"], -1)
    z = None if s["z"] is None else s["z"].to(wide).view(x.shape)
    gate = None if z is None else z * _sigmoid(z)
    xg = x * gate if c["gate"] == "before" else x
    d = xg - xg.mean(2, keepdim=True) if c["center"] else xg
    rstd = 1 / torch.sqrt((d * d).mean(2, keepdim=True) + 1e-5)
    return x, z, gate, d * rstd, rstd


def _affine(s, n, wide):
    if s["gamma"] is None:
        return n
    return n * s["gamma"].to(wide).view(n.shape[1:]) + s["beta"].to(wide).view(n.shape[1:])


def _gn(s):
    c = s["case"]
    _, _, gate, n, _ = _normed(s, torch.float32)
    o = _affine(s, n, torch.float32)
    y = o * _sigmoid(o) if c["silu"] else o
    y = y * gate if c["gate"] == "after" else y
    return y.reshape(s["x"].shape).to(s["x"].dtype)


def _gn_grads(s):
    c, dtype = s["case"], s["x"].dtype
    x, z, gate, n, rstd = _normed(s, torch.float32)
    o = _affine(s, n, torch.float32)
    q = _sigmoid(o)
    dy = s["dy"].float().view(x.shape)
    dgate = None
    if c["gate"] == "after":
        dgate = dy * (o * q if c["silu"] else o)
        dy = dy * gate
    if c["silu"]:
        dy = dy * q * (1 + o * (1 - q))
    dgamma = dbeta = None
    if s["gamma"] is not None:
        dgamma, dbeta = (dy * n).sum(0).view(-1), dy.sum(0).view(-1)
        dy = dy * s["gamma"].view(n.shape[1:])
    dx = dy - n * (dy * n).mean(2, keepdim=True)
    if c["center"]:
        dx = dx - dy.mean(2, keepdim=True)
    dx = dx * rstd
    if c["gate"] == "before":
        dgate, dx = dx * x, dx * gate
    dz = None
    if z is not None:
        qz = _sigmoid(z)
        dz = (dgate * qz * (1 + z * (1 - qz))).reshape(s["x"].shape).to(dtype)
    return dict(dx=dx.reshape(s["x"].shape).to(dtype), dgamma=dgamma, dbeta=dbeta, dz=dz)


def _copy(s):
    src = s["src"].long()
    rows = s["pool"][:, src.clamp(min=0)]
    rows = torch.where((src < 0)[:, None], 0.0, rows).to(rows.dtype)
    s["pool"][:, s["dst"].long()] = rows
    return s["pool"]


def _compact(s):
    """Kept slots behind the first `count` fill the free ones among those, both in order."""
    keep = s["keep"]
    S = keep.shape[0]
    count = keep.sum()
    i = torch.arange(S, device="cuda")
    front = i < count
    hole, late = ~keep & front, keep & ~front
    rank = late.cumsum(0) - 1
    # the holes in order, then the rest: a stable sort of truth values
    holes = torch.sort((~hole).to(torch.int32), stable=True)[1]
    moved = torch.where(late, holes[rank.clamp(min=0)], torch.where(keep, i, -1))
    filled = torch.cat([i, i[:1]])   # the last place takes what moves nothing
    filled[torch.where(late, moved, S)] = i
    take = torch.where(hole, filled[:S], i)
    s["pool"].copy_(s["pool"][:, take])
    return s["pool"], moved.to(torch.int32), count.to(torch.int32).view(1)


_PLAIN = dict(la=_la, la_train=_la_train, la_bwd=_la_bwd, la_step=_la_step, gn=_gn, gn_bwd=_gn_grads, copy=_copy,
              compact=_compact)


# ---- the library's calls --------------------------------------------------------------------


def _own(s):
    import rwkv_wkv7_delta_amd as wk
    c, op = s["case"], s["case"]["op"]
    if op == "copy":
        wk.slots_copy(s["pool"], s["src"], s["dst"])
        return s["pool"]
    if op == "compact":
        moved, count = wk.slots_compact(s["pool"], s["keep"])
        return s["pool"], moved, count
    if op in ("gn", "gn_bwd"):
        how = dict(z=s["z"], gate_first=c["gate"] == "before", silu=c["silu"], center=c["center"], eps=1e-5)
        if op == "gn":
            return wk.gnorm_forward(s["x"], c["G"], s["gamma"], s["beta"], **how)
        return wk.gnorm_backward(s["x"], s["dy"], c["G"], s["gamma"], s["beta"], **how)._asdict()
    ins = [s[n] for n in "qkvg"]
    if op == "la_step":
        return wk.linattn_step(*ins, s["s0"], slots=s["slots"], scale=s["scale"]), s["s0"]
    rows = dict(lengths=s["lengths"], starts=s["starts"], scale=s["scale"])
    if s["starts"] is not None:
        rows["max_len"] = c["T"]
    if op == "la_bwd":
        return wk.linattn_backward(*ins, s["dy"], s["ckpt"], dsT=s["dsT"], **rows)._asdict()
    y, sT, ckpt = wk.linattn_forward(*ins, s0=s["s0"], want_ckpt=op == "la_train", **rows)
    if op == "la_train":
        return dict(wk.linattn_backward(*ins, s["dy"], ckpt, dsT=s["dsT"], **rows)._asdict(), y=y, sT=sT)
    return y, sT


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op == "copy":
        return dict(bytes=2 * case["planes"] * case["n"] * case["row"] * e, flops=0)
    if op == "compact":
        # half of the slots go on, half of those lie behind the new end: a quarter is moved
        return dict(bytes=2 * case["planes"] * case["S"] // 4 * case["row"] * e, flops=0)
    if op in ("gn", "gn_bwd"):
        x = case["rows"] * case["D"]
        gate = case["gate"] is not None
        if op == "gn":
            return dict(bytes=x * e * (2 + gate) + 8 * case["D"], flops=x * (10 + 6 * gate))
        return dict(bytes=x * e * (3 + 2 * gate) + 16 * case["D"], flops=x * (20 + 12 * gate))
    B, H, G, N, P = (case[k] for k in "BHGNP")
    state = B * H * N * P * 4
    if op == "la_step":
        return dict(bytes=2 * state + B * (2 * G * N + 2 * H * P) * e, flops=5 * B * H * N * P)
    tokens = B * case["T"]
    if case["rows"] != "full":
        tokens = (B + 1) * case["T"] // 2 if case["rows"] == "padded" or B == 1 else B * case["T"] // 2
    qk, v = tokens * G * N * e, tokens * H * P * e
    g = 0 if case["fixed"] else tokens * H * e
    # Products of one token: with the state for the read-out and into the state, and with half a
    # block's keys and values.
    forward = tokens * H * (4 * N * P + CHUNK * (N + P))
    ends = state * (2 if case["state"] else 1)
    marks = tokens // CHUNK * H * N * P * e
    moved = 2 * qk + 2 * v + g + ends
    grads = 4 * qk + 3 * v + 2 * g + ends + marks
    if op == "la":
        return dict(bytes=moved, flops=forward)
    if op == "la_bwd":
        return dict(bytes=grads, flops=2 * forward + tokens * H * CHUNK * P)
    return dict(bytes=moved + grads + marks, flops=3 * forward + tokens * H * CHUNK * P)


# ---- the definition in 64 bits --------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("copy", "compact"):
        return None
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op == "gn":
        return _exact_norm(f, case)[0]
    if op == "gn_bwd":
        return _exact_norm(f, case)[1]
    if op == "la_step":
        at = list(range(case["B"])) if f["slots"] is None else f["slots"].tolist()
        rep = case["H"] // case["G"]
        state, y = f["s0"], []
        for b, i in enumerate(at):
            decay = torch.exp(f["g"] if case["fixed"] else f["g"][b])
            kb, qb = (f[n][b].repeat_interleave(rep, 0) for n in "kq")
            state[i] = decay[:, None, None] * state[i] + f["v"][b][:, :, None] * kb[:, None, :]
            y.append(f["scale"] * torch.einsum("hpn,hn->hp", state[i], qb))
        return torch.stack(y), state
    return _exact_scan(f, case)


def _exact_scan(f, case):
    """Token by token, every sequence beside the others."""
    B, T, H, G, N, P, op = (case[k] for k in ("B", "T", "H", "G", "N", "P", "op"))
    dev = f["v"].device
    if f["starts"] is not None:
        edges = f["starts"].tolist()
        first, n = edges[:-1], [b - a for a, b in zip(edges, edges[1:])]
    else:
        first = [b * T for b in range(B)]
        n = [T] * B if f["lengths"] is None else f["lengths"].tolist()

    def padded(name, size):
        x = f[name].reshape(-1, *size)
        out = x.new_zeros(T, B, *size)
        for b in range(B):
            out[:n[b], b] = x[first[b]:first[b] + n[b]]
        return out

    on = torch.tensor([[t < n[b] for b in range(B)] for t in range(T)], device=dev)
    q, k = (padded(name, (G, N)).repeat_interleave(H // G, 2) for name in "qk")
    v = padded("v", (H, P))
    g = f["g"].expand(T, B, H).clone() if case["fixed"] else padded("g", (H,))
    decay = torch.where(on[..., None], torch.exp(g), 1.0)[..., None, None]
    S = f["s0"].clone() if f["s0"] is not None else v.new_zeros(B, H, P, N)
    scale = f["scale"]

    def back(x, zero=True):
        """[T, B, ...] as the call's tensor."""
        if f["starts"] is not None:
            return torch.cat([x[:n[b], b] for b in range(B)])
        return torch.where(on.view(T, B, *[1] * (x.dim() - 2)), x, 0.0).transpose(0, 1)

    blocks = (T + CHUNK - 1) // CHUNK
    marks = []
    y = v.new_zeros(T, B, H, P)
    for t in range(T if op != "la_bwd" else 0):
        if t % CHUNK == 0:
            marks.append(S)
        S = decay[t] * S + v[t][..., None] * k[t][..., None, :]
        y[t] = scale * (S * q[t][..., None, :]).sum(-1)
    if op == "la":
        return back(y), S
    if op == "la_bwd":
        for m in range(blocks):
            row = [first[b] // CHUNK + b + m if f["starts"] is not None else b * blocks + m for b in range(B)]
            marks.append(torch.stack([f["ckpt"][row[b]] if m * CHUNK < n[b] else torch.zeros_like(f["ckpt"][0])
                                      for b in range(B)]))
    dy = padded("dy", (H, P)) * scale
    D = f["dsT"].clone() if f["dsT"] is not None else v.new_zeros(B, H, P, N)
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    for m in reversed(range(blocks)):
        states, t0, t1 = [marks[m]], m * CHUNK, min(T, m * CHUNK + CHUNK)
        for t in range(t0, t1):
            states.append(decay[t] * states[-1] + v[t][..., None] * k[t][..., None, :])
        for t in reversed(range(t0, t1)):
            D = D + dy[t][..., None] * q[t][..., None, :]
            dq[t] = (states[t - t0 + 1] * dy[t][..., None]).sum(-2)
            dv[t] = (D * k[t][..., None, :]).sum(-1)
            dk[t] = (D * v[t][..., None]).sum(-2)
            D = decay[t] * D
            dg[t] = (D * states[t - t0]).sum((-1, -2))
    dq, dk = (x.view(T, B, G, H // G, N).sum(3) for x in (dq, dk))
    out = dict(dq=back(dq), dk=back(dk), dv=back(dv), dg=None if case["fixed"] else back(dg), ds0=D)
    return out if op == "la_bwd" else dict(out, y=back(y), sT=S)


def _exact_norm(f, case):
    rows, D, G = case["rows"], case["D"], case["G"]
    width = D // G
    x = f["x"].reshape(rows * G, width)
    z = None if f["z"] is None else f["z"].reshape(rows * G, width)
    gate = None if z is None else z * torch.sigmoid(z)
    u = x * gate if case["gate"] == "before" else x
    mean = u.sum(1, keepdim=True) / width if case["center"] else torch.zeros_like(u[:, :1])
    r = ((u - mean).square().sum(1, keepdim=True) / width + 1e-5) ** -0.5
    h = (u - mean) * r
    gamma = torch.ones(D, device=x.device, dtype=x.dtype) if f["gamma"] is None else f["gamma"]
    beta = torch.zeros_like(gamma) if f["beta"] is None else f["beta"]
    gw, bw = (p.view(1, G, width).expand(rows, G, width).reshape(rows * G, width) for p in (gamma, beta))
    o = gw * h + bw
    act = o * torch.sigmoid(o) if case["silu"] else o
    y = act * gate if case["gate"] == "after" else act
    shape = f["x"].shape
    if f["dy"] is None:
        return y.view(shape), None
    e = f["dy"].reshape(rows * G, width)
    dz = None
    if case["gate"] == "after":
        dz = e * act
        e = e * gate
    if case["silu"]:
        e = e * torch.sigmoid(o) * (1 + o - act)
    dgamma, dbeta = ((e * p).view(rows, D).sum(0) for p in (h, torch.ones_like(h)))
    e = e * gw
    # u enters through itself, through the mean and through the variance
    dvar = (e * (u - mean)).sum(1, keepdim=True) * -0.5 * r ** 3
    du = e * r + dvar * 2 * (u - mean) / width
    if case["center"]:
        du = du - (e * r).sum(1, keepdim=True) / width
    if case["gate"] == "before":
        dz, du = du * x, du * gate
    if dz is not None:
        dz = (dz * (torch.sigmoid(z) + gate * (1 - torch.sigmoid(z)))).view(shape)
    affine = f["gamma"] is not None
    return y.view(shape), dict(dx=du.view(shape), dgamma=dgamma if affine else None,
                               dbeta=dbeta if affine else None, dz=dz)
