"""Measured cases of the short causal convolution, the selective state-space scan
(prompts, gradients, single tokens) and the scan's 8-bit state checkpoints.

Short convolution, per channel d with W taps:
    pre_t = bias + sum_k weight[k] x_{t-(W-1)+k},   y_t = pre_t or pre_t sigmoid(pre_t)
with the W - 1 inputs before the first token taken from a state.  W = 2 without
the activation is the token shift in front of a time-mixing layer.

Selective scan, per channel d with N states, B_t and C_t shared by the channels
of a group:
    D_t = softplus(dt_t + dt_bias),   h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t x_t B_t[n]
    y_t = (sum_n C_t[n] h_t[n] + dskip x_t) z_t sigmoid(z_t)

A training forward keeps the state entering every 16 tokens, in 32 bits or as
8-bit codes with one scale per channel; the backward recomputes the states of a
16-token block from it.
"""

import math

import torch

own = False

CHUNK = 16   # tokens per state checkpoint


def listed():
    return [
        # The token shift of a training step at the 2.9B width (40 heads of 64).
        dict(name="shift_2560", op="conv", B=8, T=4096, D=2560, W=2, dtype="bf16", silu=False,
             bias=False, state=False, lengths=False),
        # Prompts of different lengths, each continuing an earlier state; an odd width, whose
        # rows no vector access fits.
        dict(name="conv_ragged", op="conv", B=5, T=1021, D=1001, W=4, dtype="fp32", silu=True,
             bias=True, state=True, lengths=True),
        # Gradients of the convolution in a training step at the 1.5B width (32 heads of 64).
        dict(name="conv_grads", op="conv_bwd", B=4, T=4096, D=2048, W=4, dtype="bf16", silu=True,
             bias=True, state=False, lengths=False),
        # One token of one sequence: the smallest call, where latency counts.
        dict(name="conv_token", op="conv_step", B=1, D=768, W=4, dtype="bf16", silu=True, bias=True),
        # Forward of a training or prompt batch at the 1.5B width.
        dict(name="scan_2048", op="scan", B=8, T=4096, D=2048, N=16, G=1, dtype="bf16", gate=True,
             state=False, lengths=False),
        # One long prompt at the 0.19B width (12 heads of 64): few channels, many tokens.
        dict(name="scan_long", op="scan", B=1, T=16384, D=768, N=16, G=1, dtype="bf16", gate=True,
             state=True, lengths=False),
        # A padded batch in fp32 with groups, a small state and an odd width.
        dict(name="scan_ragged", op="scan", B=3, T=1021, D=1001, N=8, G=7, dtype="fp32", gate=False,
             state=True, lengths=True),
        # One training step (forward with fp32 checkpoints, then every gradient) at the 0.19B
        # shape.
        dict(name="step_768", op="scan_train", B=4, T=1024, D=768, N=16, G=1, dtype="bf16", gate=True,
             state=True, lengths=False),
        # Gradients from 8-bit checkpoints at the 1.5B width.
        dict(name="grads8_2048", op="scan_bwd8", B=4, T=4096, D=2048, N=16, G=1, dtype="bf16",
             gate=True, state=False, lengths=False),
        # The same for a padded fp32 batch with two groups, a larger state and an odd width.
        dict(name="grads8_ragged", op="scan_bwd8", B=2, T=333, D=130, N=32, G=2, dtype="fp32",
             gate=False, state=True, lengths=True),
        # The forward that writes 8-bit checkpoints.
        dict(name="ckpt8_2048", op="scan_ckpt8", B=2, T=2048, D=2048, N=16, G=1, dtype="bf16",
             gate=True, state=False, lengths=False),
        # One token of every sequence that a serving batch decodes, at the 2.9B width.
        dict(name="scan_token", op="scan_step", B=256, D=2560, N=16, G=1, dtype="bf16", gate=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "scan", "scan_train", "scan_bwd8",
                     "scan_ckpt8", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("conv"):
        c = dict(op=op, D=_spread(rng, 64, 5120), W=rng.choice([2, 3, 4]), dtype=dtype,
                 silu=rng.random() < 0.6, bias=rng.random() < 0.5)
        if op == "conv_step":
            return dict(c, B=_spread(rng, 1, 512))
        # At most half of the largest listed convolution's elements, for 4-byte types' sake.
        B = _spread(rng, 1, 32)
        most = min(8192, (1 << 25) // (B * c["D"]))
        return dict(c, B=B, T=_spread(rng, 1, max(1, most)), state=rng.random() < 0.5,
                    lengths=rng.random() < 0.3)
    N, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
    c = dict(op=op, D=G * _spread(rng, 32, 2048 // G), N=N, G=G, dtype=dtype, gate=rng.random() < 0.6)
    if op == "scan_step":
        return dict(c, B=_spread(rng, 1, 256))
    B = _spread(rng, 1, 16)
    most = (1 << 29 if op == "scan" else 1 << 28) // (B * c["D"] * N)
    return dict(c, B=B, T=_spread(rng, 1, max(1, min(8192, most))), state=rng.random() < 0.5,
                lengths=rng.random() < 0.3)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dtype, B, D, T = _type(case), case["B"], case["D"], case.get("T")
    s = dict(case=case)
    step = case["op"].endswith("step")
    tokens = (B, D) if step else (B, T, D)
    s["lengths"] = None
    if case.get("lengths"):
        # From none to all of the tokens; the longest row fills the batch.
        s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["lengths"][B - 1] = T
    s["x"] = normal(*tokens).to(dtype)
    if case["op"].startswith("conv"):
        W = case["W"]
        s["weight"] = normal(D, W, scale=W ** -0.5)
        s["bias"] = normal(D, scale=0.1) if case["bias"] else None
        s["s0"] = normal(B, W - 1, D).to(dtype) if step or case["state"] else None
        if case["op"] == "conv_bwd":
            s["dy"] = normal(B, T, D).to(dtype)
            s["dsT"] = normal(B, W - 1, D).to(dtype) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    s["dt"] = normal(*tokens, scale=0.5).to(dtype)
    # Steps of 0.001 to 0.1 around which dt varies, and decay rates from 1 to N.
    first = torch.exp(math.log(1e-3) + uniform(D) * math.log(100.0))
    s["dt_bias"] = torch.log(torch.expm1(first))
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(D, N, scale=0.2))
    s["Bm"], s["Cm"] = (normal(*tokens[:-1], G, N).to(dtype) for _ in range(2))
    s["dskip"] = 1 + normal(D, scale=0.1)
    s["z"] = normal(*tokens).to(dtype) if case["gate"] else None
    s["h0"] = normal(B, D, N, scale=0.1) if step or case["state"] else None
    if case["op"] in ("scan_train", "scan_bwd8"):
        s["dy"] = normal(B, T, D).to(dtype)
        s["dhT"] = normal(B, D, N, scale=0.1) if case["state"] else None
    if case["op"] == "scan_bwd8":
        h = _states(s)[0]
        first = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0])
        codes, scales = _codes(torch.cat([first[:, None], h[:, CHUNK - 1:T - 1:CHUNK]], 1))
        s["ckpt"] = _packed(codes, scales)
    return s


# ---- the plain form -------------------------------------------------------------------------


def _valid(s, x):
    """Truth of "token t lies within its row's length", shaped to broadcast over x [B, T, ...]."""
    if s["lengths"] is None:
        return None
    t = torch.arange(x.shape[1], device=x.device)
    return (t < s["lengths"].clamp(0, x.shape[1])[:, None]).view(x.shape[0], x.shape[1], *[1] * (x.dim() - 2))


def _tokens(s, name):
    """A token tensor in 32 bits, zero behind each row's length."""
    x = s[name].float()
    m = _valid(s, x)
    return x if m is None else torch.where(m, x, 0.0)


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _windows(s, T):
    """The convolution's inputs with the state in front, [B, W - 1 + T, D]."""
    x = _tokens(s, "x")
    W = s["case"]["W"]
    s0 = s["s0"].float() if s["s0"] is not None else x.new_zeros(x.shape[0], W - 1, x.shape[2])
    return torch.cat([s0, x], 1)


def _last_inputs(s, T):
    """Places of the last W - 1 inputs of each row in _windows, [B, W - 1, 1]."""
    W, B = s["case"]["W"], s["case"]["B"]
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long().clamp(0, T)
    return (n[:, None] + torch.arange(W - 1, device="cuda"))[:, :, None]


def _conv_sums(s, ext, T):
    w = s["weight"]
    pre = sum(ext[:, k:k + T] * w[:, k] for k in range(w.shape[1]))
    return pre if s["bias"] is None else pre + s["bias"]


def _conv(s):
    T, dtype = s["case"]["T"], s["x"].dtype
    ext = _windows(s, T)
    pre = _conv_sums(s, ext, T)
    y = pre * _sigmoid(pre) if s["case"]["silu"] else pre
    m = _valid(s, y)
    y = y if m is None else torch.where(m, y, 0.0)
    sT = torch.gather(ext, 1, _last_inputs(s, T).expand(-1, -1, ext.shape[2]))
    return y.to(dtype), sT.to(dtype)


def _conv_grads(s):
    T, dtype, w = s["case"]["T"], s["x"].dtype, s["weight"]
    W = w.shape[1]
    ext = _windows(s, T)
    g = _tokens(s, "dy")
    if s["case"]["silu"]:
        pre = _conv_sums(s, ext, T)
        q = _sigmoid(pre)
        g = g * q * (1 + pre * (1 - q))
    dext = torch.zeros_like(ext)
    for k in range(W):
        dext[:, k:k + T] += g * w[:, k]
    if s["dsT"] is not None:
        dext.scatter_add_(1, _last_inputs(s, T).expand(-1, -1, ext.shape[2]), s["dsT"].float())
    dweight = torch.stack([(g * ext[:, k:k + T]).sum((0, 1)) for k in range(W)], 1)
    dbias = g.sum((0, 1)) if s["bias"] is not None else None
    dx, ds0 = dext[:, W - 1:], dext[:, :W - 1]
    m = _valid(s, dx)
    dx = dx if m is None else torch.where(m, dx, 0.0)
    return dx.to(dtype), dweight, dbias, ds0.to(dtype)


def _conv_step(s):
    x, w = s["x"].float(), s["weight"]
    ext = torch.cat([s["s0"].float(), x[:, None]], 1)
    pre = (ext * w.t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = pre * _sigmoid(pre) if s["case"]["silu"] else pre
    s["s0"].copy_(ext[:, 1:])
    return y.to(s["x"].dtype), s["s0"]


def _along(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dimension 1, by doubling spans."""
    a, b, span = a.clone(), b.clone(), 1
    while span < a.shape[1]:
        b[:, span:] = b[:, span:] + a[:, span:] * b[:, :-span]
        a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    return b


def _rates(s):
    """D_t (zero behind each row's length) and the slope of the softplus."""
    v = s["dt"].float() + s["dt_bias"]
    d = _softplus(v)
    m = _valid(s, v) if v.dim() == 3 else None
    return (d if m is None else torch.where(m, d, 0.0)), _sigmoid(v)


def _shared(s, name):
    """B or C for every channel, [B, T, D, N]."""
    v = _tokens(s, name)
    return v.repeat_interleave(s["case"]["D"] // s["case"]["G"], dim=2)


def _states(s):
    """h_t, exp(D_t A), D_t, B_t for every token, [B, T, D, N]."""
    d = _rates(s)[0]
    a, bm = torch.exp(d[..., None] * s["A"]), _shared(s, "Bm")
    b = (d * _tokens(s, "x"))[..., None] * bm
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    return _along(a, b), a, d, bm


def _gated(s, y):
    if s["z"] is None:
        return y
    z = _tokens(s, "z") if y.dim() == 3 else s["z"].float()
    return y * z * _sigmoid(z)


def _scan(s):
    h = _states(s)[0]
    y = (h * _shared(s, "Cm")).sum(3) + s["dskip"] * _tokens(s, "x")
    return _gated(s, y).to(s["x"].dtype), h[:, -1].clone(), h


def _codes(h):
    """8-bit codes and scales of states [..., N]: one scale for the N states of a channel."""
    scales = h.abs().amax(-1) / 127
    most = h.abs().amax(-1, keepdim=True)
    codes = torch.round(h * torch.where(most > 0, 127 / most, 0.0))
    return codes.to(torch.int8), scales


def _packed(codes, scales):
    """The checkpoint as one buffer: the codes, then from a 16-byte boundary the scales."""
    flat = codes.reshape(-1).view(torch.uint8)
    pad = -flat.numel() % 16
    return torch.cat([flat, flat.new_zeros(pad), scales.reshape(-1).view(torch.uint8)])


def _unpacked(s):
    c = s["case"]
    n = (c["T"] + CHUNK - 1) // CHUNK
    size = c["B"] * n * c["D"] * c["N"]
    codes = s["ckpt"][:size].view(torch.int8).view(c["B"], n, c["D"], c["N"])
    scales = s["ckpt"][size + -size % 16:].view(torch.float32).view(c["B"], n, c["D"])
    return codes.float() * scales[..., None]


def _block_states(s, first):
    """h_{t-1} and h_t with every 16-token block started from first [B, blocks, D, N]."""
    d = _rates(s)[0]
    a, bm = torch.exp(d[..., None] * s["A"]), _shared(s, "Bm")
    b = (d * _tokens(s, "x"))[..., None] * bm
    B, T, D, N = a.shape
    n = first.shape[1]
    pad = (0, 0, 0, 0, 0, n * CHUNK - T)
    pa = torch.nn.functional.pad(a, pad).view(B * n, CHUNK, D, N)
    pb = torch.nn.functional.pad(b, pad).view(B * n, CHUNK, D, N)
    start = first.reshape(B * n, 1, D, N)
    pb[:, 0] += pa[:, 0] * start[:, 0]
    h = _along(pa, pb)
    before = torch.cat([start, h[:, :-1]], 1)
    return [v.reshape(B, n * CHUNK, D, N)[:, :T] for v in (before, h)] + [a, d, bm]


def _scan_grads(s, before, h, a, d, bm):
    dtype, x, cm = s["x"].dtype, _tokens(s, "x"), _shared(s, "Cm")
    dy, dz = _tokens(s, "dy"), None
    if s["z"] is not None:
        z = _tokens(s, "z")
        q = _sigmoid(z)
        y = (h * cm).sum(3) + s["dskip"] * x
        dz = (dy * y * q * (1 + z * (1 - q))).to(dtype)
        dy = dy * z * q
    g = dy[..., None] * cm
    if s["dhT"] is not None:
        g[:, -1] += s["dhT"]
    # g_t = dy_t C_t + exp(D_{t+1} A) g_{t+1}
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _along(later.flip(1), g.flip(1)).flip(1)
    B, T, D, N = g.shape
    G = s["case"]["G"]
    groups = (B, T, G, D // G, N)
    dC = (dy[..., None] * h).view(groups).sum(3)
    dB = (g * (d * x)[..., None]).view(groups).sum(3)
    du = (g * bm).sum(3)
    dh0 = a[:, 0] * g[:, 0]
    r = g * a * before
    dA = (r * d[..., None]).sum((0, 1))
    ddt = (du * x + (r * s["A"]).sum(3)) * _rates(s)[1]
    m = _valid(s, ddt)
    ddt = ddt if m is None else torch.where(m, ddt, 0.0)
    return dict(dx=(du * d + dy * s["dskip"]).to(dtype), ddt=ddt.to(dtype), dA=dA, dB=dB.to(dtype),
                dC=dC.to(dtype), dz=dz, ddskip=(dy * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dh0=dh0)


def _scan_train(s):
    h, a, d, bm = _states(s)
    y = _gated(s, (h * _shared(s, "Cm")).sum(3) + s["dskip"] * _tokens(s, "x")).to(s["x"].dtype)
    first = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0])
    return dict(_scan_grads(s, torch.cat([first[:, None], h[:, :-1]], 1), h, a, d, bm), y=y, hT=h[:, -1].clone())


def _scan_ckpt8(s):
    y, hT, h = _scan(s)
    first = s["h0"] if s["h0"] is not None else torch.zeros_like(hT)
    codes, scales = _codes(torch.cat([first[:, None], h[:, CHUNK - 1:-1:CHUNK]], 1))
    return y, hT, (codes.float() * scales[..., None]).to(torch.bfloat16)


def _scan_step(s):
    d, x, G = _rates(s)[0], s["x"].float(), s["case"]["G"]
    bm, cm = (s[k].float().repeat_interleave(s["case"]["D"] // G, dim=1) for k in ("Bm", "Cm"))
    h = torch.exp(d[..., None] * s["A"]) * s["h0"] + (d * x)[..., None] * bm
    s["h0"].copy_(h)
    return _gated(s, (h * cm).sum(2) + s["dskip"] * x).to(s["x"].dtype), s["h0"]


_PLAIN = dict(conv=_conv, conv_bwd=_conv_grads, conv_step=_conv_step, scan=lambda s: _scan(s)[:2],
              scan_train=_scan_train, scan_ckpt8=_scan_ckpt8, scan_step=_scan_step,
              scan_bwd8=lambda s: _scan_grads(s, *_block_states(s, _unpacked(s))))


# ---- the library's calls --------------------------------------------------------------------


def _own(s):
    import rwkv_wkv7_delta_amd as wk
    c, op = s["case"], s["case"]["op"]
    if op == "conv":
        return wk.conv_forward(s["x"], s["weight"], s["bias"], s0=s["s0"], lengths=s["lengths"],
                               silu=c["silu"], want_state=True)
    if op == "conv_bwd":
        return wk.conv_backward(s["x"], s["weight"], s["dy"], s["bias"], s0=s["s0"], dsT=s["dsT"],
                                lengths=s["lengths"], silu=c["silu"])
    if op == "conv_step":
        y = wk.conv_step(s["x"], s["weight"], s["s0"], s["bias"], silu=c["silu"])
        return y, s["s0"]
    parts = dict(z=s["z"], dskip=s["dskip"], dt_bias=s["dt_bias"])
    ins = [s[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    if op == "scan_step":
        y = wk.ssm_step(*ins, s["h0"], **parts)
        return y, s["h0"]
    parts["lengths"] = s["lengths"]
    if op == "scan_bwd8":
        return wk.ssm_backward(*ins, s["dy"], s["ckpt"], ckpt_bits=8, dhT=s["dhT"], **parts)._asdict()
    bits = dict(scan=0, scan_train=32, scan_ckpt8=8)[op]
    y, hT, ckpt = wk.ssm_forward(*ins, h0=s["h0"], ckpt_bits=bits, **parts)
    if op == "scan_train":
        grads = wk.ssm_backward(*ins, s["dy"], ckpt, ckpt_bits=32, dhT=s["dhT"], **parts)
        return dict(grads._asdict(), y=y, hT=hT)
    if op == "scan_ckpt8":
        codes, scales = wk.ssm_split_ckpt(ckpt, c["B"], c["T"], c["D"], c["N"])
        return y, hT, (codes * scales[..., None]).to(torch.bfloat16)
    return y, hT


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T, D = case["B"], case.get("T", 1), case["D"]
    tok = B * T * D * e
    op = case["op"]
    if op.startswith("conv"):
        W = case["W"]
        past = B * (W - 1) * D * e
        params = D * (W + 1) * 4
        if op == "conv_bwd":
            return dict(bytes=3 * tok + past + 2 * params, flops=4 * W * B * T * D)
        return dict(bytes=2 * tok + past * (2 if op == "conv_step" or case["state"] else 1) + params,
                    flops=2 * W * B * T * D)
    N, G = case["N"], case["G"]
    bc = 2 * B * T * G * N * e
    state = B * D * N * 4
    params = D * (N + 2) * 4
    blocks = B * ((T + CHUNK - 1) // CHUNK) * D
    # x, dt, y and the gate; a state update is a product, an exponential and two fused
    # multiply-adds, the read-out one more.
    forward = tok * (4 if case["gate"] else 3) + bc + state + params
    grads = tok * (7 if case["gate"] else 5) + 2 * bc + 2 * params
    per = 7 * B * T * D * N
    if op == "scan_bwd8":
        return dict(bytes=grads + blocks * (N + 4) + state, flops=3 * per)
    if op == "scan_train":
        return dict(bytes=forward + grads + 2 * state, flops=4 * per)
    return dict(bytes=forward + (blocks * (N + 4) if op == "scan_ckpt8" else 0) +
                (state if op == "scan_step" or (op == "scan" and case["state"]) else 0), flops=per)


# ---- the definition in 64 bits --------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return _exact_conv(f, case) if case["op"].startswith("conv") else _exact_scan(f, case)


def _inside(f, B, T):
    """[B, T] of 1 for tokens within their row's length and 0 behind it, and the lengths."""
    n = torch.full((B,), T, device="cuda") if f["lengths"] is None else f["lengths"].long()
    return torch.stack([n > t for t in range(T)], 1), n


def _exact_conv(f, case):
    B, D, W = case["B"], case["D"], case["W"]
    step = case["op"] == "conv_step"
    T = 1 if step else case["T"]
    x = f["x"].view(B, T, D)
    inside, n = _inside(f, B, T)
    x = torch.where(inside[..., None], x, torch.zeros_like(x))
    past = f["s0"] if f["s0"] is not None else x.new_zeros(B, W - 1, D)

    def back(j):   # the input j tokens before each token
        if j == 0:
            return x
        rows = torch.cat([past[:, max(0, W - 1 - j):], x], 1)
        return rows[:, :T] if j <= W - 1 else None

    inputs = [back(W - 1 - k) for k in range(W)]
    pre = x.new_zeros(B, T, D) if f["bias"] is None else f["bias"].expand(B, T, D).clone()
    for k in range(W):
        pre += f["weight"][:, k] * inputs[k]
    gate = torch.sigmoid(pre)
    y = torch.where(inside[..., None], pre * gate if case["silu"] else pre, torch.zeros_like(pre))
    rows = torch.cat([past, x], 1)
    last = torch.stack([rows[b, n[b]:n[b] + W - 1] for b in range(B)])
    if step:
        return y[:, 0], last
    if case["op"] == "conv":
        return y, last
    slope = gate + pre * gate * (1 - gate) if case["silu"] else torch.ones_like(pre)
    g = torch.where(inside[..., None], f["dy"] * slope, torch.zeros_like(pre))
    drows = torch.zeros_like(rows)
    for t0 in range(W):   # tap k of token t reads rows[t + k]
        drows[:, t0:t0 + T] += f["weight"][:, t0] * g
    if f["dsT"] is not None:
        for b in range(B):
            drows[b, n[b]:n[b] + W - 1] += f["dsT"][b]
    dx = torch.where(inside[..., None], drows[:, W - 1:], torch.zeros_like(x))
    dw = torch.stack([(g * inputs[k]).sum((0, 1)) for k in range(W)], 1)
    return dx, dw, None if f["bias"] is None else g.sum((0, 1)), drows[:, :W - 1]


def _exact_scan(f, case):
    B, D, N, G, op = case["B"], case["D"], case["N"], case["G"], case["op"]
    step = op == "scan_step"
    T = 1 if step else case["T"]
    inside, _ = _inside(f, B, T)
    on = lambda v: torch.where(inside.view(B, T, *[1] * (v.dim() - 2)), v, torch.zeros_like(v))  # noqa: E731
    x = on(f["x"].view(B, T, D))
    bm, cm = (on(f[k].view(B, T, G, N)) for k in ("Bm", "Cm"))
    raw = f["dt"].view(B, T, D) + f["dt_bias"]
    rate = on(torch.logaddexp(raw, torch.zeros_like(raw)))
    z = None if f["z"] is None else on(f["z"].view(B, T, D))
    h = f["h0"].clone() if f["h0"] is not None else x.new_zeros(B, D, N)
    A, width = f["A"], D // G
    entry = None
    if op == "scan_bwd8":
        m = (T + CHUNK - 1) // CHUNK
        size = B * m * D * N
        raw8 = f["ckpt"].cpu()
        codes = raw8[:size].view(torch.int8).double().view(B, m, D, N)
        scales = raw8[size + -size % 16:].view(torch.float32).double().view(B, m, D, 1)
        entry = (codes * scales).cuda()
    keep = op in ("scan_bwd8", "scan_train")
    hs = x.new_zeros(B, T + 1, D, N) if keep else None
    starts, marks, y = {}, [], x.new_zeros(B, T, D)
    for t in range(T):
        if t % CHUNK == 0:
            if entry is not None:
                h = entry[:, t // CHUNK].clone()
                starts[t] = h
            elif op == "scan_ckpt8":
                marks.append(h)
        bt, ct = (v[:, t].repeat_interleave(width, dim=1) for v in (bm, cm))
        h = torch.exp(rate[:, t, :, None] * A) * h + (rate[:, t] * x[:, t])[..., None] * bt
        y[:, t] = (h * ct).sum(-1) + f["dskip"] * x[:, t]
        if keep:
            hs[:, t + 1] = h
    if keep and f["h0"] is not None:
        hs[:, 0] = f["h0"]
    out = y if z is None else y * z * torch.sigmoid(z)
    if step:
        return out[:, 0], h
    if op == "scan":
        return out, h
    if op == "scan_ckpt8":
        e = torch.stack(marks, 1)
        top = e.abs().amax(-1, keepdim=True)
        return out, h, torch.round(e * 127 / torch.where(top > 0, top, torch.ones_like(top))) * (top / 127)
    dout = on(f["dy"])
    gate = torch.sigmoid(z) if z is not None else None
    dy = dout if z is None else dout * z * gate
    g = f["dhT"].clone() if f["dhT"] is not None else x.new_zeros(B, D, N)
    du, dr = torch.zeros_like(x), torch.zeros_like(x)
    dA = x.new_zeros(D, N)
    dB, dC = torch.zeros_like(bm), torch.zeros_like(cm)
    for t in reversed(range(T)):   # g: the gradient of h_t from the tokens behind it
        bt, ct = (v[:, t].repeat_interleave(width, dim=1) for v in (bm, cm))
        g = g + dy[:, t, :, None] * ct
        dC[:, t] = (dy[:, t, :, None] * hs[:, t + 1]).view(B, G, width, N).sum(2)
        dB[:, t] = (g * (rate[:, t] * x[:, t])[..., None]).view(B, G, width, N).sum(2)
        du[:, t] = (g * bt).sum(-1)
        g = g * torch.exp(rate[:, t, :, None] * A)
        q = g * starts.get(t, hs[:, t])
        dr[:, t] = (q * A).sum(-1)
        dA += (q * rate[:, t, :, None]).sum(0)
    ddt = on((du * x + dr) * torch.sigmoid(raw))
    grads = dict(dx=du * rate + dy * f["dskip"], ddt=ddt, dA=dA, dB=dB, dC=dC,
                 dz=None if z is None else dout * y * (gate + z * gate * (1 - gate)),
                 ddskip=(dy * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dh0=g)
    return grads if op == "scan_bwd8" else dict(grads, y=out, hT=h)
