"""Cases of a state space layer in its residual block: the short causal convolution
before the scan (short_conv), the selective scan with N numbers of state a channel
(ssm), and the norms before and after a block with its gate and residual scale
(block_norm), each forward, backward and for single tokens.

`run` computes a case with elementary torch operations, or, with `own` set,
through retnet_retention_gb300.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
RANK = 64  # columns before b and c in the projection they are slices of


def listed():
    """Sizes: the repository's workloads (8 x 8192 tokens, one sequence of 65,536, 256
    decoding sequences, 4 x 4096 tokens) and widths (1024, 2048, 4096), and ragged ones."""
    return [
        # a decode step of 256 sequences through 4096 channels, x a slice of the packed projection
        dict(name="conv_step", op="conv_step", B=256, T=1, D=4096, W=4, dtype="bf16", silu=True, bias=True,
             state=True, positions=False),
        # the prefill's tokens, x a slice of the packed projection
        dict(name="conv_prefill", op="conv", B=8, T=8192, D=4096, W=4, dtype="bf16", silu=True, bias=True,
             state=False, positions=False),
        # ragged, fp32, three taps without activation, documents packed behind a history
        dict(name="conv_ragged", op="conv", B=3, T=1021, D=208, W=3, dtype="f32", silu=False, bias=False,
             state=True, positions=True),
        # a training step's gradients, packed documents
        dict(name="conv_train", op="conv_bwd", B=4, T=4093, D=4096, W=4, dtype="bf16", silu=True, bias=True,
             state=False, positions=True),
        # a decode step of 256 sequences
        dict(name="ssm_token", op="ssm_step", B=256, T=1, D=4096, N=16, G=1, dtype="bf16", gate=True, skip=True,
             bias=True, softplus=True, state=True, positions=False),
        # the prefill's tokens through a 4096-wide layer
        dict(name="ssm_prefill", op="ssm", B=8, T=8192, D=4096, N=16, G=1, dtype="bf16", gate=True, skip=True,
             bias=True, softplus=True, state=False, positions=False),
        # one long row of packed documents through 1024 channels
        dict(name="ssm_long", op="ssm", B=1, T=65536, D=1024, N=16, G=1, dtype="bf16", gate=True, skip=True,
             bias=True, softplus=True, state=True, positions=True),
        # a short ragged fp32 call: two groups of channels, steps given as they are
        dict(name="ssm_short", op="ssm", B=3, T=251, D=208, N=8, G=2, dtype="f32", gate=False, skip=True,
             bias=False, softplus=False, state=True, positions=False),
        # a training step's gradients
        dict(name="ssm_train", op="ssm_bwd", B=4, T=4096, D=2048, N=16, G=1, dtype="bf16", gate=True, skip=True,
             bias=True, softplus=True, state=False, positions=True),
        # a decode step: one row for each of 256 sequences
        dict(name="block_step", op="block", B=256, T=1, D=4096, dtype="bf16", residual="bf16", post=True,
             gate="row", weights=True, center=False),
        # the prefill's rows, a gate for each sequence
        dict(name="block_prefill", op="block", B=8, T=8192, D=2048, dtype="bf16", residual="bf16", post=True,
             gate="batch", weights=True, center=False),
        # a training step's gradients, ragged length, the residual stream in fp32, centred norms
        dict(name="block_train", op="block_bwd", B=4, T=4093, D=2048, dtype="bf16", residual="f32", post=True,
             gate="row", weights=True, center=True),
    ]


MOST = 1 << 27       # entries of a drawn case's main tensor: half the largest listed one's
MOST_STATE = 1 << 29  # state entries a drawn gradient passes through: the listed one's


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_bwd", "conv_step", "ssm", "ssm", "ssm", "ssm_bwd", "ssm_bwd", "ssm_step",
                     "block", "block", "block_bwd"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    step = op.endswith("step")
    D = 16 * _logint(rng, 1, 512)
    T = 1 if step or rng.random() < 0.1 else _logint(rng, 1, 65536)
    if op.startswith("conv"):
        B = _logint(rng, 1, 512) if step else _logint(rng, 1, max(1, min(64, MOST // (T * D))))
        T = max(1, min(T, MOST // (B * D)))
        return dict(op=op, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.7,
                    bias=rng.random() < 0.6, state=step or rng.random() < 0.5,
                    positions=not step and rng.random() < 0.5)
    if op.startswith("block"):
        D = min(D, 8192)
        B = _logint(rng, 1, max(1, min(256, MOST // (T * D))))
        T = max(1, min(T, MOST // (B * D)))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, residual=rng.choice([dtype, "f32"]),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "row", "batch"]),
                    weights=rng.random() < 0.7, center=rng.random() < 0.4)
    N = rng.choice([8, 16, 16, 16, 32, 64])
    most = (MOST_STATE if op == "ssm_bwd" else 16 * MOST) // N
    D = min(D, 4096)
    B = _logint(rng, 1, 512 if step else max(1, min(64, most // (T * D))))
    T = max(1, min(T, most // (B * D)))
    return dict(op=op, B=B, T=T, D=D, N=N, G=rng.choice([1, 1, 2]), dtype=dtype, gate=rng.random() < 0.7,
                skip=rng.random() < 0.7, bias=rng.random() < 0.7, softplus=rng.random() < 0.8,
                state=step or rng.random() < 0.5, positions=not step and rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    return (x * scale if scale != 1.0 else x).to(dtype)


def _positions(g, B, T, continues):
    """Each token's place in its document: documents of about 512 tokens one after
    another, the first one begun 7000 tokens earlier where a state comes in."""
    start = torch.rand(B, T, generator=g, device=DEV) < 1.0 / 512
    t = torch.arange(T, device=DEV).expand(B, T)
    first = torch.where(start, t, torch.full_like(t, -7000 if continues else 0))
    return (t - first.cummax(1).values).to(torch.int32)


def prepare(case, seed):
    """Activations as projections leave them (slices of packed rows), step sizes between
    1e-3 and 1e-1 around their bias, decay rates between 0.5 and 1.5 N."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    B, T, D = case["B"], case["T"], case["D"]
    s = dict(case=case)
    if op.startswith("block"):
        s["o"] = _randn(g, B, T, D, dtype=dt, scale=2.0)
        s["h"] = _randn(g, B, T, D, dtype=TYPES[case["residual"]], scale=3.0)
        s["w_post"] = 1.0 + _randn(g, D, scale=0.1) if case["weights"] and case["post"] else None
        s["w_pre"] = 1.0 + _randn(g, D, scale=0.1) if case["weights"] else None
        s["gate"] = {"none": None, "row": _randn(g, D, scale=0.5), "batch": _randn(g, B, D, scale=0.5)}[case["gate"]]
        if op == "block_bwd":  # h: the stream the forward pass left
            s["dy"] = _randn(g, B, T, D, dtype=dt)
            s["dh"] = _randn(g, B, T, D, dtype=TYPES[case["residual"]])
        return s
    s["positions"] = _positions(g, B, T, case["state"]) if case["positions"] else None
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = _randn(g, B, T, 2 * D, dtype=dt)[..., :D]
        s["w"] = _randn(g, D, W, scale=0.5)
        s["bias"] = _randn(g, D, scale=0.5) if case["bias"] else None
        s["state"] = _randn(g, B, W - 1, D, dtype=dt) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = _randn(g, B, T, D, dtype=dt)
            s["dstate"] = _randn(g, B, W - 1, D, dtype=dt) if case["state"] else None
        if op == "conv_step":
            s["x"], s["positions"] = s["x"][:, 0], None
            s["state1"] = torch.empty_like(s["state"])
        return s
    N, G = case["N"], case["G"]
    s["x"] = _randn(g, B, T, D, dtype=dt, scale=0.7)
    usual = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(D, generator=g, device=DEV))
    if case["softplus"]:
        before = torch.log(torch.expm1(usual))
        s["dt"] = _randn(g, B, T, D, dtype=dt, scale=0.5)
        s["bias"] = before if case["bias"] else None
        if not case["bias"]:
            s["dt"] = (s["dt"] + before).to(dt)
    else:
        s["dt"] = (usual * (0.5 + torch.rand(B, T, D, generator=g, device=DEV))).to(dt)
        s["bias"] = 0.01 * torch.rand(D, generator=g, device=DEV) if case["bias"] else None
    s["A"] = -(torch.arange(1, N + 1, device=DEV) * (0.5 + torch.rand(D, N, generator=g, device=DEV)))
    row = _randn(g, B, T, RANK + 2 * G * N, dtype=dt)
    s["b"] = row[..., RANK:RANK + G * N].view(B, T, G, N)
    s["c"] = row[..., RANK + G * N:].view(B, T, G, N)
    s["skip"] = 1.0 + _randn(g, D, scale=0.1) if case["skip"] else None
    s["gate"] = _randn(g, B, T, 2 * D, dtype=dt)[..., D:] if case["gate"] else None
    s["h0"] = _randn(g, B, D, N) if case["state"] else None
    if op == "ssm_bwd":
        s["dy"] = _randn(g, B, T, D, dtype=dt)
        s["dhT"] = _randn(g, B, D, N) if case["state"] else None
    if op == "ssm_step":
        for n in ("x", "dt", "b", "c", "gate"):
            s[n] = None if s[n] is None else s[n][:, 0]
        s["h1"] = torch.empty_like(s["h0"])
    return s


# ---- plain forms ---------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _taps(s, x, T):
    """The row of history and tokens in 32 bits, and for each tap the tokens it counts at."""
    W = s["case"]["W"]
    before = s["state"]
    if before is None:
        before = torch.zeros(x.shape[0], W - 1, x.shape[2], device=DEV, dtype=x.dtype)
    row = torch.cat((before, x), 1)
    p = s["positions"]
    use = [None if p is None or j == W - 1 else (p >= W - 1 - j).float().unsqueeze(-1) for j in range(W)]
    return row, use


def _conv_u(s, row, use, T):
    u = None
    for j, m in enumerate(use):
        v = row[:, j:j + T].float() * s["w"][:, j]
        v = v if m is None else v * m
        u = v if u is None else u.add_(v)
    return u if s["bias"] is None else u.add_(s["bias"])


def _conv_plain(s):
    c = s["case"]
    T, W = c["T"], c["W"]
    x = s["x"] if c["op"] == "conv" else s["x"].unsqueeze(1)
    row, use = _taps(s, x, T)
    u = _conv_u(s, row, use, T)
    if c["silu"]:
        u = u * _sigmoid(u)
    y = u.to(x.dtype)
    return (y if c["op"] == "conv" else y[:, 0]), row[:, T:T + W - 1].clone()


def _conv_bwd_plain(s):
    c = s["case"]
    T, W = c["T"], c["W"]
    row, use = _taps(s, s["x"], T)
    du = s["dy"].float()
    if c["silu"]:
        u = _conv_u(s, row, use, T)
        sg = _sigmoid(u)
        du = du * (sg * (1.0 + u * (1.0 - sg)))
    d_row = torch.zeros(row.shape, device=DEV)
    if s["dstate"] is not None:
        d_row[:, T:] += s["dstate"].float()
    dw = []
    for j, m in enumerate(use):
        g = du if m is None else du * m
        dw.append((g * row[:, j:j + T].float()).sum((0, 1)))
        d_row[:, j:j + T] += g * s["w"][:, j]
    out = [d_row[:, W - 1:].to(s["x"].dtype), torch.stack(dw, 1)]
    if s["bias"] is not None:
        out.append(du.sum((0, 1)))
    if s["state"] is not None:
        out.append(d_row[:, :W - 1].to(s["x"].dtype))
    return tuple(out)


def _delta(s, dt):
    v = dt.float()
    v = v if s["bias"] is None else v + s["bias"]
    if not s["case"]["softplus"]:
        return v
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _heads(v, D):
    """[B, T, G, N] to [B, T, D, N] by repetition over a group's channels, in 32 bits."""
    B, T, G, N = v.shape
    return v.float().unsqueeze(3).expand(B, T, G, D // G, N).reshape(B, T, D, N)


def _span(c):
    """Tokens whose [B, tokens, D, N] products are held at once: a power of two."""
    n = 1
    while n < 32 and 2 * n * c["B"] * c["D"] * c["N"] <= 1 << 27:
        n *= 2
    return n


def _doubling(a, v):
    """Every h_t = a_t h_(t-1) + v_t along dim 1 (h before the first 0), in place, by
    composing spans of 1, 2, 4, ... tokens."""
    step = 1
    while step < a.shape[1]:
        v[:, step:] += a[:, step:] * v[:, :-step]
        a[:, step:] *= a[:, :-step].clone()
        step *= 2
    return v


def _states(s, t0, t1, h):
    """(delta, decays, states) of tokens t0 .. t1 - 1 from the state h before them."""
    D = s["case"]["D"]
    part = lambda n: s[n][:, t0:t1]
    d = _delta(s, part("dt"))
    a = torch.exp(d.unsqueeze(-1) * s["A"])
    if s["positions"] is not None:
        a *= (part("positions") != 0).float()[:, :, None, None]
    v = (d * part("x").float()).unsqueeze(-1) * _heads(part("b"), D)
    v[:, 0] += a[:, 0] * h
    return d, a, _doubling(a.clone(), v)


def _ssm_y(s, t0, t1, hs):
    part = lambda n: s[n][:, t0:t1]
    u = (hs * _heads(part("c"), s["case"]["D"])).sum(-1)
    return u if s["skip"] is None else u + s["skip"] * part("x").float()


def _ssm_plain(s):
    c = s["case"]
    B, T, D, N = c["B"], c["T"], c["D"], c["N"]
    h = s["h0"] if s["h0"] is not None else torch.zeros(B, D, N, device=DEV)
    y = torch.empty(B, T, D, device=DEV, dtype=s["x"].dtype)
    span = _span(c)
    for t0 in range(0, T, span):
        t1 = min(T, t0 + span)
        hs = _states(s, t0, t1, h)[2]
        u = _ssm_y(s, t0, t1, hs)
        if s["gate"] is not None:
            g = s["gate"][:, t0:t1].float()
            u = u * (g * _sigmoid(g))
        y[:, t0:t1] = u.to(y.dtype)
        h = hs[:, -1].clone()
    return y, h


def _ssm_step_plain(s):
    c = s["case"]
    one = dict(s, case=c, positions=None, **{n: None if s[n] is None else s[n].unsqueeze(1)
                                             for n in ("x", "dt", "b", "c", "gate")})
    y, h = _ssm_plain(one)
    return y[:, 0], h


def _ssm_bwd_plain(s):
    c = s["case"]
    B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
    dt = s["x"].dtype
    span = _span(c)
    starts = list(range(0, T, span))
    h = s["h0"] if s["h0"] is not None else torch.zeros(B, D, N, device=DEV)
    enter = []
    for t0 in starts:
        enter.append(h)
        h = _states(s, t0, min(T, t0 + span), h)[2][:, -1].clone()
    dx, ddt = (torch.empty(B, T, D, device=DEV, dtype=dt) for _ in range(2))
    dgate = torch.empty(B, T, D, device=DEV, dtype=dt) if s["gate"] is not None else None
    db, dc = (torch.empty(B, T, G, N, device=DEV, dtype=dt) for _ in range(2))
    dA, dskip, dbias = torch.zeros(D, N, device=DEV), torch.zeros(D, device=DEV), torch.zeros(D, device=DEV)
    carry = s["dhT"] if s["dhT"] is not None else torch.zeros(B, D, N, device=DEV)
    for t0, h in zip(reversed(starts), reversed(enter)):
        t1 = min(T, t0 + span)
        part = lambda n: s[n][:, t0:t1]
        d, a, hs = _states(s, t0, t1, h)
        x, du = part("x").float(), part("dy").float()
        if dgate is not None:
            g = part("gate").float()
            sg = _sigmoid(g)
            dgate[:, t0:t1] = (du * _ssm_y(s, t0, t1, hs) * (sg * (1.0 + g * (1.0 - sg)))).to(dt)
            du = du * (g * sg)
        dc[:, t0:t1] = (hs * du.unsqueeze(-1)).view(B, t1 - t0, G, D // G, N).sum(3).to(dt)
        dh = _heads(part("c"), D) * du.unsqueeze(-1)
        dh[:, -1] += carry
        later = torch.cat((torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)), 1)  # the decay behind each token
        dh = _doubling(later, dh.flip(1)).flip(1)
        carry = a[:, 0] * dh[:, 0]
        b = _heads(part("b"), D)
        along = (dh * b).sum(-1)
        db[:, t0:t1] = (dh * (d * x).unsqueeze(-1)).view(B, t1 - t0, G, D // G, N).sum(3).to(dt)
        q = torch.cat((h.unsqueeze(1), hs[:, :-1]), 1) * a * dh
        dA += (q * d.unsqueeze(-1)).sum((0, 1))
        dd = along * x + (q * s["A"]).sum(-1)
        if c["softplus"]:
            v = part("dt").float()
            dd = dd * _sigmoid(v if s["bias"] is None else v + s["bias"])
        dbias += dd.sum((0, 1))
        ddt[:, t0:t1] = dd.to(dt)
        v = along * d
        if s["skip"] is not None:
            v = v + s["skip"] * du
            dskip += (du * x).sum((0, 1))
        dx[:, t0:t1] = v.to(dt)
    out = [dx, ddt, dA, db, dc, dskip if s["skip"] is not None else None, dgate,
           dbias if s["bias"] is not None else None, carry]
    return tuple(t for t in out if t is not None)


def _norm(x, center):
    if center:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_bwd(dn, n, r, center):
    v = dn - n * (dn * n).mean(-1, keepdim=True)
    if center:
        v = v - dn.mean(-1, keepdim=True)
    return r * v


ALPHA, BETA = 0.8, 1.25  # the branch's and the residual's scale


def _block_gate(s):
    g = s["gate"]
    return None if g is None else (g if g.dim() == 1 else g.unsqueeze(1))


def _times(v, w):
    return v if w is None else v * w


def _block_plain(s):
    c = s["case"]
    p = s["o"].float()
    if c["post"]:
        p = _times(_norm(p, c["center"])[0], s["w_post"])
    h = BETA * s["h"].float() + ALPHA * _times(p, _block_gate(s))
    y = _times(_norm(h, c["center"])[0], s["w_pre"])
    return h.to(s["h"].dtype), y.to(s["o"].dtype)


def _block_bwd_plain(s):
    c, gate = s["case"], _block_gate(s)
    n, r = _norm(s["h"].float(), c["center"])
    dy = s["dy"].float()
    dw_pre = (dy * n).sum((0, 1))
    dt = s["dh"].float() + _norm_bwd(_times(dy, s["w_pre"]), n, r, c["center"])
    out = [(BETA * dt).to(s["h"].dtype)]
    p, r = s["o"].float(), None
    if c["post"]:
        p, r = _norm(p, c["center"])
    dt = ALPHA * dt
    if gate is not None:
        dgate = (dt * _times(p, s["w_post"])).sum((0, 1) if gate.dim() == 1 else 1)
        dt = dt * gate
    if c["post"]:
        dw_post = (dt * p).sum((0, 1))
        dt = _norm_bwd(_times(dt, s["w_post"]), p, r, c["center"])
    out.insert(0, dt.to(s["o"].dtype))
    if s["w_post"] is not None:
        out.append(dw_post)
    if gate is not None:
        out.append(dgate)
    if s["w_pre"] is not None:
        out.append(dw_pre)
    return tuple(out)


# ---- one pass ------------------------------------------------------------------------

PLAIN = dict(conv=_conv_plain, conv_step=_conv_plain, conv_bwd=_conv_bwd_plain, ssm=_ssm_plain,
             ssm_step=_ssm_step_plain, ssm_bwd=_ssm_bwd_plain, block=_block_plain, block_bwd=_block_bwd_plain)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](s)
    import retnet_retention_gb300 as la
    if op.startswith("conv"):
        opts = dict(bias=s["bias"], silu=c["silu"])
        if op == "conv_step":
            y = la.short_conv_step(s["x"], s["w"], s["state"], state_out=s["state1"], **opts)
            return y, s["state1"]
        opts.update(state=s["state"], positions=s["positions"])
        if op == "conv":
            return la.short_conv_fwd(s["x"], s["w"], **opts)
        out = la.short_conv_bwd(s["x"], s["w"], s["dy"], dstate_T=s["dstate"],
                                state_grads=s["state"] is not None, **opts)
        return tuple(t for t in out if t is not None)
    if op.startswith("ssm"):
        opts = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["bias"], softplus=c["softplus"])
        if op == "ssm_step":
            y = la.ssm_step(s["x"], s["dt"], s["A"], s["b"], s["c"], s["h0"], h_out=s["h1"], **opts)
            return y, s["h1"]
        opts.update(h0=s["h0"], positions=s["positions"])
        if op == "ssm":
            return la.ssm_fwd(s["x"], s["dt"], s["A"], s["b"], s["c"], **opts)
        out = la.ssm_bwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["dy"], dh_T=s["dhT"], **opts)
        return tuple(t for t in out if t is not None)
    opts = dict(post_norm=c["post"], post_weight=s["w_post"], gate=s["gate"], scale=ALPHA, residual_scale=BETA,
                pre_weight=s["w_pre"], center=c["center"], eps=EPS)
    if op == "block":
        return la.block_norm_fwd(s["o"], s["h"], **opts)
    out = la.block_norm_bwd(s["o"], s["h"], s["dy"], s["dh"], **opts)
    return tuple(t for t in out if t is not None)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    B, T, D = case["B"], case["T"], case["D"]
    n = B * T * D
    if op.startswith("block"):
        r = 2 if case["residual"] == "bf16" else 4
        small = 4 * D * (2 * case["weights"] + (case["gate"] == "row")) + 4 * B * D * (case["gate"] == "batch")
        if op == "block":
            return dict(bytes=n * (2 * e + 2 * r) + small, flops=16 * n)
        return dict(bytes=n * (3 * e + 3 * r) + 2 * small, flops=40 * n)
    pos = 4 * B * T if case["positions"] else 0
    if op.startswith("conv"):
        W = case["W"]
        weights, state = 4 * D * (W + case["bias"]), (W - 1) * B * D * e
        if op == "conv_bwd":
            return dict(bytes=3 * n * e + 2 * weights + pos + 3 * state * case["state"], flops=n * (6 * W + 12))
        return dict(bytes=2 * n * e + weights + pos + state * (1 + case["state"]), flops=n * (2 * W + 6))
    N, G = case["N"], case["G"]
    weights, state = 4 * D * (N + case["skip"] + case["bias"]), 4 * B * D * N
    shared = 2 * B * T * G * N * e
    if op == "ssm_bwd":
        return dict(bytes=n * e * (5 + 2 * case["gate"]) + 2 * shared + 2 * weights + pos
                    + state * (3 if case["state"] else 1), flops=n * (24 * N + 40))
    return dict(bytes=n * e * (3 + case["gate"]) + shared + weights + pos + state * (1 + case["state"]),
                flops=n * (7 * N + 20))


# ---- the definition in 64 bits -------------------------------------------------------

MOST_EXACT = 1 << 32  # state entries walked token by token
MOST_TOKENS = 1 << 17


def exact(case, seed):
    op = case["op"]
    if op.startswith("ssm") and (case["B"] * case["T"] * case["D"] * case["N"] > MOST_EXACT
                                 or case["T"] > MOST_TOKENS):
        return None
    s = prepare(case, seed)
    wide = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for n, t in s.items()}
    if op.startswith("ssm"):
        return _ssm_exact(case, wide)
    if op.startswith("conv"):
        return _conv_exact(case, wide)
    return _block_exact(case, wide)


def _conv_exact(case, s):
    """As a product with the windows of W tokens; gradients by differentiation of that."""
    W, T, x = case["W"], case["T"], s["x"]
    if case["op"] == "conv_step":
        x = x.unsqueeze(1)
    before = s["state"]
    if before is None:
        before = torch.zeros(x.shape[0], W - 1, case["D"], device=DEV, dtype=torch.float64)
    grads = case["op"] == "conv_bwd"
    bias = s["bias"] if s["bias"] is not None else torch.zeros(case["D"], device=DEV, dtype=torch.float64)
    leaves = [x, s["w"], bias, before]
    if grads:
        leaves = [t.clone().requires_grad_() for t in leaves]
    x, w, bias, before = leaves
    row = torch.cat((before, x), 1)
    if s["positions"] is None:
        u = torch.nn.functional.conv1d(row.transpose(1, 2), w.unsqueeze(1), groups=case["D"]).transpose(1, 2)
    else:
        back = torch.arange(W - 1, -1, -1, device=DEV)
        keep = (s["positions"].unsqueeze(-1) >= back).double()
        u = sum(row[:, j:j + T] * keep[:, :, j:j + 1] * w[:, j] for j in range(W))
    u = u + bias
    y = u * torch.sigmoid(u) if case["silu"] else u
    last = row[:, T:]
    if not grads:
        return (y[:, 0] if case["op"] == "conv_step" else y), last
    loss = (y * s["dy"]).sum()
    if s["dstate"] is not None:
        loss = loss + (last * s["dstate"]).sum()
    dx, dw, db, d0 = torch.autograd.grad(loss, leaves)
    out = [dx, dw, db if s["bias"] is not None else None, d0 if s["state"] is not None else None]
    return tuple(t for t in out if t is not None)


def _ssm_exact(case, s):
    """Token by token; the gradients by the reversed walk over stored states."""
    B, T, D, N, G = (case[n] for n in "BTDNG")
    step = case["op"] == "ssm_step"
    seq = {n: s[n].unsqueeze(1) if step and s[n] is not None else s[n] for n in ("x", "dt", "b", "c", "gate")}
    x, raw = seq["x"], seq["dt"]
    if s["bias"] is not None:
        raw = raw + s["bias"]
    d = torch.logaddexp(raw, torch.zeros_like(raw)) if case["softplus"] else raw
    A = s["A"].view(G, D // G, N)
    grouped = lambda v: v.reshape(B, G, D // G)
    zero = torch.zeros(B, G, D // G, N, device=DEV, dtype=torch.float64)
    h = zero if s["h0"] is None else s["h0"].view(B, G, D // G, N)
    keep = None if s["positions"] is None else (s["positions"] != 0).double()
    act = 1.0 if seq["gate"] is None else seq["gate"] * torch.sigmoid(seq["gate"])
    grads = case["op"] == "ssm_bwd"
    hs = [h]
    u = torch.empty(B, T, D, device=DEV, dtype=torch.float64)

    def decay(t):
        a = torch.exp(grouped(d[:, t]).unsqueeze(-1) * A)
        return a if keep is None else a * keep[:, t].view(B, 1, 1, 1)

    for t in range(T):
        h = decay(t) * h + grouped(d[:, t] * x[:, t]).unsqueeze(-1) * seq["b"][:, t].unsqueeze(2)
        u[:, t] = torch.einsum("bgdn,bgn->bgd", h, seq["c"][:, t]).reshape(B, D)
        if grads:
            hs.append(h)
    if s["skip"] is not None:
        u += s["skip"] * x
    if not grads:
        y = u * act
        return (y[:, 0] if step else y), h.reshape(B, D, N)
    du = s["dy"] * act
    dgate = None
    if seq["gate"] is not None:
        sg = torch.sigmoid(seq["gate"])
        dgate = s["dy"] * u * (sg + act * (1.0 - sg))
    g = zero if s["dhT"] is None else s["dhT"].view(B, G, D // G, N)
    dx, dd = torch.empty_like(x), torch.empty_like(x)
    db, dc = torch.empty_like(s["b"]), torch.empty_like(s["c"])
    dA = torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        dut = grouped(du[:, t])
        g = g + dut.unsqueeze(-1) * s["c"][:, t].unsqueeze(2)
        dc[:, t] = torch.einsum("bgdn,bgd->bgn", hs.pop(), dut)
        db[:, t] = torch.einsum("bgdn,bgd->bgn", g, grouped(d[:, t] * x[:, t]))
        into = torch.einsum("bgdn,bgn->bgd", g, s["b"][:, t]).reshape(B, D)
        g = g * decay(t)
        q = g * hs[-1]
        dA += torch.einsum("bgdn,bgd->gdn", q, grouped(d[:, t]))
        dx[:, t] = into * d[:, t]
        dd[:, t] = into * x[:, t] + torch.einsum("bgdn,gdn->bgd", q, A).reshape(B, D)
    if case["softplus"]:
        dd = dd * torch.sigmoid(raw)
    dskip = None
    if s["skip"] is not None:
        dskip = (du * x).sum((0, 1))
        dx = dx + s["skip"] * du
    out = [dx, dd, dA.reshape(D, N), db, dc, dskip, dgate, dd.sum((0, 1)) if s["bias"] is not None else None,
           g.reshape(B, D, N)]
    return tuple(t for t in out if t is not None)


def _block_exact(case, s):
    """The definition; gradients by differentiation of it, a sequence at a time."""

    def norm(v):
        if case["center"]:
            v = v - v.sum(-1, keepdim=True) / case["D"]
        return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / case["D"] + EPS)

    one = torch.ones(case["D"], device=DEV, dtype=torch.float64)
    w_post, w_pre = (one if s[n] is None else s[n] for n in ("w_post", "w_pre"))
    gates = one.expand(case["B"], -1) if s["gate"] is None else s["gate"].expand(case["B"], -1)
    parts = []
    for i in range(case["B"]):
        branch = lambda o, w, g: ALPHA * g * (norm(o) * w if case["post"] else o)
        o, h = s["o"][i], s["h"][i]
        if case["op"] == "block":
            h = BETA * h + branch(o, w_post, gates[i])
            parts.append((h, norm(h) * w_pre))
            continue
        o, h, wp, wq, g = (t.clone().requires_grad_() for t in (o, h, w_post, w_pre, gates[i]))
        into, dw_pre = torch.autograd.grad((norm(h) * wq * s["dy"][i]).sum(), (h, wq))
        dh = s["dh"][i] + into
        d_o, dw_post, dg = torch.autograd.grad((branch(o, wp, g) * dh).sum(), (o, wp, g), allow_unused=True)
        parts.append((d_o, BETA * dh, dw_post, dg, dw_pre))
    cols = list(zip(*parts))
    if case["op"] == "block":
        return tuple(torch.stack(v) for v in cols)
    out = [torch.stack(cols[0]), torch.stack(cols[1])]
    if s["w_post"] is not None:
        out.append(torch.stack(cols[2]).sum(0))
    if s["gate"] is not None:
        dg = torch.stack(cols[3])
        out.append(dg.sum(0) if s["gate"].dim() == 1 else dg)
    if s["w_pre"] is not None:
        out.append(torch.stack(cols[4]).sum(0))
    return tuple(out)
