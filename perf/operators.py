"""Cases of the layer operators around retention: queries and keys normed and
rotated into the layout retention reads (qk_rotate), the per-head norm and gate
of its output (head_gate), and the per-channel gated recurrence (scan), each
forward, backward and for single tokens.

`run` computes a case with elementary torch operations, or, with `own` set,
through retnet_retention_gb300.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    """Sizes: the repository's workloads (8 x 8192 tokens of 16 heads, one sequence of
    65,536 tokens, 256 decoding sequences of 32 heads, 4 x 4096 tokens), their widths
    (64, 128, 256), and ragged ones."""
    return [
        # a decode step of 256 sequences, each at its own position, from packed projections
        dict(name="qk_step", op="qk", B=256, T=1, H=32, HK=32, d=128, rot=128, pairs="adjacent",
             norm=True, weight=True, dtype="bf16", positions=True),
        # the multi-scale retention prefill: all heads of 8 x 8192 tokens
        dict(name="qk_prefill", op="qk", B=8, T=8192, H=16, HK=16, d=128, rot=128, pairs="adjacent",
             norm=True, weight=True, dtype="bf16", positions=False),
        # ragged, fp32, shared keys, a partial rotation of split halves
        dict(name="qk_ragged", op="qk", B=3, T=1021, H=6, HK=2, d=80, rot=32, pairs="halves",
             norm=True, weight=False, dtype="f32", positions=True),
        # a training step's gradients at the linear-attention length
        dict(name="qk_train", op="qk_bwd", B=4, T=4096, H=16, HK=16, d=128, rot=128, pairs="halves",
             norm=True, weight=True, dtype="bf16", positions=False),
        # the smallest call: one sequence decoding one token through 8 heads
        dict(name="gate_step", op="gate", B=1, T=1, H=8, d=64, dtype="bf16", gate=True, weight=True,
             center=False, source="heads"),
        # the multi-scale retention's output, 256 wide, into the layer's row
        dict(name="gate_prefill", op="gate", B=8, T=8192, H=16, d=256, dtype="bf16", gate=True,
             weight=False, center=False, source="heads"),
        # gradients of a centred norm with its weights, ragged length
        dict(name="gate_train", op="gate_bwd", B=4, T=4093, H=16, d=128, dtype="bf16", gate=True,
             weight=True, center=True, source="heads"),
        # one long sequence through 1024 channels, documents packed one after another
        dict(name="scan_long", op="scan", B=1, T=65536, D=1024, dtype="bf16", state=True, restarts=True),
        # the prefill's tokens through a 4096-wide layer
        dict(name="scan_wide", op="scan", B=8, T=8192, D=4096, dtype="bf16", state=False, restarts=False),
        # a short ragged fp32 call
        dict(name="scan_short", op="scan", B=3, T=251, D=208, dtype="f32", state=True, restarts=False),
        # a training step's gradients
        dict(name="scan_train", op="scan_bwd", B=4, T=4096, D=2048, dtype="bf16", state=True, restarts=True),
        # a decode step of 256 sequences through 4096 channels
        dict(name="scan_token", op="step", B=256, T=1, D=4096, dtype="bf16", state=True, restarts=False),
    ]


MOST = 1 << 27  # elements of a drawn case's main tensor: half the largest listed one's


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["qk", "qk", "qk_bwd", "gate", "gate", "gate_bwd", "scan", "scan", "scan_bwd", "step"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op == "step":
        return dict(op=op, B=_logint(rng, 1, 512), T=1, D=16 * _logint(rng, 1, 512), dtype=dtype,
                    state=True, restarts=rng.random() < 0.5)
    T = 1 if (op in ("qk", "gate") and rng.random() < 0.3) else _logint(rng, 1, 65536)
    if op.startswith("scan"):
        D = 16 * _logint(rng, 1, 512)
        B = _logint(rng, 1, max(1, min(64, MOST // (T * D))))
        return dict(op=op, B=B, T=max(1, min(T, MOST // (B * D))), D=D, dtype=dtype,
                    state=rng.random() < 0.5, restarts=rng.random() < 0.5)
    d = 16 * rng.randint(1, 16)
    H = _logint(rng, 1, 32)
    T = max(1, min(T, MOST // (H * d * 2)))
    B = _logint(rng, 1, max(1, min(256, MOST // (T * H * d * 2))))
    if op.startswith("qk"):
        return dict(op=op, B=B, T=T, H=H, HK=rng.choice([H, H, max(1, H // 4), 1]), d=d,
                    rot=rng.choice([d, 16 * rng.randint(0, d // 16)]),
                    pairs=rng.choice(["adjacent", "halves"]), norm=rng.random() < 0.8,
                    weight=rng.random() < 0.6, dtype=dtype, positions=rng.random() < 0.5)
    return dict(op=op, B=B, T=T, H=H, d=d, dtype=dtype, gate=rng.random() < 0.8,
                weight=rng.random() < 0.6, center=rng.random() < 0.4,
                source=rng.choice(["heads", "heads", "rows"]))


# ---- inputs --------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    return (x * scale if scale != 1.0 else x).to(dtype)


def prepare(case, seed):
    """Projections as the layer's matrix product leaves them ([B, T, heads, d], q, k and v
    side by side in one row), retention outputs per head, decays between 1e-4 and 1 in
    the log, -inf where a document starts."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    B, T = case["B"], case["T"]
    s = dict(case=case)
    if op.startswith("qk"):
        H, HK, d, rot = case["H"], case["HK"], case["d"], case["rot"]
        packed = _randn(g, B, T, H + 2 * HK, d, dtype=dt)
        s["q"], s["k"] = packed[:, :, :H], packed[:, :, H:H + HK]
        weighted = case["norm"] and case["weight"]
        s["wq"] = 1.0 + _randn(g, d, scale=0.1) if weighted else None
        s["wk"] = 1.0 + _randn(g, d, scale=0.1) if weighted else None
        s["inv_freq"] = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
        s["positions"] = None
        if case["positions"]:
            start = torch.randint(0, 65536, (B, 1), generator=g, device=DEV, dtype=torch.int32)
            s["positions"] = start + torch.arange(T, device=DEV, dtype=torch.int32)
        if op == "qk_bwd":
            s["dyq"] = _randn(g, B, H, T, d, dtype=dt)
            s["dyk"] = _randn(g, B, HK, T, d, dtype=dt)
    elif op.startswith("gate"):
        H, d = case["H"], case["d"]
        if case["source"] == "heads":
            s["o"] = _randn(g, B, H, T, d, dtype=dt, scale=3.0)
        else:  # the recurrence's [B, T, channels], taken as heads
            s["o"] = _randn(g, B, T, H, d, dtype=dt, scale=3.0).permute(0, 2, 1, 3)
        s["g"] = _randn(g, B, T, H, d, dtype=dt, scale=1.5) if case["gate"] else None
        s["w"] = 1.0 + _randn(g, H, d, scale=0.1) if case["weight"] else None
        if op == "gate_bwd":
            s["dy"] = _randn(g, B, T, H, d, dtype=dt)
    else:
        D = case["D"]
        shape = (B, D) if op == "step" else (B, T, D)
        u = torch.rand(*shape, generator=g, device=DEV, dtype=torch.float32)
        la = -torch.exp(u * math.log(1e4) - math.log(1e4))
        if case["restarts"]:
            n = shape[0] if op == "step" else T
            start = torch.rand(n, generator=g, device=DEV) < 1.0 / 512
            la[start if op == "step" else (slice(None), start)] = float("-inf")
        s["log_a"] = la
        s["x"] = _randn(g, *shape, dtype=dt)
        s["h0"] = _randn(g, B, D, scale=2.0) if case["state"] else None
        if op == "step":  # where the step leaves its state: a pass starts from the same one
            s["h1"] = torch.empty_like(s["h0"])
        if op == "scan_bwd":  # h: the forward's output, dh: its gradient; x is not read
            s["h"] = _scan_plain(s["x"], la, s["h0"])[0]
            s["dh"] = s.pop("x").neg_()
            s["dhT"] = _randn(g, B, D) if case["state"] else None
    return s


# ---- plain forms ---------------------------------------------------------------------

def _angles(s, T):
    """cos and sin [B or 1, T, 1, rot/2]; the angle in 64 bits, far positions keep it."""
    p = s["positions"]
    p = torch.arange(T, device=DEV).unsqueeze(0) if p is None else p
    f = torch.tensor(s["inv_freq"], device=DEV, dtype=torch.float64)
    a = (p.double().unsqueeze(-1) * f).unsqueeze(2)
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, pairs):
    if rot == 0:
        return x
    r, rest = x[..., :rot], x[..., rot:]
    if pairs == "adjacent":
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, rest), -1)


def _qk_plain(s):
    c = s["case"]
    cos, sin = _angles(s, c["T"])
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        dt, x = x.dtype, x.float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            x = x if w is None else x * w
        out.append(_rotate(x, cos, sin, c["rot"], c["pairs"]).transpose(1, 2).contiguous().to(dt))
    return tuple(out)


def _qk_bwd_plain(s):
    c = s["case"]
    cos, sin = _angles(s, c["T"])
    dx, dw = [], []
    for x, w, dy in ((s["q"], s["wq"], s["dyq"]), (s["k"], s["wk"], s["dyk"])):
        dt, x = x.dtype, x.float()
        g = _rotate(dy.float().transpose(1, 2), cos, -sin, c["rot"], c["pairs"])
        if c["norm"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            if w is not None:
                dw.append((g * x * r).sum((0, 1, 2)))
                g = g * w
            g = r * (g - x * (r * r * (g * x).mean(-1, keepdim=True)))
        dx.append(g.to(dt))
    return tuple(dx + dw)


def _gate_plain(s):
    c, o = s["case"], s["o"].float()
    if c["center"]:
        o = o - o.mean(-1, keepdim=True)
    u = (o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)).transpose(1, 2)
    if s["w"] is not None:
        u = u * s["w"]
    if s["g"] is not None:
        g = s["g"].float()
        u = u * (g / (1.0 + torch.exp(-g)))
    return (u.contiguous().to(s["o"].dtype),)


def _gate_bwd_plain(s):
    c, dt = s["case"], s["o"].dtype
    o = s["o"].float()
    if c["center"]:
        o = o - o.mean(-1, keepdim=True)
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS).transpose(1, 2)
    n = o.transpose(1, 2) * r
    du, out = s["dy"].float(), []
    if s["g"] is not None:
        g = s["g"].float()
        sg = 1.0 / (1.0 + torch.exp(-g))
        u = n if s["w"] is None else n * s["w"]
        out.append((du * u * (sg * (1.0 + g * (1.0 - sg)))).to(dt))
        du = du * (g * sg)
    if s["w"] is not None:
        out.append((du * n).sum((0, 1)))
        du = du * s["w"]
    m = (du * n).mean(-1, keepdim=True)
    if c["center"]:
        du = du - du.mean(-1, keepdim=True)
    return tuple([(r * (du - n * m)).transpose(1, 2).contiguous().to(dt)] + out)


def _doubling(a, b):
    """Every h_t = a_t h_(t-1) + b_t along dim 1 (h before the first 0), in place, by
    composing spans of 1, 2, 4, ... tokens."""
    step = 1
    while step < a.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] *= a[:, :-step].clone()
        step *= 2
    return b


def _scan_plain(x, log_a, h0):
    a, b = torch.exp(log_a), x.float() if x.dtype != torch.float32 else x.clone()
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _doubling(a, b)
    return h.to(x.dtype), h[:, -1].clone()


def _scan_bwd_plain(s):
    h, h0, dh = s["h"], s["h0"], s["dh"].float()
    a = torch.exp(s["log_a"])
    c = a * dh  # c_t = a_t (dh_t + c_(t+1))
    if s["dhT"] is not None:
        c[:, -1] += a[:, -1] * s["dhT"]
    c = _doubling(a.flip(1), c.flip(1)).flip(1)
    dx = dh
    dx[:, :-1] += c[:, 1:]
    if s["dhT"] is not None:
        dx[:, -1] += s["dhT"]
    dla = torch.empty_like(c)
    dla[:, 1:] = c[:, 1:] * h[:, :-1].float()
    dla[:, 0] = 0.0 if h0 is None else c[:, 0] * h0
    return dx.to(h.dtype), dla, c[:, 0].clone()


def _step_plain(s):
    h = torch.exp(s["log_a"]) * s["h0"] + s["x"].float()
    return h.to(s["x"].dtype), h


# ---- one pass ------------------------------------------------------------------------

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "qk":
            return _qk_plain(s)
        if op == "qk_bwd":
            return _qk_bwd_plain(s)
        if op == "gate":
            return _gate_plain(s)
        if op == "gate_bwd":
            return _gate_bwd_plain(s)
        if op == "scan":
            return _scan_plain(s["x"], s["log_a"], s["h0"])
        if op == "scan_bwd":
            return _scan_bwd_plain(s)
        return _step_plain(s)
    import retnet_retention_gb300 as la
    if op.startswith("qk"):
        opts = dict(positions=s["positions"], rot=c["rot"], inv_freq=s["inv_freq"],
                    interleaved=c["pairs"] == "adjacent", norm=c["norm"], q_weight=s["wq"],
                    k_weight=s["wk"], eps=EPS)
        if op == "qk":
            return la.qk_rotate_fwd(s["q"], s["k"], **opts)
        dq, dk, dwq, dwk = la.qk_rotate_bwd(s["q"], s["k"], s["dyq"], s["dyk"], **opts)
        return (dq, dk) if dwq is None else (dq, dk, dwq, dwk)
    if op == "gate":
        return (la.head_gate_fwd(s["o"], s["g"], weight=s["w"], eps=EPS, center=c["center"]),)
    if op == "gate_bwd":
        out = la.head_gate_bwd(s["o"], s["g"], s["dy"], weight=s["w"], eps=EPS, center=c["center"])
        return tuple(t for t in out if t is not None)
    if op == "scan":
        return la.scan_fwd(s["x"], s["log_a"], h0=s["h0"])
    if op == "scan_bwd":
        return la.scan_bwd(s["log_a"], s["h"], s["dh"], h0=s["h0"], dh_T=s["dhT"])
    return la.scan_step(s["x"], s["log_a"], s["h0"], h_out=s["h1"]), s["h1"]


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    if op.startswith("qk"):
        n = B * T * (case["H"] + case["HK"]) * case["d"]
        small = (4 * B * T if case["positions"] else 0) + (
            8 * case["d"] if case["norm"] and case["weight"] else 0)
        return dict(bytes=n * e * (2 if op == "qk" else 3) + small * (1 if op == "qk" else 2),
                    flops=n * (10 if op == "qk" else 20))
    if op.startswith("gate"):
        n = B * T * case["H"] * case["d"]
        small = 4 * case["H"] * case["d"] if case["weight"] else 0
        tensors = (2, 3) if op == "gate" else (3, 5)
        return dict(bytes=n * e * tensors[case["gate"]] + small * (1 if op == "gate" else 2),
                    flops=n * (12 if op == "gate" else 30))
    n, state = B * T * case["D"], 4 * B * case["D"]
    if op == "scan":
        return dict(bytes=n * (4 + 2 * e) + state * (2 if case["state"] else 1), flops=3 * n)
    if op == "scan_bwd":
        return dict(bytes=n * (8 + 3 * e) + state * (3 if case["state"] else 1), flops=5 * n)
    return dict(bytes=n * (4 + 2 * e) + 2 * state, flops=3 * n)


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d64 = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for n, t in s.items()}
    if op.startswith("qk"):
        return _qk_exact(case, d64)
    if op.startswith("gate"):
        return _gate_exact(case, d64)
    return _recurrence_exact(case, d64)


def _qk_exact(case, s):
    """As complex numbers: a pair times e^(i p f), the gradient times its conjugate."""
    B, T, d, rot = case["B"], case["T"], case["d"], case["rot"]
    p = s["positions"]
    p = torch.arange(T, device=DEV).expand(B, T) if p is None else p
    f = torch.tensor(s["inv_freq"], device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones(B, T, 1, rot // 2, device=DEV, dtype=torch.float64),
                       (p.to(torch.float64)[:, :, None] * f)[:, :, None])
    first = torch.arange(rot // 2, device=DEV)
    first, second = (2 * first, 2 * first + 1) if case["pairs"] == "adjacent" else (first, first + rot // 2)

    def turned(x, by):
        y = x.clone()
        if rot:
            z = torch.complex(x[..., first], x[..., second]) * by
            y[..., first], y[..., second] = z.real, z.imag
        return y

    out, weights = [], []
    for x, w, name in ((s["q"], s["wq"], "dyq"), (s["k"], s["wk"], "dyk")):
        size = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS) if case["norm"] else torch.ones_like(x[..., :1])
        unit = x / size
        scale = torch.ones(d, device=DEV, dtype=torch.float64) if w is None else w
        if case["op"] == "qk":
            out.append(turned(unit * scale, turn).permute(0, 2, 1, 3).contiguous())
            continue
        back = turned(s[name].permute(0, 2, 1, 3), turn.conj())
        if w is not None:
            weights.append(torch.einsum("bthd,bthd->d", back, unit))
        back = back * scale
        if case["norm"]:
            back = (back - unit * ((back * unit).sum(-1, keepdim=True) / d)) / size
        out.append(back)
    return tuple(out + weights)


def _gate_exact(case, s):
    o = s["o"].permute(0, 2, 1, 3)
    if case["center"]:
        o = o - o.sum(-1, keepdim=True) / case["d"]
    size = torch.sqrt(o.pow(2).sum(-1, keepdim=True) / case["d"] + EPS)
    unit = o / size
    w = torch.ones(case["H"], case["d"], device=DEV, dtype=torch.float64) if s["w"] is None else s["w"]
    sig = None if s["g"] is None else torch.sigmoid(s["g"])
    act = 1.0 if sig is None else s["g"] * sig
    if case["op"] == "gate":
        return (unit * w * act,)
    dy = s["dy"]
    back = dy * act * w
    along = (back * unit).sum(-1, keepdim=True) / case["d"]
    mean = back.sum(-1, keepdim=True) / case["d"] if case["center"] else 0.0
    out = [((back - mean - unit * along) / size).permute(0, 2, 1, 3).contiguous()]
    if sig is not None:
        out.append(dy * unit * w * (sig + act * (1.0 - sig)))
    if s["w"] is not None:
        out.append(torch.einsum("bthd,bthd->hd", dy * act, unit))
    return tuple(out)


def _recurrence_exact(case, s):
    """Token by token."""
    a = torch.exp(s["log_a"])
    if case["op"] == "step":
        h = a * s["h0"] + s["x"]
        return h, h
    B, T, D = a.shape
    zero = torch.zeros(B, D, device=DEV, dtype=torch.float64)
    start = zero if s["h0"] is None else s["h0"]
    if case["op"] == "scan":
        h = s["x"]
        last = start
        for t in range(T):
            last = h[:, t].addcmul_(a[:, t], last)
        return h, last.clone()
    dx = s["dh"]
    carry = zero if s["dhT"] is None else s["dhT"]
    dla = torch.empty_like(a)
    for t in range(T - 1, -1, -1):
        dx[:, t] += carry
        carry = torch.mul(a[:, t], dx[:, t], out=dla[:, t])
    dh0 = carry.clone()
    dla[:, 1:] *= s["h"][:, :-1]
    dla[:, 0] *= start
    return dx, dla, dh0
