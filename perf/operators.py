"""The sequence recurrence and the parameter update, as a training or serving program calls them.

Two families of cases:

* ``glr``: the gated linear recurrence, forward alone or forward and backward,
      s = c softplus(lam) sigmoid(r),  a = exp(-s),  u = sqrt(1 - a^2) sigmoid(i) x,  h_t = a_t h_{t-1} + u_t
  per sequence and channel, in either direction, over dense, padded and packed batches, with and without a
  start state; a one-token step updates its state in place.
* ``adamw``: one AdamW step over every parameter of a stack of layers (conv taps and bias, four projections,
  gate weight and bias, norm scale each), states in 32 or in 8 bits, with or without clipping by the global
  gradient norm.

``own`` false computes them with elementary torch operations, true with this repository's kernels.
"""
import math
import random

import torch

own = False

C = 8.0           # the recurrence's decay constant
LR, BETAS, EPS, WD, MAX_NORM, SEED = 1e-3, (0.9, 0.999), 1e-8, 0.01, 1.0, 77
BLOCK = 256       # values that share a scale in the 8-bit states
T0 = 10           # steps already taken


# ----------------------------------------------------------------- cases
def _glr(name, B, L, d, dtype="bf16", train=False, form="dense", lo=1, reverse=False, state=False, packed=False):
    c = {"op": "glr", "B": B, "L": L, "d": d, "dtype": dtype, "train": train, "form": form, "lo": lo,
         "reverse": reverse, "state": state, "packed": packed}
    return dict(c, name=name) if name else c


def _adamw(name, d, H, dh, layers, bits, param="bf16", grad="f32", clip=False):
    c = {"op": "adamw", "d": d, "H": H, "dh": dh, "layers": layers, "bits": bits, "param": param, "grad": grad, "clip": clip}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new event for each of 16 users whose state is kept: latency counts
        _glr("glr step B16 d512", 16, 1, 512, state=True),
        # the encoder's ordinary batch
        _glr("glr fwd B32 L2048 d512", 32, 2048, 512),
        # the other direction of a bidirectional encoder over long histories, projections from one matrix product
        _glr("glr fwd rev B8 L32768 d512", 8, 32768, 512, reverse=True, packed=True),
        # one very long history alone: few independent channels, the scan itself counts
        _glr("glr fwd B1 L65536 d512", 1, 65536, 512, state=True),
        # packed histories of every length, continued from their states
        _glr("glr fwd varlen d1024", 64, 16384, 1024, form="varlen", lo=64, state=True),
        # a small odd layer in fp32, trained: latency and ragged edges
        _glr("glr train f32 B2 L257 d72", 2, 257, 72, dtype="f32", train=True, form="padded", lo=1),
        # the training step's batch
        _glr("glr train B16 L8192 d512", 16, 8192, 512, train=True),
        # packed training batch
        _glr("glr train varlen d1024", 64, 8192, 1024, train=True, form="varlen", lo=64, reverse=True, state=True),
        # the tiny fp32 layer's nine tensors: latency
        _adamw("adamw f32 tiny", 64, 2, 32, 1, 32, param="f32"),
        # a bf16 encoder of 12 layers with fp32 masters, clipped
        _adamw("adamw bf16 12 layers d512", 512, 8, 64, 12, 32, clip=True),
        # a wide one of 48 layers with 8-bit states, clipped
        _adamw("adamw 8bit 48 layers d1024", 1024, 8, 128, 48, 8, clip=True),
        # odd sizes, bf16 gradients
        _adamw("adamw 8bit odd", 200, 3, 52, 2, 8, param="f32", grad="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        step = rng.random() < 0.15
        while True:
            form = "dense" if step else rng.choice(["dense", "padded", "varlen"])
            d = rng.choice([64, 128, 256, 512, 1024, _log_int(rng, 8, 1024)])
            L = 1 if step else _log_int(rng, 2, 65536)
            B = _log_int(rng, 1, 512)
            if B * L * d <= 60_000_000:
                break
        return _glr(None, B, L, d, dtype=rng.choice(["bf16", "bf16", "f32"]), train=not step and rng.random() < 0.5, form=form,
                    lo=rng.randint(0, min(L, 64)), reverse=rng.random() < 0.5, state=step or rng.random() < 0.5,
                    packed=d <= 512 and rng.random() < 0.4)
    while True:
        H, dh = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([32, 64, 128, rng.randint(8, 128)])
        d, layers = rng.choice([64, 256, 512, 1024, rng.randint(16, 1024)]), _log_int(rng, 1, 48)
        if layers * d * H * dh * 4 <= 200_000_000:
            break
    return _adamw(None, d, H, dh, layers, rng.choice([8, 32]), param=rng.choice(["bf16", "f32"]),
                  grad=rng.choice(["f32", "f32", "bf16"]), clip=rng.random() < 0.5)


def _lengths(case):
    """The sequences' lengths, by the case alone: log-uniform from `lo` to L, the longest L."""
    B, L, lo = case["B"], case["L"], case["lo"]
    if case["form"] == "dense":
        return [L] * B
    rng = random.Random(B * 1000003 + L * 31 + lo)
    ln = [int(math.exp(rng.uniform(math.log(lo + 1), math.log(L + 1)))) - 1 for _ in range(B)]
    ln = [max(lo, min(L, n)) for n in ln]
    ln[rng.randrange(B)] = L
    return ln


def _sizes(case):
    d, HD, H = case["d"], case["H"] * case["dh"], case["H"]
    one = [(d, 4), (d,), (d, HD), (d, HD), (d, HD), (d, HD), (d, H), (H,), (case["dh"],)]
    return one * case["layers"]


def work(case):
    if case["op"] == "glr":
        es, d = (2 if case["dtype"] == "bf16" else 4), case["d"]
        n = sum(_lengths(case)) * d
        st = case["B"] * d * 4 * (2 if case["state"] else 0)
        # forward: x, r, i in, y out; backward (after the rest of the net): x, r, i, dy in, dx, dr, di out
        b = 4 * es * n + st + 4 * d
        if case["train"]:
            b += 7 * es * n + 8 * d + 3 * case["B"] * d * 4 * (1 if case["state"] else 0)
        return {"bytes": b, "flops": (70 if case["train"] else 25) * n}
    n = sum(math.prod(s) for s in _sizes(case))
    p = 10 if case["param"] == "bf16" else 8            # bf16 copy written, fp32 master read and written
    g = 4 if case["grad"] == "f32" else 2
    s = 16 if case["bits"] == 32 else 4 + 16 / BLOCK    # m and v read and written (and their scales)
    return {"bytes": n * (p + g + s), "flops": n * 18}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _gen(seed)
    f = dict(generator=g, device="cuda", dtype=torch.float32)
    if case["op"] == "glr":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        ln, d, B = _lengths(case), case["d"], case["B"]
        rows = sum(ln) if case["form"] == "varlen" else B * case["L"]
        s = {"case": case, "lens": ln, "rows": rows}
        if case["packed"]:  # [x | r | i] as one projection leaves them
            xri = torch.randn(rows, 3 * d, **f).to(dt)
            s["x"], s["r"], s["i"] = xri[:, :d], xri[:, d:2 * d], xri[:, 2 * d:]
        else:
            s["x"], s["r"], s["i"] = (torch.randn(rows, d, **f).to(dt) for _ in range(3))
        # decays at r -> infinity between 0.9 and 0.999
        a1 = 0.9 + 0.099 * torch.rand(d, **f)
        s["lam"] = torch.log(torch.expm1(-torch.log(a1) / C))
        if case["state"]:
            s["h0"] = torch.randn(B, d, **f)
        if case["train"]:
            s["dy"] = torch.randn(rows, d, **f).to(dt)
            if case["state"]:
                s["dhT"] = torch.randn(B, d, **f)
        if case["form"] == "varlen":
            s["cu"] = torch.tensor([0] + ln, device="cuda").cumsum(0).to(torch.int32)
        elif case["form"] == "padded":
            s["seq_lens"] = torch.tensor(ln, dtype=torch.int32, device="cuda")
        return s
    sizes = _sizes(case)
    at, off = [], 0
    for z in sizes:
        at.append(off)
        off += -(-math.prod(z) // BLOCK) * BLOCK
    live = torch.zeros(off, dtype=torch.bool, device="cuda")
    for z, o in zip(sizes, at):
        live[o:o + math.prod(z)] = True
    rnd = lambda scale: torch.where(live, torch.randn(off, **f) * scale, torch.zeros((), device="cuda"))  # noqa: E731
    cut = lambda t: [t[o:o + math.prod(z)].view(z) for z, o in zip(sizes, at)]  # noqa: E731
    pt = torch.bfloat16 if case["param"] == "bf16" else torch.float32
    gt = torch.float32 if case["grad"] == "f32" else torch.bfloat16
    size = torch.exp(2 * torch.randn(off, **f))  # gradients differ in size from parameter to parameter
    master = rnd(0.05)
    s = {"case": case, "grad": (rnd(1e-3) * size).to(gt), "step": torch.full((1,), T0, dtype=torch.int64, device="cuda")}
    m, r = rnd(3e-4) * size, rnd(1e-3).abs() * size
    del size
    s["param"] = master.to(pt) if pt == torch.bfloat16 else master
    if pt == torch.bfloat16:
        s["master"] = master
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        half = torch.full((off,), 1 << 15, dtype=torch.int64, device="cuda")
        s["m"], s["m_scale"] = _encode(m, half)
        s["v"], s["v_scale"] = _encode(r, half, root=True)
        s["m_scales"] = [s["m_scale"][o // BLOCK:o // BLOCK + -(-math.prod(z) // BLOCK)] for z, o in zip(sizes, at)]
        s["v_scales"] = [s["v_scale"][o // BLOCK:o // BLOCK + -(-math.prod(z) // BLOCK)] for z, o in zip(sizes, at)]
    s["views"] = {k: cut(s[k]) for k in ("param", "master", "grad", "m", "v") if k in s}
    return s


# ----------------------------------------------- the recurrence, plain form
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan(a, u, longest):
    """h_t = a_t h_{t-1} + u_t along dim 1 by doubling; a is 0 where a sequence starts."""
    h, a = u.clone(), a.clone()
    s = 1
    while s < longest:
        h[:, s:] = h[:, s:] + a[:, s:] * h[:, :-s]
        a[:, s:] = a[:, s:] * a[:, :-s]
        s *= 2
    return h


def _plain_glr(st):
    case = st["case"]
    d, B, train, form = case["d"], case["B"], case["train"], case["form"]
    dev = st["x"].device
    n = 1 if form == "varlen" else B
    rows = st["rows"] // n
    cut = lambda t: t.float().reshape(n, rows, d)  # noqa: E731
    turn = (lambda t: t.flip(1)) if case["reverse"] else (lambda t: t)
    # where each sequence's rows begin and end, in the order of the recurrence
    pos = torch.arange(rows, device=dev)
    if form == "varlen":
        cu = st["cu"].long()
        lens = cu[1:] - cu[:-1]
        has = lens > 0
        lo, hi = cu[:-1], cu[1:] - 1
        valid = torch.ones(1, rows, dtype=torch.bool, device=dev)
        seq = torch.zeros(B, dtype=torch.long, device=dev)
    else:
        lens = st["seq_lens"].long() if form == "padded" else torch.full((B,), rows, device=dev)
        has = lens > 0
        lo, hi = torch.zeros(B, dtype=torch.long, device=dev), lens - 1
        valid = pos[None, :] < lens[:, None]
        seq = torch.arange(B, device=dev)
    if case["reverse"]:
        lo, hi = rows - 1 - hi, rows - 1 - lo
        valid = valid.flip(1)
    seq, lo, hi = seq[has], lo[has], hi[has]
    x, r, i = turn(cut(st["x"])), turn(cut(st["r"])), turn(cut(st["i"]))
    v = valid[..., None]
    sp = _softplus(st["lam"])
    sr = _sigmoid(r)
    s = C * sp * sr
    a = torch.exp(-s)
    m = torch.sqrt(-torch.expm1(-2 * s))
    gi = _sigmoid(i)
    u = torch.where(v, m * gi * x, 0.0)
    h0 = st["h0"] if case["state"] else torch.zeros(B, d, device=dev)
    a_in = torch.where(v, a, 0.0)
    u[seq, lo] += a[seq, lo] * h0[has]
    a_in[seq, lo] = 0
    h = _scan(a_in, u, case["L"])
    y = turn(torch.where(v, h, 0.0)).reshape(st["rows"], d).to(st["x"].dtype)
    hT = h0.clone()
    hT[has] = h[seq, hi]
    if not train:
        if case["state"]:
            st["h0"].copy_(hT)  # the kept state, in place
            return {"y": y, "h": st["h0"]}
        return {"y": y}
    before = torch.zeros_like(h)
    before[:, 1:] = h[:, :-1]
    before[seq, lo] = h0[has]
    w = torch.where(v, turn(cut(st["dy"])), 0.0)
    if case["state"]:
        w[seq, hi] += st["dhT"][has]
    nxt = torch.zeros_like(a)
    nxt[:, :-1] = a_in[:, 1:]
    w = _scan(nxt.flip(1), w.flip(1), case["L"]).flip(1)
    w = torch.where(v, w, 0.0)
    q = torch.where(m > 0, s / m, 0.0)
    ds = -w * (a * before * s - gi * x * a * a * q)   # s dL/ds
    dr = ds * (1 - sr)
    dx, di = w * m * gi, w * m * x * gi * (1 - gi)
    back = lambda t: turn(torch.where(v, t, 0.0)).reshape(st["rows"], d).to(st["x"].dtype)  # noqa: E731
    out = {"y": y, "dx": back(dx), "dr": back(dr), "di": back(di),
           "dlam": torch.where(v, ds, 0.0).sum((0, 1)) * _sigmoid(st["lam"]) / sp}
    if case["state"]:
        dh0 = st["dhT"].clone()
        dh0[has] = a[seq, lo] * w[seq, lo]
        out["hT"], out["dh0"] = hT, dh0
    return out


def _own_glr(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    if "shape" not in st:  # what a program keeps: the shape and its workspaces
        n = case["B"] if case["form"] != "varlen" else 1
        rows = case["L"] if case["form"] != "varlen" else st["rows"]
        st["shape"] = gbla.glr_shape(n, rows, case["d"], dtype=case["dtype"], cu_seqlens=st.get("cu"), seq_lens=st.get("seq_lens"))
        st["ws"] = gbla.workspace(st["shape"], gbla.GBLA_OP_GLR_FORWARD)
        if case["train"]:
            st["ws_b"] = gbla.workspace(st["shape"], gbla.GBLA_OP_GLR_BACKWARD)
    kw = dict(c=C, reverse=case["reverse"], h0=st.get("h0"))
    if not case["train"]:
        y, hT, _ = gbla.glr_forward(st["shape"], st["x"], st["r"], st["i"], st["lam"], hT=st.get("h0"), ws=st["ws"], **kw)
        return {"y": y, "h": hT} if case["state"] else {"y": y}
    y, hT, saved = gbla.glr_forward(st["shape"], st["x"], st["r"], st["i"], st["lam"], hT=case["state"] or None, saved=True,
                                    ws=st["ws"], **kw)
    g = gbla.glr_backward(st["shape"], st["x"], st["r"], st["i"], st["lam"], saved, st["dy"], dhT=st.get("dhT"),
                          ws=st["ws_b"], **kw)
    out = {"y": y, "dx": g["dx"], "dr": g["dr"], "di": g["di"], "dlam": g["dlam"]}
    if case["state"]:
        out["hT"], out["dh0"] = hT, g["dh0"]
    return out


# ------------------------------------------- the parameter update, plain form
def _encode(x, dither, root=False):
    """e4m3 values of x and their scales: a block's largest magnitude becomes 448, and each value is rounded up with the
    probability that the 16-bit `dither` stands for.  A `root` above 0 keeps a value above 0."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    live = top >= 2.0 ** -100
    scale = torch.where(live, top / 448, 0.0)
    t = torch.clamp((b.abs() * torch.where(live, 448 / top, 0.0)[:, None]).view(-1), max=448.0)
    normal = ((t.view(torch.int32).long() + (dither << 4)) >> 20) - ((127 - 7) << 3)
    small = torch.floor(t * 2.0 ** 9 + dither.float() * 2.0 ** -16).long()
    code = torch.where(t >= 2.0 ** -6, normal, small)
    code = torch.where(t > 0, code.clamp(min=1), code) if root else code + 128 * torch.signbit(x).long()
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale


def _decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _mix(x):
    """A 32-bit hash (shifts and odd multiplications) on int64 values."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dither(n, step):
    """The 32 random bits of every value, from the seed, the step and the value's place."""
    at = torch.arange(n, device=step.device)
    key = _mix((_mix((step & 0xFFFFFFFF) ^ 0x9E3779B9) + SEED) & 0xFFFFFFFF)
    return _mix(((at & 0xFFFFFFFF) * 0x9E3779B9 + (at >> 32) * 0xBB67AE85 + key) & 0xFFFFFFFF)


def _plain_adamw(st):
    case = st["case"]
    g = st["grad"].float()
    out = {}
    if case["clip"]:
        norm = g.double().square().sum().sqrt().float()
        g = g * torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
        out["norm"] = norm
    st["step"] += 1
    t = st["step"].double()
    b1, b2 = BETAS
    p = st.get("master", st["param"])
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m, v = _decode(st["m"], st["m_scale"]), _decode(st["v"], st["v_scale"])  # v is kept as its root
        v = v * v
    m = b1 * m + (1 - b1) * g
    v = b2 * v + ((1 - b2) * g) * g
    root = torch.sqrt(v)
    step = (LR / (1 - b1 ** t)).float()
    den = root * (1 / torch.sqrt(1 - b2 ** t)).float() + EPS
    p.copy_(p * (1 - LR * WD) - step * (m / den))
    if "master" in st:
        st["param"].copy_(p)
        out["master"] = p
    out["param"] = st["param"]
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        out["m"], out["v"] = st["m"], st["v"]
    else:
        z = _dither(g.numel(), st["step"])
        for k, x, dither in (("m", m, z & 0xFFFF), ("v", root, z >> 16)):
            code, scale = _encode(x, dither, root=k == "v")
            st[k].copy_(code)
            st[k + "_scale"].copy_(scale)
            out[k], out[k + "_scale"] = st[k], st[k + "_scale"]
    out["step"] = st["step"]
    return out


def _own_adamw(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    if "plan" not in st:  # what a program keeps: which tensors are updated, by which gradients and states
        w = st["views"]
        st["plan"] = gbla.gbla_adamw_plan(w["param"], w["grad"], {
            "step": st["step"], "m": w["m"], "v": w["v"], "master": w.get("master"),
            "m_scale": st.get("m_scales"), "v_scale": st.get("v_scales")})
    out = {}
    norm = None
    if case["clip"]:
        out["norm"] = norm = gbla.gbla_grad_norm(st["plan"])
    gbla.gbla_adamw_step(st["plan"], lr=LR, betas=BETAS, eps=EPS, weight_decay=WD, norm=norm,
                         max_norm=MAX_NORM if case["clip"] else None, seed=SEED)
    if "master" in st:
        out["master"] = st["master"]
    out["param"] = st["param"]
    for k in ("m", "v", "m_scale", "v_scale", "step"):
        if k in st:
            out[k] = st[k]
    return out


def run(state):
    if state["case"]["op"] == "glr":
        return _own_glr(state) if own else _plain_glr(state)
    return _own_adamw(state) if own else _plain_adamw(state)


# --------------------------------------------------------- in 64 bits
def _exact_glr(st):
    """Token by token in 64 bits, over the sequences from the longest on."""
    case, d, B = st["case"], st["case"]["d"], st["case"]["B"]
    dev, ln = st["x"].device, st["lens"]
    X, R, I = (st[k].double() for k in "xri")
    lam = st["lam"].double()
    sp = torch.nn.functional.softplus(lam, threshold=100)
    sr, si = torch.sigmoid(R), torch.sigmoid(I)
    loga = -C * sp * sr
    del R, I
    A = loga.exp()
    M = (-torch.expm1(2 * loga)).sqrt()
    U = M * si * X
    first, n = [], 0
    for k in range(B):
        first.append(n if case["form"] == "varlen" else k * case["L"])
        n += ln[k]
    order = sorted(range(B), key=lambda k: -ln[k])
    by_len = sorted(ln)
    start = torch.tensor([first[k] for k in order], device=dev)
    size = torch.tensor([ln[k] for k in order], device=dev)
    perm = torch.tensor(order, device=dev)
    rev = case["reverse"]
    active, j = [], 0  # how many sequences have a token t
    for t in range(case["L"]):
        while j < B and by_len[j] <= t:
            j += 1
        active.append(B - j)
    at = lambda t, k: (start[:k] + (size[:k] - 1 - t)) if rev else start[:k] + t  # noqa: E731
    h = st["h0"].double()[perm] if case["state"] else torch.zeros(B, d, dtype=torch.float64, device=dev)
    H, P = torch.zeros_like(X), torch.zeros_like(X)
    for t in range(case["L"]):
        k = active[t]
        rows = at(t, k)
        P[rows] = h[:k]
        h[:k] = A[rows] * h[:k] + U[rows]
        H[rows] = h[:k]
    hT = torch.empty_like(h)
    hT[perm] = h
    if not case["train"]:
        return {"y": H, "h": hT} if case["state"] else {"y": H}
    w = st["dhT"].double()[perm] if case["state"] else torch.zeros_like(h)
    W, DY = torch.zeros_like(X), st["dy"].double()
    for t in reversed(range(case["L"])):
        k = active[t]
        rows = at(t, k)
        now = w[:k] + DY[rows]
        W[rows] = now
        w[:k] = A[rows] * now
    dh0 = torch.empty_like(w)
    dh0[perm] = w
    dl = W * A * (P - si * X * A / M)   # dL/d(log a)
    out = {"y": H, "dx": W * M * si, "dr": dl * loga * (1 - sr), "di": W * U * (1 - si),
           "dlam": (dl * -C * sr).sum(0) * torch.sigmoid(lam)}
    if case["state"]:
        out["hT"], out["dh0"] = hT, dh0
    return out


def _exact_adamw(st):
    case = st["case"]
    g = st["grad"].double()
    out = {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = norm
        g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
    t = T0 + 1
    p = st.get("master", st["param"]).double()
    if case["bits"] == 32:
        m, v = st["m"].double(), st["v"].double()
    else:  # the value of every code, from a table
        k = torch.arange(256, device=g.device)
        e, f = (k >> 3) & 15, (k & 7).double() / 8
        table = torch.where(e > 0, (1 + f) * torch.exp2(e.double() - 7), f * 2.0 ** -6) * torch.where(k < 128, 1.0, -1.0)
        m, v = ((table[st[n].view(torch.uint8).long()].view(-1, BLOCK) * st[n + "_scale"].double()[:, None]).view(-1) for n in "mv")
        v = v ** 2
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * g ** 2
    p = p - LR * WD * p - LR * (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)).sqrt() + EPS)
    out["param"] = p
    if "master" in st:
        out["master"] = p
    if case["bits"] == 32:  # which way an 8-bit state is rounded is the 32-bit arithmetic's own
        out["m"], out["v"] = m, v
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_glr(st) if case["op"] == "glr" else _exact_adamw(st)
