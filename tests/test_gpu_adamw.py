"""gbla_adamw_step and gbla_grad_norm: fp32 states against the formulas in 64
bits, 8-bit states bit for bit against the same fp32 operations in numpy, their
rounding's mean, clipping, skipped steps, sizes around the blocks and tables,
alignment, graphs, and a training step of the layer and the recurrence with its
update.

Bounds (none fitted): m and v are two products and a sum, so at most 4 * 2^-24 of
the sum of magnitudes each, and the clip factor 3 * 2^-24 relative; the update's
quotient m / (sqrt(v) inv + eps) adds the root, product, sum, quotient (2 ulp) and
the step's rounding: 16 * 2^-24 of the update and 3 * 2^-24 of p; a bf16 parameter
is rounded once (2^-8)."""
import numpy as np
import pytest
import torch

import oracle
from generative_retrieval_encoder_gb300 import build, gbla
from glr_cases import check, reference

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
LR, BETAS, EPS, WD = 3e-3, (0.9, 0.999), 1e-8, 0.02
SIZES = [1, 5, 31, 255, 256, 257, 2047, 2048, 2049, 6000, 0, 70000]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gbla.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, param="f32", grad="f32", bits=32, seed=0, offset=0, master=None, warm=True):
    """params, grads, state: `offset` values into a larger buffer each (so of the element's alignment alone)."""
    gen = torch.Generator().manual_seed(seed)
    pt, gt = (torch.bfloat16 if k == "bf16" else torch.float32 for k in (param, grad))

    def place(t):
        b = torch.zeros(t.numel() + offset + 8, dtype=t.dtype if t.dtype.itemsize > 1 else torch.uint8, device="cuda")
        v = b[offset:offset + t.numel()]
        v.copy_(t if t.dtype.itemsize > 1 else t.view(torch.uint8))
        return v if t.dtype.itemsize > 1 else v.view(t.dtype)

    P = [place((torch.randn(n, generator=gen) * 0.1).to(pt)) for n in sizes]
    G = [place((torch.randn(n, generator=gen) * torch.exp(2 * torch.randn(n, generator=gen)) * 1e-2).to(gt)) for n in sizes]
    st = gbla.gbla_adamw_state(P, bits=bits, master=master)
    for k in ("m", "v", "m_scale", "v_scale"):
        if k in st:
            st[k] = [place(t.cpu()) for t in st[k]]
    if st.get("master"):
        st["master"] = [None if t is None else place(t.cpu()) for t in st["master"]]
    if warm and bits == 32:
        for m, v, g in zip(st["m"], st["v"], G):
            m.copy_(torch.randn(m.numel(), generator=gen).cuda() * g.float().abs())
            v.copy_(g.float() ** 2 * torch.rand(v.numel(), generator=gen).cuda())
        st["step"].fill_(20)
    return P, G, st


def test64(p, m, v, g, t, wd, clip=1.0, lr=LR):
    """(p, m, v) after step t in 64 bits, and their bounds without the outputs' own rounding."""
    b1, b2 = BETAS
    g = g * clip
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    bm = 4 * E * (np.abs(b1 * m) + np.abs((1 - b1) * g)) + 3 * E * np.abs((1 - b1) * g)
    bv = 4 * E * v1 + 6 * E * (1 - b2) * g * g + 1e-45
    den = np.sqrt(v1 / (1 - b2 ** t)) + EPS
    up = lr / (1 - b1 ** t) * m1 / den
    dden = bv / np.maximum(2 * np.sqrt(v1 * (1 - b2 ** t)), 1e-30)
    bp = 3 * E * np.abs(p) + 16 * E * np.abs(up) + lr / (1 - b1 ** t) * (bm / den + np.abs(m1) / den ** 2 * dden)
    return (p * (1 - lr * wd) - up, m1, v1), (bp, bm, bv)


test64.__test__ = False


@pytest.mark.parametrize("param,grad,master,offset", [("f32", "f32", None, 0), ("f32", "bf16", None, 1), ("bf16", "f32", None, 0),
                                                       ("bf16", "f32", False, 0), ("bf16", "bf16", None, 3), ("bf16", "bf16", False, 0)])
@pytest.mark.parametrize("clip", [False, True])
def test_fp32_states_match_formulas(param, grad, master, offset, clip):
    P, G, st = make(SIZES, param, grad, master=master, offset=offset, seed=offset + 7)
    plan = gbla.gbla_adamw_plan(P, G, st)
    wd = [WD * (j % 3) for j in range(len(P))]
    norm = gbla.gbla_grad_norm(plan) if clip else None
    w_norm = np.sqrt(sum((f64(g) ** 2).sum() for g in G))
    if clip:
        assert abs(float(norm) - w_norm) <= 1.01 * E * w_norm  # one rounding
    cf = min(1.0, 0.5 / (w_norm + 1e-6)) if clip else 1.0
    src = st["master"] if param == "bf16" and master is None else P
    want = [test64(f64(s), f64(m), f64(v), f64(g), 21, w, cf) for s, m, v, g, w in zip(src, st["m"], st["v"], G, wd)]
    gbla.gbla_adamw_step(plan, LR, BETAS, EPS, wd, norm=norm, max_norm=0.5 if clip else None)
    torch.cuda.synchronize()
    assert int(st["step"]) == 21
    for j, ((p, m, v), (bp, bm, bv)) in enumerate(want):
        assert (np.abs(f64(st["m"][j]) - m) <= bm).all(), j
        assert (np.abs(f64(st["v"][j]) - v) <= bv).all(), j
        if src is not P:
            assert (np.abs(f64(src[j]) - p) <= bp).all(), j
            assert torch.equal(P[j], src[j].bfloat16())
        else:
            half = 2.0 ** -8 if param == "bf16" else E
            assert (np.abs(f64(P[j]) - p) <= bp + half * np.abs(p)).all(), j


# ---------------------------------------------------------------- 8 bits
def f32(x):
    return np.asarray(x, np.float32)


def mix(x):
    x = x.astype(np.uint32)
    x = x ^ (x >> np.uint32(16))
    x = x * np.uint32(0x6A09E667)
    x = x ^ (x >> np.uint32(15))
    x = x * np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


TABLE = np.array([(1 + (k & 7) / 8) * 2.0 ** ((k >> 3) - 7) if k >> 3 else (k & 7) / 8 * 2.0 ** -6 for k in range(128)], np.float32)


def decode(code, scale):
    v = TABLE[code & 127] * np.repeat(scale, 256)[:code.size]
    return np.where(code & 128, -v, v).astype(np.float32)


def encode(x, d, root):
    n = x.size
    b = np.zeros(-(-n // 256) * 256, np.float32)
    b[:n] = np.abs(x)
    top = b.reshape(-1, 256).max(1)
    live = top >= np.float32(2.0 ** -100)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(live, f32(np.float32(1) / top) * np.float32(448), np.float32(0)).astype(np.float32)
    scale = np.where(live, top * np.float32(1 / 448), np.float32(0)).astype(np.float32)
    t = np.minimum(np.abs(x) * np.repeat(inv, 256)[:n], np.float32(448)).astype(np.float32)
    normal = ((t.view(np.uint32) + (d.astype(np.uint32) << np.uint32(4))) >> np.uint32(20)).astype(np.int64) - 960
    small = np.floor(t * np.float32(512) + d.astype(np.float32) * np.float32(2.0 ** -16)).astype(np.int64)
    code = np.where(t >= np.float32(2.0 ** -6), normal, small)
    code = np.where(t > 0, np.maximum(code, 1), code) if root else code + 128 * np.signbit(x)
    return code.astype(np.uint8), scale


def step8(codes, scales, g, t, place, seed, clip=np.float32(1)):
    """The new codes, scales and fp32 (m, root) of a tensor, in fp32 operations each rounded once."""
    c = [np.float32(v) for v in (BETAS[0], 1 - BETAS[0], BETAS[1], 1 - BETAS[1])]
    g = f32(g * clip)
    m, r = decode(codes[0], scales[0]), decode(codes[1], scales[1])
    v = r * r
    m = c[0] * m + c[1] * g
    v = c[2] * v + (c[3] * g) * g
    root = np.sqrt(v)
    with np.errstate(over="ignore"):
        key = mix(mix(np.array([t ^ 0x9E3779B9])) + np.uint32(seed))
        at = np.uint32(place) + np.arange(g.size, dtype=np.uint32)
        z = mix(at * np.uint32(0x9E3779B9) + key)
    (cm, sm), (cv, sv) = encode(m, z & np.uint32(0xFFFF), False), encode(root, z >> np.uint32(16), True)
    return (cm, cv), (sm, sv), (m, root)


@pytest.mark.parametrize("param,grad,offset", [("f32", "f32", 0), ("bf16", "f32", 0), ("f32", "bf16", 1), ("bf16", "bf16", 3)])
@pytest.mark.parametrize("clip", [False, True])
def test_8bit_states_bit_for_bit(param, grad, offset, clip):
    P, G, st = make(SIZES, param, grad, bits=8, offset=offset, seed=30 + offset)
    plan = gbla.gbla_adamw_plan(P, G, st)
    u8 = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    src = st["master"] if param == "bf16" else P
    for t in range(1, 5):
        for j, g in enumerate(G):
            g.mul_(-0.7 if t % 2 else 1.3)
            if j == 4:
                g.zero_()  # a block of zeros stays one
        place, want = 0, []
        norm = gbla.gbla_grad_norm(plan) if clip else None
        cf = np.float32(1)
        if clip:
            cf = min(np.float32(1) / (norm.cpu().numpy() + np.float32(1e-6)) * np.float32(0.25), np.float32(1))
        for j, g in enumerate(G):
            codes, scales = (u8(st["m"][j]), u8(st["v"][j])), (st["m_scale"][j].cpu().numpy(), st["v_scale"][j].cpu().numpy())
            old = f64(src[j])
            new = step8(codes, scales, g.float().cpu().numpy(), t, place, 1234567, cf)
            m, v = decode(codes[0], scales[0]).astype(np.float64), decode(codes[1], scales[1]).astype(np.float64) ** 2
            want.append((new, test64(old, m, v, f64(g), t, WD, float(cf))))
            place += -(-g.numel() // 256) * 256
        gbla.gbla_adamw_step(plan, LR, BETAS, EPS, WD, norm=norm, max_norm=0.25 if clip else None, seed=1234567)
        torch.cuda.synchronize()
        for j, ((codes, scales, _), ((p, _, _), (bp, _, _))) in enumerate(want):
            assert np.array_equal(u8(st["m"][j]), codes[0]) and np.array_equal(u8(st["v"][j]), codes[1]), (t, j)
            assert np.array_equal(st["m_scale"][j].cpu().numpy(), scales[0]), (t, j)
            assert np.array_equal(st["v_scale"][j].cpu().numpy(), scales[1]), (t, j)
            assert (np.abs(f64(src[j]) - p) <= bp).all(), (t, j)
            if src is not P:
                assert torch.equal(P[j], src[j].bfloat16())


def test_8bit_rounding_has_the_right_mean():
    """The mean over many values of one block's repeated state is that state: within 5 standard errors of the step's odds."""
    n = 256 * 4096
    x = np.linspace(0.001, 1.0, 256, dtype=np.float32)  # each block the same values, the last the block's largest
    g = torch.from_numpy(np.tile(x, n // 256)).cuda()
    P, st = [torch.zeros(n, device="cuda")], None
    st = gbla.gbla_adamw_state(P, bits=8)
    gbla.gbla_adamw_step(gbla.gbla_adamw_plan(P, [g], st), LR, seed=5)
    for name, c, full in (("m", 0.1, x * 0.1), ("v", 0.001, np.sqrt(0.001) * x)):
        got = (st[name][0].float().view(-1, 256) * st[name + "_scale"][0][:, None]).double().cpu().numpy()
        step = full.max() / 448 * np.maximum(2.0 ** (np.floor(np.log2(np.maximum(full / full.max() * 448, 2.0 ** -6))) - 3), 2.0 ** -9)
        err = np.abs(got.mean(0) - full) - 1e-6 * full
        assert (err <= 5 * 0.5 * step / np.sqrt(n // 256)).all(), name  # a step's rounding deviates by at most half of it
        assert (np.abs(got - full) <= step * 1.001).all()


def test_8bit_states_follow_the_fp32_ones():
    """Forty steps on noisy gradients: sqrt(v) of 8 bits stays near that of 32 on average (it would stand still under
    rounding to nearest: a step moves v by a thousandth), and zeros stay zero."""
    n = 1 << 16
    gen = torch.Generator().manual_seed(8)
    P = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
    G = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
    s32, s8 = gbla.gbla_adamw_state(P[:1]), gbla.gbla_adamw_state(P[1:], bits=8)
    p32, p8 = gbla.gbla_adamw_plan(P[:1], G[:1], s32), gbla.gbla_adamw_plan(P[1:], G[1:], s8)
    for _ in range(40):
        g = torch.randn(n, generator=gen)
        g[:1024] = 0
        for t in G:
            t.copy_(g)
        gbla.gbla_adamw_step(p32, LR, weight_decay=0.0)
        gbla.gbla_adamw_step(p8, LR, weight_decay=0.0)
    r32 = s32["v"][0].sqrt()[1024:]
    r8 = (s8["v"][0].float().view(-1, 256) * s8["v_scale"][0][:, None]).view(-1)
    assert (r8[:1024] == 0).all() and (P[1][:1024] == 0).all()
    # 64k roundings of at most 1/8 each a step, 40 steps: the mean's deviation is below 0.125 * sqrt(40 / 65000) = 0.4 %; the
    # root of a mean is at most the root mean square: allow the variance of 40 roundings, 40 / 40^2 * 1/64 < 2 %
    assert abs(float(r8[1024:].mean() / r32.mean()) - 1) < 0.025


def test_nonfinite_norm_skips_the_step():
    for bits in (8, 32):
        P, G, st = make([300, 5000], "bf16", bits=bits, seed=50)
        plan = gbla.gbla_adamw_plan(P, G, st)
        gbla.gbla_adamw_step(plan, LR)
        for bad in (float("nan"), float("inf"), float("-inf"), 3e38):
            keep = G[1][77].clone()
            G[1][77] = bad
            norm = gbla.gbla_grad_norm(plan)
            assert not torch.isfinite(norm)
            before = [t.clone() for t in P + st["m"] + st["v"] + st["master"]] + [st["step"].clone()]
            gbla.gbla_adamw_step(plan, LR, norm=norm, max_norm=1.0)
            for a, b in zip(before, P + st["m"] + st["v"] + st["master"] + [st["step"]]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            G[1][77] = keep


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_gradient_without_norm_spoils_its_block_alone(bad):
    P, G, st = make([1000], bits=8, seed=51)
    G[0][300] = bad
    gbla.gbla_adamw_step(gbla.gbla_adamw_plan(P, G, st), LR)
    m = st["m"][0].float() * st["m_scale"][0].repeat_interleave(256)[:1000]
    v = st["v"][0].float() * st["v_scale"][0].repeat_interleave(256)[:1000]
    for t in (m, v):
        assert torch.isnan(t[256:512]).all() and torch.isfinite(t[:256]).all() and torch.isfinite(t[512:]).all()
    ok = torch.ones(1000, dtype=torch.bool)
    ok[300] = False
    assert torch.isfinite(P[0].cpu()[ok]).all()


@pytest.mark.parametrize("count", [0, 1, 36, 37, 336, 337, 700])
def test_table_sizes(count):
    sizes = [(7 * j) % 611 + (5000 if j == 30 else 0) for j in range(count)]
    P, G, st = make(sizes, seed=52) if count else ([], [], {"step": torch.full((1,), 20, dtype=torch.int64, device="cuda"), "m": [], "v": []})
    plan = gbla.gbla_adamw_plan(P, G, st)
    want = [test64(f64(s), f64(m), f64(v), f64(g), 21, WD) for s, m, v, g in zip(P, st["m"], st["v"], G)]
    norm = gbla.gbla_grad_norm(plan)
    gbla.gbla_adamw_step(plan, LR, BETAS, EPS, WD, norm=norm)
    w = np.sqrt(sum((f64(g) ** 2).sum() for g in G))
    assert abs(float(norm) - w) <= 1.01 * E * w
    assert int(st["step"]) == 21
    for j, ((p, m, v), (bp, bm, bv)) in enumerate(want):
        assert (np.abs(f64(P[j]) - p) <= bp + E * np.abs(p)).all() and (np.abs(f64(st["m"][j]) - m) <= bm).all(), j


def test_norm_of_many_small_squares_and_wide_ranges():
    """2^24 equal squares (an fp32 sum would stop growing), and values from 1e-18 to 1e18."""
    g = [torch.full((1 << 24,), 0.3, device="cuda"), torch.tensor([1e-18, 1e18, 3.0], device="cuda")]
    for sel in ([0], [1], [0, 1]):
        G = [g[j] for j in sel]
        P = [torch.zeros_like(t) for t in G]
        n = gbla.gbla_grad_norm(gbla.gbla_adamw_plan(P, G, gbla.gbla_adamw_state(P)))
        w = np.sqrt(sum((f64(t) ** 2).sum() for t in G))
        assert abs(float(n) - w) <= 1.01 * E * w


def test_a_tensor_beyond_32_bits():
    """2^31 + 1000 values with 8-bit states, bf16 values and gradients: its last blocks bit for bit, the norm of all."""
    n, tail = 2 ** 31 + 1000, 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[n - tail:] = torch.linspace(-1, 1, tail, device="cuda").bfloat16()
    w = np.sqrt(2.0 ** 31 * 0.25 + (f64(g[n - tail:]) ** 2).sum())
    st = gbla.gbla_adamw_state([p], bits=8, master=False)
    plan = gbla.gbla_adamw_plan([p], [g], st)
    assert abs(float(gbla.gbla_grad_norm(plan)) - w) <= 1.01 * E * w
    gbla.gbla_adamw_step(plan, LR, seed=9)
    at = (n - tail) // 256 * 256  # 2^31: a block's first value
    gt = g[at:].float().cpu().numpy()
    c = [np.float32(v) for v in (1 - BETAS[0], 1 - BETAS[1])]
    m, root = c[0] * gt, np.sqrt((c[1] * gt) * gt)
    with np.errstate(over="ignore"):
        key = mix(mix(np.array([1 ^ 0x9E3779B9])) + np.uint32(9))
        z = mix((np.uint32(at) + np.arange(gt.size, dtype=np.uint32)) * np.uint32(0x9E3779B9) + key)
    for name, v, dither in (("m", m, z & np.uint32(0xFFFF)), ("v", root, z >> np.uint32(16))):
        code, scale = encode(v.astype(np.float32), dither, name == "v")
        assert np.array_equal(st[name][0][at:].view(torch.uint8).cpu().numpy(), code), name
        assert np.array_equal(st[name + "_scale"][0][at // 256:].cpu().numpy(), scale), name
    # the first step moves every value by lr against its gradient's sign
    assert (p[:2 ** 31:1 << 20].float() + LR).abs().max() <= LR * (2.0 ** -8 + 1e-5)
    del p, g, st, plan
    torch.cuda.empty_cache()


def test_writes_nothing_around_its_tensors():
    for bits in (8, 32):
        bufs = {k: torch.full((4, 600), 1, dtype=torch.uint8, device="cuda") for k in ("m", "v")} if bits == 8 else \
            {k: torch.ones(4, 600, device="cuda") for k in ("m", "v")}
        p, g = torch.ones(4, 600, device="cuda"), torch.ones(600, device="cuda")
        st = {"step": torch.ones(3, dtype=torch.int64, device="cuda")[1:2]}
        for k, t in bufs.items():
            st[k] = [t[2].view(torch.float8_e4m3fn) if bits == 8 else t[2]]
        if bits == 8:
            sc = {k: torch.ones(5, device="cuda") for k in ("m_scale", "v_scale")}
            st.update({k: [t[1:4]] for k, t in sc.items()})
        gbla.gbla_adamw_step(gbla.gbla_adamw_plan([p[2]], [g], st), LR)
        torch.cuda.synchronize()
        for t in [p, *bufs.values()]:
            assert (t[[0, 1, 3]] == 1).all()
        assert not (p[2] == 1).any()  # (m stays 1: 0.9 + 0.1)
        if bits == 8:
            assert all(float(t[0]) == 1 and float(t[4]) == 1 for t in sc.values())


@pytest.mark.parametrize("bits", [8, 32])
def test_deterministic_captured_and_on_other_streams(bits):
    def fresh():
        return make([300, 70000, 12], "bf16", bits=bits, seed=53, warm=False)

    def run(P, G, st, steps, how):
        plan = gbla.gbla_adamw_plan(P, G, st)
        go = lambda: gbla.gbla_adamw_step(plan, LR, norm=gbla.gbla_grad_norm(plan), max_norm=0.1, seed=3)  # noqa: E731
        if how == "graph":
            norm = torch.empty((), device="cuda")
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                gbla.gbla_grad_norm(plan, norm)
                gbla.gbla_adamw_step(plan, LR, norm=norm, max_norm=0.1, seed=3)
            for _ in range(steps):
                graph.replay()
        elif how == "stream":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for _ in range(steps):
                    go()
        else:
            for _ in range(steps):
                go()
        torch.cuda.synchronize()
        return [t.view(torch.uint8) for t in P + st["m"] + st["v"] + st["master"]] + [st["step"]]

    a, b, c = (run(*fresh(), 4, how) for how in ("plain", "stream", "graph"))
    assert int(a[-1]) == 4
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


def test_plan_refusals():
    P, G, st = make([100, 200], "bf16", bits=8, seed=54)
    plan = lambda p=P, g=G, **kw: gbla.gbla_adamw_plan(p, g, {**st, **kw})  # noqa: E731
    plan()
    for bad in (lambda: plan(p=[P[0], P[0]]), lambda: plan(p=[P[0]]), lambda: plan(g=G[:1]), lambda: plan(g=[G[0], G[1][:-1]]),
                lambda: plan(p=[P[0], P[1].half()]), lambda: plan(m=st["v"]), lambda: plan(m_scale=None), lambda: plan(m=st["m_scale"]),
                lambda: plan(p=[P[0].float(), P[1]]), lambda: plan(step=torch.zeros(1, device="cuda")), lambda: plan(g=[G[0], G[1].cpu()]),
                lambda: plan(v_scale=[st["v_scale"][0], st["v_scale"][1][:0]]), lambda: plan(g={"a": G[0], "b": G[1]}),
                lambda: plan(p=[P[0], torch.empty(200, 2, dtype=torch.bfloat16, device="cuda")[:, 0]])):
        with pytest.raises(ValueError):
            bad()
    q = plan()
    for kw in (dict(max_norm=1.0), dict(weight_decay=[0.1]), dict(norm=torch.zeros(2, device="cuda")), dict(norm=torch.zeros(()))):
        with pytest.raises(ValueError):
            gbla.gbla_adamw_step(q, LR, **kw)
    for kw in (dict(lr=-1.0), dict(lr=LR, betas=(1.0, 0.9)), dict(lr=LR, eps=0.0), dict(lr=LR, weight_decay=-1.0)):
        with pytest.raises(gbla.GblaError):
            gbla.gbla_adamw_step(q, **kw)
    assert int(st["step"]) == 0


# ----------------------------------------------------- a training step, whole
@pytest.mark.parametrize("bits", [8, 32])
def test_training_step_of_layer_and_recurrence(bits):
    """gbla_forward, then the recurrence over its output (projected into x | r | i), their backwards, the norm and the
    update of all parameters; gradients against the 64-bit layer and recurrence, the update against the formulas."""
    from generative_retrieval_encoder_gb300.workloads import Workload
    wl = Workload("train", 2, 150, 64, 1, 64, backward=True, seed=60)
    B, L, d = 2, 150, 64
    shape, rs = gbla.make_shape(B, L, d, 1, 64), gbla.glr_shape(B, L, 64)
    x = wl.x().bfloat16().cuda()
    gen = torch.Generator().manual_seed(61)
    P = {k: t.bfloat16().cuda() for k, t in wl.params().items()}
    P["W_glr"] = (torch.randn(64, 192, generator=gen) / 8).bfloat16().cuda()
    P["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(64, generator=gen)) / 8)).cuda()
    dy = torch.randn(B * L, 64, generator=gen).bfloat16().cuda()
    st = gbla.gbla_adamw_state(P, bits=bits)
    plan = None
    for t in range(1, 4):
        y, saved = gbla.gbla_forward(shape, x, P, saved=True)
        xri = y @ P["W_glr"]
        z, _, s2 = gbla.glr_forward(rs, xri[:, :64], xri[:, 64:128], xri[:, 128:], P["lam"], saved=True)
        dxri = torch.empty_like(xri)
        out = {"dx": dxri[:, :64], "dr": dxri[:, 64:128], "di": dxri[:, 128:], "dlam": torch.empty(64, device="cuda")}
        gbla.glr_backward(rs, xri[:, :64], xri[:, 64:128], xri[:, 128:], P["lam"], s2, dy, out=out)
        grads = gbla.gbla_backward(shape, x, P, saved, dxri @ P["W_glr"].t())
        grads.update(W_glr=(y.float().t() @ dxri.float()), dlam=out["dlam"])
        if t == 1:  # the gradients, each side on the values that the other hands it
            starts, lens = [0, L], [L, L]
            want = reference(f64(xri[:, :64]), f64(xri[:, 64:128]), f64(xri[:, 128:]), f64(P["lam"]), 8.0, starts, lens, dy=f64(dy))
            check({"y": z, **{k: v for k, v in out.items()}}, want)
            o_st, o_ln = oracle.seqs(B, L)
            Pr = {k: f64(P[k]) for k in gbla.PARAMS}
            ref = oracle.gbla_backward(f64(x), Pr, f64(dxri @ P["W_glr"].t()), 1, 64, o_st, o_ln)
            for k in ("dx", "dW_q", "dconv_w", "drms_w"):
                assert np.abs(f64(grads[k]).reshape(ref[k].shape) - ref[k]).max() <= 2e-2 * np.abs(ref[k]).max(), k
        if plan is None:
            plan = gbla.gbla_adamw_plan(P, grads, st)
        else:
            plan.set_grads(grads)
        norm = gbla.gbla_grad_norm(plan)
        G = {k: f64(grads["d" + k] if "d" + k in grads else grads[k]).ravel() for k in P}
        w = np.sqrt(sum((v ** 2).sum() for v in G.values()))
        assert abs(float(norm) - w) <= 1.01 * E * w
        src = [f64(m if m is not None else p).ravel() for m, p in zip(st["master"], P.values())]
        val = lambda k, j: f64(st[k][j]) if bits == 32 else f64(st[k][j].float() * st[k + "_scale"][j].repeat_interleave(256)[:st[k][j].numel()])  # noqa: E731
        want = [test64(src[j], val("m", j), val("v", j) ** (1 if bits == 32 else 2), G[k], t, WD, min(1.0, 1.0 / (w + 1e-6)))
                for j, k in enumerate(P)]
        gbla.gbla_adamw_step(plan, LR, BETAS, EPS, WD, norm=norm, max_norm=1.0, seed=t)
        for j, (k, p) in enumerate(P.items()):
            got = f64(st["master"][j] if st["master"][j] is not None else p).ravel()
            assert (np.abs(got - want[j][0][0]) <= want[j][1][0] + E * np.abs(want[j][0][0])).all(), (t, k)
    assert int(st["step"]) == 3


def test_states_and_types_mixed_in_one_plan():
    """Every tensor its own types, states and alignment: each the bits it gets in a plan of its kind, at the same place."""
    kinds = [("f32", "f32", 32, 0), ("bf16", "bf16", 8, 0), ("f32", "bf16", 8, 1), ("bf16", "f32", 32, 3)]
    sizes = [300, 2500, 256, 1]
    alone = [make(sizes, p, g, bits=b, offset=o, seed=90 + k) for k, (p, g, b, o) in enumerate(kinds)]
    mixed = [make(sizes, p, g, bits=b, offset=o, seed=90 + k) for k, (p, g, b, o) in enumerate(kinds)]
    state = {"step": torch.full((1,), 20, dtype=torch.int64, device="cuda")}
    for name in ("m", "v", "m_scale", "v_scale", "master"):
        state[name] = [(mixed[j % 4][2].get(name) or [None] * 4)[j] for j in range(4)]
    plan = gbla.gbla_adamw_plan([mixed[j][0][j] for j in range(4)], [mixed[j][1][j] for j in range(4)], state)
    gbla.gbla_adamw_step(plan, LR, BETAS, EPS, WD, seed=3)
    places = np.concatenate([[0], np.cumsum([-(-n // 256) * 256 for n in sizes])])
    for j, (P, G, st) in enumerate(alone):
        st["step"].fill_(20)
        # tensors of other kinds before it take its blocks' places
        lead = torch.zeros(int(places[j]), device="cuda")
        one = {"step": st["step"]}
        pad = gbla.gbla_adamw_state([lead], bits=32)
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            one[name] = [(pad.get(name) or [None])[0], (st.get(name) or [None] * 4)[j]]
        gbla.gbla_adamw_step(gbla.gbla_adamw_plan([lead, P[j]], [torch.zeros_like(lead), G[j]], one), LR, BETAS, EPS, WD, seed=3)
        assert torch.equal(plan._keep[0][j], P[j]), j
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            a, b = state[name][j], one[name][1]
            assert (a is None) == (b is None) and (a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))), (j, name)
    assert int(state["step"]) == 21


def test_norm_reads_the_gradients_alone():
    g = torch.randn(5000, device="cuda")
    t = (gbla.AdamWTensor * 2)()
    for k, (at, n) in enumerate(((g, 3001), (g[3001:], 1999))):
        t[k].grad, t[k].n, t[k].grad_dtype = at.data_ptr(), n, gbla.GBLA_F32
    ws = torch.empty(gbla.lib().gbla_adamw_workspace_size(t, 2), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    assert gbla.lib().gbla_grad_norm(t, 2, norm.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    want = float(g.double().norm())
    assert abs(float(norm) - want) <= 2 * E * want  # the sum is good to 2^-40; one rounding of the root


def test_8bit_codes_of_small_values_bit_for_bit():
    """Blocks whose values spread over many powers of two: half of them are below the smallest normal code, where a last bit of
    the quotient decides once in some million values."""
    n = 1 << 24
    gen = torch.Generator().manual_seed(95)
    g = (torch.randn(n, generator=gen) * torch.exp(4 * torch.randn(n, generator=gen)) * 1e-4).cuda()
    P = [torch.zeros(n, device="cuda")]
    st = gbla.gbla_adamw_state(P, bits=8)
    zero, scale = np.zeros(n, np.uint8), np.zeros(n // 256, np.float32)
    codes, scales, (m, root) = step8((zero, zero), (scale, scale), g.cpu().numpy(), 1, 0, 77)
    for x, s in ((np.abs(m), scales[0]), (root, scales[1])):
        assert ((x < np.repeat(s, 256) * np.float32(2.0 ** -6)).mean() > 0.3)
    gbla.gbla_adamw_step(gbla.gbla_adamw_plan(P, [g], st), LR, BETAS, EPS, WD, seed=77)
    for k, name in enumerate(("m", "v")):
        assert np.array_equal(st[name + "_scale"][0].cpu().numpy(), scales[k]), name
        off = np.count_nonzero(st[name][0].view(torch.uint8).cpu().numpy() != codes[k])
        assert off == 0, f"{name}: {off} codes"


def test_norm_of_large_gradients_whose_squares_are_finite():
    """2048 squares of 1e38 each: a thread has eight of them, and four are over the fp32 range; the norm, 4.5e20, is not."""
    for g in (torch.full((2048,), 1e19, device="cuda"), torch.full((5000,), 1e19, device="cuda").bfloat16(),
              torch.cat([torch.full((3,), 1.8e19, device="cuda"), torch.randn(300000, device="cuda")])):
        P = [torch.zeros(g.numel(), device="cuda")]
        st = gbla.gbla_adamw_state(P)
        plan = gbla.gbla_adamw_plan(P, [g], st)
        norm = gbla.gbla_grad_norm(plan)
        w = np.sqrt((f64(g) ** 2).sum())
        assert abs(float(norm) - w) <= 1.01 * E * w  # one rounding
        gbla.gbla_adamw_step(plan, LR, norm=norm, max_norm=1.0)
        assert int(st["step"]) == 1


@pytest.mark.parametrize("bits", [8, 32])
def test_a_good_call_reports_ok(bits):
    P, G, st = make([300, 5000], bits=bits, seed=56)
    plan = gbla.gbla_adamw_plan(P, G, st)
    plan.ws.fill_(255)
    norm = gbla.gbla_grad_norm(plan)
    assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK
    plan.ws.fill_(255)
    gbla.gbla_adamw_step(plan, LR, norm=norm, max_norm=0.5)
    assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK
    G[0][7] = float("nan")
    gbla.gbla_adamw_step(plan, LR, norm=gbla.gbla_grad_norm(plan))  # skipped: no error either
    assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK


def test_norm_takes_no_other_field():
    """Whatever the other fields hold (addresses that are not even aligned, a NaN, no type): the same bits."""
    g = torch.randn(100003, device="cuda")
    norms = torch.zeros(2, device="cuda")
    for other in (0, 1):
        t = (gbla.AdamWTensor * 1)()
        t[0].grad, t[0].n, t[0].grad_dtype = g.data_ptr(), g.numel(), gbla.GBLA_F32
        if other:
            t[0].param, t[0].master, t[0].m, t[0].v, t[0].m_scale, t[0].v_scale = range(1, 13, 2)
            t[0].param_dtype, t[0].weight_decay = 9, float("nan")
        ws = torch.empty(gbla.lib().gbla_adamw_workspace_size(t, 1), dtype=torch.uint8, device="cuda")
        assert gbla.lib().gbla_grad_norm(t, 1, norms[other:].data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert norms[0] == norms[1]
    w = float(g.double().norm())
    assert abs(float(norms[0]) - w) <= 1.01 * E * w
