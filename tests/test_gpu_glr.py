"""The gated linear recurrence (glr_forward, glr_backward) against its formulas
in 64 bits (glr_cases): dense, padded and packed batches, both directions, with
and without a start state, odd widths and lengths from one token up, packed
projections, extreme logits, masked rows, pieces and single steps, streams and
graphs, bad sequence data."""
import numpy as np
import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla
from glr_cases import Case, check, reference, sigmoid, softplus

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gbla.lib()


CASES = [
    dict(dtype="bf16", d=64, L=1),
    dict(dtype="f32", d=1, L=1),
    dict(dtype="bf16", d=512, L=1, B=5),
    dict(dtype="f32", d=3, L=7, B=3, reverse=True),
    dict(dtype="bf16", d=130, L=63, B=2),
    dict(dtype="f32", d=64, L=64, B=2, packed=True),
    dict(dtype="bf16", d=72, L=65, B=3, reverse=True, state=False),
    dict(dtype="bf16", d=33, L=200, B=2, packed=True),
    dict(dtype="f32", d=66, L=129, B=2, seq_lens=[129, 1]),
    dict(dtype="bf16", d=64, L=300, B=5, seq_lens=[300, 0, 64, 1, 257], reverse=True),
    dict(dtype="f32", d=40, L=20, B=7, seq_lens=[20, 0, 1, 19, 2, 20, 5]),
    dict(dtype="f32", d=48, lengths=[5, 0, 300, 1, 64, 129, 0, 1000]),
    dict(dtype="bf16", d=64, lengths=[0, 0, 64, 64, 1, 1, 1, 61, 128, 2, 700, 0], reverse=True),
    dict(dtype="bf16", d=130, lengths=[1] * 150 + [3] * 40, state=False),
    dict(dtype="f32", d=8, lengths=[1], reverse=True),
    dict(dtype="bf16", d=64, L=2048, B=3),
    dict(dtype="f32", d=8, L=20000),                       # chunks of several levels of the scan
    dict(dtype="f32", d=8, L=20011, reverse=True, packed=True),
    dict(dtype="bf16", d=5, lengths=[17000, 3, 17500]),
    dict(dtype="f32", d=6, lengths=[3, 18000, 0, 1, 16400], reverse=True),
    dict(dtype="bf16", d=2040, lengths=[700, 0, 2500, 1, 128, 1300, 0, 3003]),  # packed sequences cut one by one
    dict(dtype="f32", d=1030, lengths=[129, 5000, 1, 0, 64, 3900, 2048], reverse=True),
]


def _id(c):
    return "-".join(f"{k}{len(v) if isinstance(v, list) else v}" for k, v in c.items())


@pytest.mark.parametrize("kw", CASES, ids=[_id(c) for c in CASES])
def test_glr_matches_formulas(kw):
    c = Case(seed=CASES.index(kw), **kw)
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    y2, _, _ = c.forward()  # inference: the same values
    torch.cuda.synchronize()
    want = c.reference()
    check({"y": y, "hT": hT, **g}, want)
    assert torch.equal(y, y2)
    pad = np.ones(c.T, bool)
    for a, n in zip(c.starts, c.lens):
        pad[a:a + n] = False
    pad = torch.from_numpy(pad).cuda()
    for t in (y, g["dx"], g["dr"], g["di"]):
        assert (t[pad] == 0).all()


def test_glr_without_optional_tensors_and_with_strided_outputs():
    c = Case("bf16", 96, L=150, B=3, state=False, seed=40)
    y, hT, saved = c.forward(saved=True)
    assert hT is None
    buf = torch.full((c.T, 3 * 96 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = {"dx": buf[:, :96], "dr": buf[:, 96:192], "di": buf[:, 192:288]}
    c.backward(saved, out=out)
    torch.cuda.synchronize()
    want = c.reference()
    check({"y": y, **out}, want)
    assert (buf[:, 288:] == 7).all()


def test_glr_writes_nothing_around_its_outputs():
    c = Case("f32", 33, lengths=[70, 0, 5, 129], seed=41)
    T, d, n = c.T, c.d, c.n
    guard = lambda r: torch.full((r + 2, d), 5.0, device="cuda")  # noqa: E731
    y, hT, dx, dr, di, dh0 = guard(T), guard(n), guard(T), guard(T), guard(T), guard(n)
    dlam = torch.full((3, d), 5.0, device="cuda")
    saved = torch.full((gbla.glr_saved_size(c.shape) + 512,), 9, dtype=torch.uint8, device="cuda")
    ws_f = torch.full((gbla.gbla_workspace_size(c.shape, gbla.GBLA_OP_GLR_FORWARD) + 256,), 9, dtype=torch.uint8, device="cuda")
    ws_b = torch.full((gbla.gbla_workspace_size(c.shape, gbla.GBLA_OP_GLR_BACKWARD) + 256,), 9, dtype=torch.uint8, device="cuda")
    c.forward(y=y[1:-1], hT=hT[1:-1], saved=saved[:-512], ws=ws_f[:-256])
    c.backward(saved[:-512], ws=ws_b[:-256], out={"dx": dx[1:-1], "dr": dr[1:-1], "di": di[1:-1], "dh0": dh0[1:-1], "dlam": dlam[1]})
    torch.cuda.synchronize()
    check({"y": y[1:-1], "hT": hT[1:-1], "dx": dx[1:-1], "dr": dr[1:-1], "di": di[1:-1], "dh0": dh0[1:-1], "dlam": dlam[1]}, c.reference())
    for t in (y, hT, dx, dr, di, dh0, dlam):
        assert (t[0] == 5).all() and (t[-1] == 5).all()
    assert (saved[-512:] == 9).all() and (ws_f[-256:] == 9).all() and (ws_b[-256:] == 9).all()


@pytest.mark.parametrize("reverse", [False, True])
def test_glr_padded_rows_may_hold_anything(reverse):
    """Infinities, NaN and the type's lowest value in rows of no sequence reach nothing."""
    c = Case("bf16", 64, L=100, B=4, seq_lens=[0, 37, 100, 64], reverse=reverse, seed=42)
    want = c.reference()
    for b, n in enumerate(c.lens):
        for t, bad in ((c.x, float("nan")), (c.r, float("inf")), (c.i, torch.finfo(torch.bfloat16).min), (c.dy, float("-inf"))):
            t[b * 100 + n:(b + 1) * 100] = bad
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    torch.cuda.synchronize()
    check({"y": y, "hT": hT, **g}, want)


def test_glr_a_sequence_with_nan_leaves_the_others_alone():
    lens = [100, 700, 3, 150]
    c = Case("f32", 16, lengths=lens, seed=43)
    want = c.reference()
    c.x[150] = float("nan")   # in sequence 1
    c.h0[1] = float("inf")
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    torch.cuda.synchronize()
    keep = [t for b in (0, 2, 3) for t in range(c.starts[b], c.starts[b] + lens[b])]
    for n, t in {"y": y, "dx": g["dx"], "dr": g["dr"], "di": g["di"]}.items():
        check({n: t[keep]}, {n: tuple(w[keep] for w in want[n])})
    for n, t in {"hT": hT, "dh0": g["dh0"]}.items():
        check({n: t[[0, 2, 3]]}, {n: tuple(w[[0, 2, 3]] for w in want[n])})
    assert torch.isnan(y[799]).all() and torch.isnan(hT[1]).all()


def test_glr_extreme_logits_and_decays():
    """r = -inf keeps the state, r = +inf and +-1e4 saturate; lam from -200 (no decay) to 50 (no memory)."""
    d = 24
    lam = torch.cat([torch.linspace(-200, 50, 12), torch.linspace(-12, 3, 12)])
    c = Case("f32", d, L=130, seed=44, lam=lam)
    big = torch.tensor([-1e4, -80.0, -30.0, 30.0, 1e4, 0.0], device="cuda")
    c.r[10:16] = big[:, None]
    c.i[40:46] = big[:, None]
    c.r[100] = float("-inf")
    c.r[101] = float("inf")
    c.i[102] = float("-inf")
    c.i[103] = float("inf")
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    torch.cuda.synchronize()
    assert torch.equal(y[100], y[99])
    want = c.reference()
    # sigmoids below 2^-126 are 0 in the kernels: absolute, far below any output here
    check({"y": y, "hT": hT, **g}, want, floor=1e-18)


def test_glr_in_pieces_and_in_place_steps():
    """Prefill in pieces and then token by token, the state updated in place: the whole sequence's outputs."""
    B, L, d = 3, 210, 40
    c = Case("f32", d, L=L, B=B, seed=45)
    want = c.reference(backward=False)
    h = c.h0.clone()
    at, out = 0, []
    cut = lambda t, a, n: t.view(B, L, d)[:, a:a + n].reshape(B * n, d).contiguous()  # noqa: E731
    for n in [130, 64] + [1] * 16:
        sh = gbla.glr_shape(B, n, d, dtype="f32")
        y, hT, _ = gbla.glr_forward(sh, cut(c.x, at, n), cut(c.r, at, n), cut(c.i, at, n), c.lam, h0=h, hT=h)
        assert hT is h
        out.append(y.view(B, n, d))
        at += n
    torch.cuda.synchronize()
    check({"y": torch.cat(out, 1).reshape(B * L, d), "hT": h}, want)


@pytest.mark.parametrize("d,lengths", [(72, None), (72, [100, 0, 5000, 1, 63]), (1024, [0, 3000, 100, 6000, 1])])
def test_glr_long_state_in_place(d, lengths):
    kw = dict(lengths=lengths) if lengths else dict(L=1500, B=3)
    c = Case("bf16", d, seed=46, reverse=True, **kw)
    want = c.reference(backward=False)
    y, hT, _ = gbla.glr_forward(c.shape, c.x, c.r, c.i, c.lam, reverse=True, h0=c.h0, hT=c.h0)
    torch.cuda.synchronize()
    assert hT is c.h0
    check({"y": y, "hT": hT}, want)


def test_glr_gradients_by_differences():
    """<dy, y> + <dhT, hT> of the formulas (64 bits) moved by each input, against the kernel's gradients."""
    c = Case("f32", 4, lengths=[7, 0, 70], seed=47, reverse=True)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    A = {k: f(getattr(c, k)) for k in ("x", "r", "i", "lam", "h0")}

    def loss(**kw):
        v = {**A, **kw}
        o = reference(v["x"], v["r"], v["i"], v["lam"], 8.0, c.starts, c.lens, True, v["h0"], io="f32")
        return float((o["y"][0] * f(c.dy)).sum() + (o["hT"][0] * f(c.dhT)).sum())

    _, _, saved = c.forward(saved=True)
    g = c.backward(saved)
    rng = np.random.default_rng(3)
    for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("h0", "dh0")):
        got = f(g[grad])
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in A[name].shape)
            up, dn = A[name].copy(), A[name].copy()
            e = 1e-5
            up[at] += e
            dn[at] -= e
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * e)
            # central differences in 64 bits: e^2 of the third derivative and 1e-16 / e of the loss; the kernel fp32
            assert abs(got[at] - num) <= 1e-4 * max(1.0, abs(num)), (name, at, got[at], num)


def test_glr_is_deterministic_on_streams_and_in_graphs():
    c = Case("bf16", 256, L=4096, B=4, seed=48)
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for s in (s1, s2):  # two calls at once, each with its own workspaces
        with torch.cuda.stream(s):
            a = c.forward(hT=True, saved=True)
            res.append((a, c.backward(a[2])))
    torch.cuda.synchronize()
    for a, b in res:
        assert torch.equal(a[0], y) and torch.equal(a[1], hT)
        assert all(torch.equal(b[k], g[k]) for k in g)
    # captured and replayed with new inputs in the same buffers
    yb, hb, sb = torch.empty_like(y), torch.empty_like(hT), torch.empty_like(saved)
    gb = {k: torch.empty_like(v) for k, v in g.items()}
    ws = [gbla.workspace(c.shape, op) for op in (gbla.GBLA_OP_GLR_FORWARD, gbla.GBLA_OP_GLR_BACKWARD)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(y=yb, hT=hb, saved=sb, ws=ws[0])
        c.backward(sb, out=gb, ws=ws[1])
    for k in range(3):
        c.x.add_(0.25)
        graph.replay()
        a = c.forward(hT=True, saved=True)
        b = c.backward(a[2])
        torch.cuda.synchronize()
        assert torch.equal(a[0], yb) and torch.equal(a[1], hb) and all(torch.equal(b[n], gb[n]) for n in b)


@pytest.mark.parametrize("form", ["dense", "varlen", "steps"])
def test_glr_offsets_beyond_32_bits(form):
    """2.2e9 values (offsets in elements and bytes pass 2^31 and 2^32): the last sequence against the formulas, one tensor
    serving as x, r and i."""
    d, L = 2048, 1024 if form != "steps" else 4
    B = (2 ** 31 + 2 ** 27) // (d * L)
    T = B * L
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(70))
    lam = torch.log(torch.expm1(-torch.log(torch.linspace(0.9, 0.999, d)) / 8)).cuda()
    cu = torch.arange(0, T + 1, L, dtype=torch.int32, device="cuda")
    sh = gbla.glr_shape(1, T, d, cu_seqlens=cu) if form == "varlen" else gbla.glr_shape(B, L, d)
    y, hT, saved = gbla.glr_forward(sh, x, x, x, lam, hT=True, saved=True if form != "steps" else None)
    v = x[T - L:].double().cpu().numpy()
    want = reference(v, v, v, lam.double().cpu().numpy(), 8.0, [0], [L], dy=v)
    check({"y": y[T - L:], "hT": hT[B - 1:]}, want)
    del y
    if form == "steps":
        return
    g = gbla.glr_backward(sh, x, x, x, lam, saved, x)
    check({n: g[n][T - L:] for n in ("dx", "dr", "di")}, want)
    del g, saved, x
    torch.cuda.empty_cache()


def test_glr_bad_sequence_data_is_reported():
    """cu_seqlens that decrease or end elsewhere, seq_lens over L: nothing is written, the status says so."""
    d, T = 16, 100
    x = torch.randn(T, d, device="cuda")
    lam = torch.zeros(d, device="cuda")
    for kw in ({"cu_seqlens": [0, 60, 40, 100]}, {"cu_seqlens": [0, 60, 99]}, {"cu_seqlens": [1, 60, 100]},
               {"cu_seqlens": [0, 1 << 30, 100]}, {"cu_seqlens": [0, -5, 100]}, {"seq_lens": [51, 3]}, {"seq_lens": [-1, 3]}):
        t = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in kw.items()}
        B, L = (1, T) if "cu_seqlens" in kw else (2, 50)
        sh = gbla.glr_shape(B, L, d, dtype="f32", **t)
        ws = gbla.workspace(sh, gbla.GBLA_OP_GLR_FORWARD)
        y = torch.full((T, d), 3.0, device="cuda")
        saved = torch.zeros(gbla.glr_saved_size(sh), dtype=torch.uint8, device="cuda")
        gbla.glr_forward(sh, x, x, x, lam, y=y, ws=ws, saved=saved)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK, kw
        assert (y == 3).all()
        ws = gbla.workspace(sh, gbla.GBLA_OP_GLR_BACKWARD)
        out = {n: torch.full((T, d), 3.0, device="cuda") for n in ("dx", "dr", "di")}
        gbla.glr_backward(sh, x, x, x, lam, saved, x, ws=ws, out=out)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK, kw
        assert all((t == 3).all() for t in out.values())


def test_glr_bad_sequence_data_of_long_sequences_is_reported():
    """The same where packed sequences are cut one by one."""
    d, T = 1024, 8192
    x = torch.randn(T, d, device="cuda").bfloat16()
    lam = torch.zeros(d, device="cuda")
    for cu in ([0, 5000, 4000, T], [0, 5000, T - 1], [0, 1 << 30, T], [0, -5, T], [2, 5000, T]):
        sh = gbla.glr_shape(1, T, d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        ws = gbla.workspace(sh, gbla.GBLA_OP_GLR_FORWARD)
        y = torch.full_like(x, 3.0)
        saved = torch.zeros(gbla.glr_saved_size(sh), dtype=torch.uint8, device="cuda")
        gbla.glr_forward(sh, x, x, x, lam, y=y, ws=ws, saved=saved)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK, cu
        ws = gbla.workspace(sh, gbla.GBLA_OP_GLR_BACKWARD)
        out = {n: torch.full_like(x, 3.0) for n in ("dx", "dr", "di")}
        gbla.glr_backward(sh, x, x, x, lam, saved, x, ws=ws, out=out)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK, cu
        assert (y == 3).all() and all((t == 3).all() for t in out.values())


def test_glr_good_call_reports_ok_and_checks_its_arguments():
    c = Case("f32", 16, L=100, B=2, seed=49)
    ws = gbla.workspace(c.shape, gbla.GBLA_OP_GLR_FORWARD)
    c.forward(ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    call = lambda **kw: gbla.glr_forward(c.shape, **{**dict(x=c.x, r=c.r, i=c.i, lam=c.lam, h0=c.h0), **kw})  # noqa: E731
    for bad in (dict(x=c.x[:-1]), dict(r=c.r.bfloat16()), dict(i=c.i.cpu()), dict(lam=c.lam[:-1]), dict(lam=c.lam.double()),
                dict(h0=c.h0[:1]), dict(r=torch.cat([c.r, c.r], 1)[:, :16]), dict(x=c.x.t().contiguous().t()),
                dict(y=torch.empty(200, 17, device="cuda")[:, :16]), dict(hT=torch.empty(3, 16, device="cuda")),
                dict(saved=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(gbla.GblaError):
        call(ws=ws[:-1])
    with pytest.raises(gbla.GblaError):
        call(c=0.0)
    with pytest.raises(ValueError):
        gbla.glr_shape(2, 100, 16, dtype="f32", seq_lens=torch.ones(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("form", ["padded", "stream", "seqs"])
def test_glr_bad_sequence_data_leaves_every_output(form):
    """The outputs that are sums or states too (dlam, hT, dh0) keep what they held."""
    d, T = (1024, 8192) if form == "seqs" else (16, 2400)
    bad = torch.tensor([T // 2 + 1, 3] if form == "padded" else [0, T // 2, T - 1], dtype=torch.int32, device="cuda")
    sh = gbla.glr_shape(2, T // 2, d, seq_lens=bad) if form == "padded" else gbla.glr_shape(1, T, d, cu_seqlens=bad)
    x = torch.randn(T, d, device="cuda").bfloat16()
    lam, h0, kept = torch.zeros(d, device="cuda"), torch.ones(2, d, device="cuda"), torch.full((2, d), 3.0, device="cuda")
    ws, y, saved = gbla.workspace(sh, gbla.GBLA_OP_GLR_FORWARD), torch.full_like(x, 3.0), torch.full((gbla.glr_saved_size(sh),), 3, dtype=torch.uint8, device="cuda")
    gbla.glr_forward(sh, x, x, x, lam, h0=h0, y=y, hT=kept, saved=saved, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
    assert (kept == 3).all() and (y == 3).all() and (saved == 3).all()
    ws = gbla.workspace(sh, gbla.GBLA_OP_GLR_BACKWARD)
    out = {n: torch.full((T, d), 3.0, device="cuda", dtype=torch.bfloat16) for n in ("dx", "dr", "di")}
    out["dlam"], out["dh0"] = torch.full((d,), 3.0, device="cuda"), kept
    gbla.glr_backward(sh, x, x, x, lam, saved, x, h0=h0, dhT=h0, out=out, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
    for n, t in out.items():
        assert (t == 3).all(), n


@pytest.mark.parametrize("form", ["padded", "stream", "seqs"])
def test_glr_captured_call_follows_its_sequence_data(form):
    """Lengths are read on the device: a replay with others in the same tensor gives what a call with those gives."""
    d, T = (1024, 8192) if form == "seqs" else (48, 2400)
    n = 3
    sets = [[800, 0, 17], [1, 799, 800], [0, 0, 64]] if form == "padded" else \
        [[0, T // 3, T // 2, T], [0, 0, 1, T], [0, T, T, T], [0, 100, 164, T]]
    at = torch.tensor(sets[0], dtype=torch.int32, device="cuda")
    sh = gbla.glr_shape(n, T // n, d, seq_lens=at) if form == "padded" else gbla.glr_shape(1, T, d, cu_seqlens=at)
    gen = torch.Generator("cuda").manual_seed(71)
    x, r, i, dy = (torch.randn(T, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    lam = torch.full((d,), -4.0, device="cuda")
    h0, dhT = (torch.randn(n, d, generator=gen, device="cuda") for _ in range(2))

    def run():
        y, hT, saved = gbla.glr_forward(sh, x, r, i, lam, h0=h0, hT=True, saved=True)
        return {"y": y, "hT": hT, **gbla.glr_backward(sh, x, r, i, lam, saved, dy, h0=h0, dhT=dhT)}

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for s in sets + sets[:1]:
        at.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for k, t in want.items():
            assert torch.equal(got[k], t), (s, k)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    starts, lens = ([0, 800, 1600], sets[0]) if form == "padded" else (sets[0][:-1], [b - a for a, b in zip(sets[0], sets[0][1:])])
    cols = slice(0, 48)  # (columns are independent)
    check({k: t[..., cols] for k, t in got.items()},
          reference(f(x)[:, cols], f(r)[:, cols], f(i)[:, cols], f(lam)[cols], 8.0, starts, lens, False, f(h0)[:, cols], f(dy)[:, cols], f(dhT)[:, cols]))


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lengths", [[100, 300, 200, 1, 1000, 7, 3000, 500], [3, 2, 1] * 700])
def test_glr_a_nan_decay_stays_in_its_sequence(lengths, reverse):
    """A gate that is NaN makes its sequence's decay NaN; what the tiles compose across a sequence's border is not."""
    c, clean = (Case("f32", 40, lengths=lengths, reverse=reverse, seed=80) for _ in range(2))
    bad = [1, 4, len(lengths) - 2]
    for b in bad:
        c.r[c.starts[b] + lengths[b] // 2] = float("nan")
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    y0, hT0, saved0 = clean.forward(hT=True, saved=True)
    g0 = clean.backward(saved0)
    torch.cuda.synchronize()
    rows = torch.ones(c.T, dtype=torch.bool, device="cuda")
    seqs = torch.ones(c.n, dtype=torch.bool, device="cuda")
    for b in bad:
        rows[c.starts[b]:c.starts[b] + lengths[b]] = False
        seqs[b] = False
    assert torch.isnan(hT[bad]).all() and torch.isnan(g["dlam"]).all()
    assert torch.equal(y[rows], y0[rows]) and torch.equal(hT[seqs], hT0[seqs]) and torch.equal(g["dh0"][seqs], g0["dh0"][seqs])
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][rows], g0[n][rows]), n


@pytest.mark.parametrize("reverse", [False, True])
def test_glr_a_nan_decay_of_long_slots_stays_in_its_channel(reverse):
    """A NaN gate and a NaN lam in chains of many tiles: the calls end, their channels alone are NaN."""
    c = Case("bf16", 72, L=3000, B=3, reverse=reverse, seed=81)
    want = c.reference()
    c.r[3000 + 1500, 5] = float("nan")  # sequence 1
    c.lam[8] = float("nan")
    ws = [gbla.workspace(c.shape, op) for op in (gbla.GBLA_OP_GLR_FORWARD, gbla.GBLA_OP_GLR_BACKWARD)]
    y, hT, saved = c.forward(hT=True, saved=True, ws=ws[0])
    g = c.backward(saved, ws=ws[1])
    assert all(gbla.gbla_check_device_status(w) == gbla.GBLA_OK for w in ws)
    ok = [ch for ch in range(72) if ch not in (5, 8)]
    check({n: t[..., ok] for n, t in {"y": y, "hT": hT, **g}.items()}, {n: tuple(w[..., ok] for w in v) for n, v in want.items()})
    for b in (0, 2):  # the other sequences' channel 5
        rows = slice(3000 * b, 3000 * b + 3000)
        check({n: t[rows, 5] for n, t in {"y": y, "dx": g["dx"], "dr": g["dr"], "di": g["di"]}.items()},
              {n: tuple(w[rows, 5] for w in want[n]) for n in ("y", "dx", "dr", "di")})
    assert torch.isnan(hT[1, 5]) and torch.isnan(hT[:, 8]).all() and torch.isnan(g["dlam"][[5, 8]]).all()


def _nonfinite(t):
    return (~torch.isfinite(t)).all()


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lam", [None, 0.0, 30.0], ids=["slow", "fast", "instant"])
@pytest.mark.parametrize("kw", [dict(dtype="f32", d=40, L=9001, B=2), dict(dtype="bf16", d=40, L=9001, B=2, seq_lens=[9001, 8700]),
                                dict(dtype="bf16", d=2056, lengths=[700, 9001, 600]), dict(dtype="f32", d=40, lengths=[9001] + [1, 5, 300] * 9)],
                         ids=["dense", "padded", "seqs", "stream"])
def test_glr_a_nonfinite_state_lasts_to_its_sequence_end(kw, lam, reverse):
    """A NaN or an infinity in h0, x or a gate, in dhT or dy, reaches every later row of its channel, however small the product of
    the decays in between is (it is 0 in fp32 over a tile, over some tiles, and in each row), and nothing else."""
    make = lambda: Case(seed=90, reverse=reverse, lam=None if lam is None else torch.full((kw["d"],), lam), **kw)  # noqa: E731
    c, clean = make(), make()
    b = 1 if "lengths" in kw and kw["d"] > 100 else 0  # the long sequence
    n, r0 = c.lens[b], c.starts[b]
    order = list(range(r0 + n - 1, r0 - 1, -1)) if reverse else list(range(r0, r0 + n))
    inf, nan = float("inf"), float("nan")
    c.h0[b, 3], c.h0[b, 5] = inf, nan
    c.x[order[3], 7], c.x[order[130], 9], c.r[order[3], 11] = nan, inf, nan
    first = {3: 0, 5: 0, 7: 3, 9: 130, 11: 3}
    y, hT, saved = c.forward(hT=True, saved=True)
    y0, hT0, saved0 = clean.forward(hT=True, saved=True)
    for ch, k in first.items():
        assert _nonfinite(y[order[k:], ch]) and _nonfinite(hT[b, ch]), ch
    ok = torch.ones_like(y, dtype=torch.bool)
    for ch, k in first.items():
        ok[order[k:], ch] = False
    okT = torch.ones_like(hT, dtype=torch.bool)
    okT[b, list(first)] = False
    assert torch.equal(y[ok], y0[ok]) and torch.equal(hT[okT], hT0[okT])
    # what comes from behind, on clean states
    g0 = clean.backward(saved0)
    clean.dhT[b, 13], clean.dhT[b, 15] = inf, nan
    clean.dy[order[-4], 17], clean.dy[order[-131], 19] = nan, inf
    last = {13: n, 15: n, 17: n - 3, 19: n - 130}
    g = clean.backward(saved0)
    ok = torch.ones_like(y, dtype=torch.bool)
    for ch, k in last.items():
        assert _nonfinite(g["dx"][order[:k], ch]) and _nonfinite(g["dr"][order[:k], ch]) and _nonfinite(g["dh0"][b, ch]), ch
        assert _nonfinite(g["dlam"][ch]), ch
        ok[order[:k], ch] = False
    okT = torch.ones_like(hT, dtype=torch.bool)
    okT[b, list(last)] = False
    for name in ("dx", "dr", "di"):
        assert torch.equal(g[name][ok], g0[name][ok]), name
    assert torch.equal(g["dh0"][okT], g0["dh0"][okT])
    rest = [ch for ch in range(c.d) if ch not in last]
    assert torch.equal(g["dlam"][rest], g0["dlam"][rest])


@pytest.mark.parametrize("dtype,B,L,d,step", [("bf16", 16, 1, 512, True), ("bf16", 16, 8, 512, True), ("f32", 16, 64, 512, False),
                                              ("bf16", 300, 2048, 512, False), ("f32", 150, 1024, 512, False), ("bf16", 512, 600, 512, False),
                                              ("bf16", 1024, 40, 512, True), ("f32", 600, 37, 500, True), ("f32", 4800, 20, 33, True)])
@pytest.mark.parametrize("reverse", [False, True])
def test_glr_dense_inference_by_the_faster_kernel(dtype, B, L, d, step, reverse):
    """Rows one after the other where those are few or the sequences many, tiles elsewhere (each of these sides is at least 1.3
    times the other's time away from the choice); the first, middle and last sequences against the formulas."""
    gen = torch.Generator("cuda").manual_seed(91)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, r, i = (torch.randn(B * L, d, generator=gen, device="cuda").to(dt) for _ in range(3))
    h0 = torch.randn(B, d, generator=gen, device="cuda")
    lam = torch.linspace(-5, 0, d, device="cuda")
    sh = gbla.glr_shape(B, L, d, dtype=dtype)
    gbla.gbla_profiling_read()
    gbla.gbla_profiling_enable(True)
    try:
        y, hT, _ = gbla.glr_forward(sh, x, r, i, lam, reverse=reverse, h0=h0, hT=True)
        names = [n for n, _ in gbla.gbla_profiling_read()]
    finally:
        gbla.gbla_profiling_enable(False)
    assert ("glr step" in names) == step and ("glr fwd" in names) != step, names
    assert torch.isfinite(y).all() and torch.isfinite(hT).all()
    cols = slice(0, min(d, 64))
    f = lambda t: t[..., cols].double().cpu().numpy()  # noqa: E731
    for b in sorted({0, B // 2, B - 1}):
        at = slice(b * L, b * L + L)
        check({"y": y[at, cols], "hT": hT[b:b + 1, cols]},
              reference(f(x[at]), f(r[at]), f(i[at]), f(lam), 8.0, [0], [L], reverse, f(h0[b:b + 1]), io=dtype))


def _spread(n, lo, hi, seed):
    """n lengths from lo to hi, odd ones among them, and an empty sequence at either end and in the middle."""
    v = np.random.default_rng(seed).integers(lo, hi + 1, n).tolist()
    v[0] = v[n // 2] = v[-1] = 0
    return v


@pytest.mark.parametrize("kw", [dict(dtype="bf16", d=1030, L=100, B=71), dict(dtype="f32", d=1028, L=65, B=110, reverse=True, packed=True),
                                dict(dtype="bf16", d=1032, L=257, B=30, reverse=True), dict(dtype="f32", d=1032, L=511, B=15),
                                dict(dtype="bf16", d=1032, L=200, B=40, seq_lens=_spread(40, 1, 200, 1)),
                                dict(dtype="f32", d=1032, L=129, B=60, seq_lens=_spread(60, 0, 129, 2), reverse=True),
                                dict(dtype="bf16", d=2040, lengths=_spread(60, 40, 300, 3)),
                                dict(dtype="f32", d=2040, lengths=_spread(20, 100, 900, 4), reverse=True),
                                dict(dtype="bf16", d=4104, lengths=_spread(140, 1, 128, 5), reverse=True)], ids=_id)
def test_glr_short_sequences_one_by_one(kw):
    """Calls of several rounds of tiles: slots and packed sequences from some 50 rows on are cut by themselves."""
    c = Case(seed=92, **kw)
    h = c.h0.clone()
    y, hT, saved = c.forward(hT=True, saved=True)
    g = c.backward(saved)
    names = {"y": y, "hT": hT, **g}
    y2, h2, _ = gbla.glr_forward(c.shape, c.x, c.r, c.i, c.lam, reverse=c.reverse, h0=h, hT=h)  # in place, nothing saved
    if "B" not in kw or "seq_lens" in kw:  # (dense: perhaps by the row-by-row kernel)
        assert torch.equal(y2, y) and torch.equal(h2, hT)
    cols = [0, 1, 63, 64, 65, c.d // 2, c.d - 3, c.d - 2, c.d - 1]  # (columns are independent)
    f = lambda t: t[..., cols].double().cpu().numpy()  # noqa: E731
    want = reference(f(c.x), f(c.r), f(c.i), f(c.lam), c.c, c.starts, c.lens, c.reverse, f(c.h0), f(c.dy), f(c.dhT), c.dtype)
    check({n: t[..., cols] for n, t in names.items()}, want)
    check({"y": y2[:, cols], "hT": h2[:, cols]}, want)
    pad = torch.ones(c.T, dtype=torch.bool)
    for a, n in zip(c.starts, c.lens):
        pad[a:a + n] = False
    for n in ("y", "dx", "dr", "di"):
        assert torch.isfinite(names[n]).all() and (names[n][pad.cuda()] == 0).all(), n


def test_glr_short_packed_sequences_follow_their_data():
    """A captured call of packed sequences cut one by one, replayed with other lengths, bad ones in between: those write nothing."""
    d, T, n = 2048, 8192, 24
    gen = torch.Generator("cuda").manual_seed(93)
    x, r, i, dy = (torch.randn(T, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    lam = torch.full((d,), -4.0, device="cuda")
    h0 = torch.randn(n, d, generator=gen, device="cuda")
    even = [T * k // n for k in range(n + 1)]
    good = [even, [0] * n + [T], [0] + [T] * n, sorted([0, T] + np.random.default_rng(6).integers(0, T, n - 1).tolist())]
    bad = [even[:5] + [even[7], even[6]] + even[7:], even[:-1] + [T - 1], [1] + even[1:], even[:3] + [1 << 30] + even[4:], even[:3] + [-7] + even[4:]]
    cu = torch.tensor(even, dtype=torch.int32, device="cuda")
    sh = gbla.glr_shape(1, T, d, cu_seqlens=cu)
    ws = [gbla.workspace(sh, op) for op in (gbla.GBLA_OP_GLR_FORWARD, gbla.GBLA_OP_GLR_BACKWARD)]

    def run(ws):
        y, hT, saved = gbla.glr_forward(sh, x, r, i, lam, h0=h0, hT=True, saved=True, ws=ws[0])
        return {"y": y, "hT": hT, **gbla.glr_backward(sh, x, r, i, lam, saved, dy, h0=h0, dhT=h0, ws=ws[1])}

    gbla.gbla_profiling_read()
    gbla.gbla_profiling_enable(True)
    try:
        run(ws)
        assert [k for k, _ in gbla.gbla_profiling_read()].count("glr order") == 2
    finally:
        gbla.gbla_profiling_enable(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ws)
    for k in range(5):
        cu.copy_(torch.tensor(bad[k], dtype=torch.int32))
        for t in got.values():
            t.fill_(3.0)
        graph.replay()
        assert all(gbla.gbla_check_device_status(w) == gbla.GBLA_ERR_DEVICE_CHECK for w in ws), k
        assert all((t == 3).all() for t in got.values()), k
        cu.copy_(torch.tensor(good[k % 4], dtype=torch.int32))
        graph.replay()
        assert all(gbla.gbla_check_device_status(w) == gbla.GBLA_OK for w in ws), k
        want = run([None, None])
        assert all(torch.equal(got[name], want[name]) for name in want), k
