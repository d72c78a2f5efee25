"""layer_norm_forward and layer_norm_backward against their formulas in 64 bits:
every type, widths from one value to rows that no group of threads holds, odd
and unaligned rows, strided inputs, with and without residual, scale and bias,
padded slots, far means, bad lengths, in-place updates, streams and graphs.

Bounds (none fitted; E = 2^-24, A = the most additions a value of a row's sum goes
through, 60 in groups, d / 256 + 60 in passes):
* s is one sum, rounded to fp32 and to the io type;
* mean: (A + 3) E mean |s|; a difference c = s - m: that and E |c|;
  variance: 2 dm mean |c| + dm^2 + (A + 5) E v, so r is off by half of it over
  v + eps, and 4 E; z = c r and y = z w + b add 2 E of each term;
* backward: z by 4 E |z| + 2 E |s - m| r from the saved statistics, g = dy w by E,
  the two means by (A + 8) E of their mean magnitudes, dx by 6 E of its terms;
* dw, db: (T + 100) E of the sum of magnitudes, each term 5 E;
* an output is rounded once: 2^-8 (bf16) or E (fp32) of its value."""
import numpy as np
import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": E}
TINY = 1e-36


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gbla.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().double().cpu().numpy()


def adds(d):
    return 60 if d <= 8192 else d // 256 + 60


def forward64(s, w, b, eps, half):
    """y and its bound, mean and r and theirs, of rows s as they are stored."""
    d = s.shape[1]
    m = s.mean(1, keepdims=True)
    c = s - m
    dm = (adds(d) + 3) * E * np.abs(s).mean(1, keepdims=True)
    v = (c ** 2).mean(1, keepdims=True)
    dv = 2 * dm * np.abs(c).mean(1, keepdims=True) + dm ** 2 + (adds(d) + 5) * E * v
    r = 1 / np.sqrt(v + eps)
    rel = np.minimum(dv / (2 * (v + eps)) * 1.1 + 4 * E, 1.0)
    z = c * r
    dz = np.abs(z) * (rel + 2 * E) + (dm + E * np.abs(c)) * r * (1 + rel)
    y = z * w + b
    by = np.abs(w) * dz + 2 * E * (np.abs(z * w) + np.abs(y)) + half * np.abs(y) + TINY
    return (y, by), (m, dm + E * np.abs(m) + TINY), (r, r * rel + TINY)


def backward64(s, w, st, dy, ds, half):
    d = s.shape[1]
    T = s.shape[0]
    m, r = st[:, :1], st[:, 1:]
    z = (s - m) * r
    bz = 4 * E * np.abs(z) + 2 * E * np.abs(s - m) * r
    g = dy * w
    c0, c1 = g.mean(1, keepdims=True), (g * z).mean(1, keepdims=True)
    b0 = (adds(d) + 8) * E * np.abs(g).mean(1, keepdims=True)
    b1 = (adds(d) + 8) * E * np.abs(g * z).mean(1, keepdims=True) + (np.abs(g) * bz).mean(1, keepdims=True)
    dx = r * (g - c0 - z * c1) + ds
    bx = r * (6 * E * (np.abs(g) + np.abs(c0) + np.abs(z * c1)) + b0 + np.abs(z) * b1 + np.abs(c1) * bz) + 3 * E * (np.abs(ds) + np.abs(dx)) \
        + half * np.abs(dx) + TINY
    dw, db = (dy * z).sum(0), dy.sum(0)
    bw = ((T + 100) * E + 5 * E) * np.abs(dy * z).sum(0) + (np.abs(dy) * bz).sum(0) + TINY
    bb = (T + 100) * E * np.abs(dy).sum(0) + TINY
    return {"dx": (dx, bx), "dw": (dw, bw), "db": (db, bb)}


def near(name, got, want):
    err = np.abs(f64(got) - want[0])
    assert np.isfinite(err).all(), name
    assert (err <= want[1]).all(), (name, (err - want[1]).max(), err.max())


def place(t, offset):
    b = torch.full((t.numel() + offset + 8,), 77, dtype=t.dtype, device="cuda")
    v = b[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    return v, b


def run(B, L, d, dtype="bf16", seq_lens=None, res=True, affine=True, cols=0, offset=0, eps=1e-5, mean=0.3, seed=0, inplace=None):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, g = B * L, gen(seed)
    x, _ = place((torch.randn(T, d + cols, generator=g) * 1.5 + mean).to(dt), offset)
    x = x[:, :d]
    mk = lambda *s, k=1.0, m=0.0: place((torch.randn(*s, generator=g) * k + m).to(dt), offset)[0]  # noqa: E731
    r = mk(T, d) if res else None
    w, b = (mk(d, k=0.3, m=1.0), mk(d, k=0.3)) if affine else (None, None)
    dy, ds = mk(T, d), (mk(T, d) if res else None)
    lens = None if seq_lens is None else torch.tensor(seq_lens, dtype=torch.int32, device="cuda")
    shape = gbla.glr_shape(B, L, d, dtype=dtype, seq_lens=lens)
    ws = gbla.layer_norm_workspace(shape, True)
    ws.fill_(0xA5)
    y, yb = place(torch.zeros(T, d, dtype=dt), offset)
    valid = np.ones(T, bool) if seq_lens is None else (np.arange(L)[None] < np.asarray(seq_lens)[:, None]).reshape(-1)
    s64 = f64(x)
    if res:
        s_want = (x.float() + r.float()).to(dt)
    total = None
    if inplace == "res":
        total = r
    elif inplace == "x":
        total = x
    y, total, stats = gbla.layer_norm_forward(shape, x, w, b, eps=eps, res=r, total=total, y=y, stats=True, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    if res:
        assert torch.equal(total, torch.where(torch.as_tensor(valid).cuda()[:, None], s_want, torch.zeros((), dtype=dt, device="cuda")))
        s64 = f64(s_want)
    else:
        assert total is None
    W, Bb = (f64(w), f64(b)) if affine else (np.ones(d), np.zeros(d))
    wy, wm, wr = forward64(s64[valid], W, Bb, eps, HALF[dtype])
    near("y", y[torch.as_tensor(valid)], wy)
    near("mean", stats[torch.as_tensor(valid)][:, :1], wm)
    near("r", stats[torch.as_tensor(valid)][:, 1:], wr)
    assert (y[torch.as_tensor(~valid)] == 0).all() and (stats[torch.as_tensor(~valid)] == 0).all()
    n = total if res else x
    dx, dxb = place(torch.zeros(T, d, dtype=dt), offset)
    ds64 = f64(ds) if res else np.zeros((T, d))
    out = {"dx": ds if inplace and res else dx}
    if affine:
        out["dw"], out["db"] = (torch.full((d,), 7.0, device="cuda") for _ in range(2))
    got = gbla.layer_norm_backward(shape, n, w, stats, dy, ds=ds, affine=affine, ws=ws, out=out)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    want = backward64(s64[valid], W, f64(stats)[valid], f64(dy)[valid], ds64[valid], HALF[dtype])
    near("dx", got["dx"][torch.as_tensor(valid)], want["dx"])
    assert (got["dx"][torch.as_tensor(~valid)] == 0).all()
    for k in ("dw", "db"):
        if affine:
            near(k, got[k], want[k])
    for buf, t in ((yb, y), (dxb, dx)):
        assert (buf[:offset] == 77).all() and (buf[offset + t.numel():] == 77).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 2), (5, 8), (40, 63), (33, 64), (17, 72), (20, 128), (9, 129), (700, 200), (31, 256), (12, 257), (1300, 512), (7, 520),
                                    (50, 1000), (5, 1024), (6, 1032), (3, 2048), (4, 2049), (3, 4096), (2, 4100), (5, 8192), (3, 8193), (20, 9000)])
def test_layer_norm_matches_formulas(dtype, rows, d):
    run(1, rows, d, dtype, seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("res,affine", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("d", [40, 384, 9001])
def test_layer_norm_without_optional_tensors(dtype, res, affine, d):
    run(3, 37, d, dtype, res=res, affine=affine, seed=d)


@pytest.mark.parametrize("dtype,d,cols,offset", [("bf16", 64, 64, 0), ("bf16", 64, 3, 0), ("bf16", 96, 0, 1), ("f32", 65, 0, 0), ("f32", 512, 512, 0), ("f32", 512, 0, 3),
                                                 ("bf16", 1001, 0, 0), ("bf16", 1000, 24, 5), ("f32", 8200, 1, 1)])
def test_layer_norm_rows_of_any_stride_and_alignment(dtype, d, cols, offset):
    run(2, 45, d, dtype, cols=cols, offset=offset, seed=d)
    run(2, 45, d, dtype, cols=cols, offset=offset, seed=d, res=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [48, 512, 777, 2000, 8300])
def test_layer_norm_padded_slots(dtype, d):
    run(5, 23, d, dtype, seq_lens=[23, 0, 1, 22, 9], seed=d)


@pytest.mark.parametrize("inplace", ["res", "x"])
@pytest.mark.parametrize("d", [64, 513, 1024, 8500])
def test_layer_norm_in_place(inplace, d):
    run(2, 30, d, "bf16", inplace=inplace, seed=d)
    run(2, 30, d, "f32", inplace=inplace, seed=d + 1, seq_lens=[30, 11])


@pytest.mark.parametrize("d", [64, 512, 2000, 8200])
def test_layer_norm_far_means_and_constant_rows(d):
    run(1, 40, d, "f32", mean=100.0, seed=d)
    shape = gbla.glr_shape(1, 4, d, dtype="f32")
    x = torch.full((4, d), 3.0, device="cuda")
    x[1] = 0
    x[2] = -1e30
    x[3] = 2.0 ** -100
    w, b = torch.ones(d, device="cuda"), torch.full((d,), 0.25, device="cuda")
    y, _, st = gbla.layer_norm_forward(shape, x, w, b, stats=True)
    # sums of equal values: off by A E of the value, so |z| <= 60 E |x| / sqrt(eps); a far constant has no variance beyond its rounding
    assert ((y[:2] - 0.25).abs() <= 64 * E * 3 / np.sqrt(1e-5) + E).all() and ((y[3] - 0.25).abs() <= 1e-6).all()
    assert torch.isfinite(st[[0, 1, 3]]).all()


@pytest.mark.parametrize("rows,d", [(60000, 1), (90000, 7), (60000, 30), (90000, 33), (45000, 57), (45000, 95), (45000, 100), (25000, 187), (12000, 250), (12000, 381),
                                    (8000, 505), (6000, 511), (6000, 766), (3500, 1001), (2500, 1530), (2500, 2041), (1500, 2900), (1500, 4001), (1000, 6001),
                                    (1000, 8001), (700, 8180), (3, 8185), (3, 8191)])
def test_layer_norm_many_rows_that_begin_anywhere(rows, d):
    """bf16 rows that are not whole pieces of 16 bytes, several to each of the groups of threads of a launch."""
    run(1, rows, d, "bf16", seed=d)


@pytest.mark.parametrize("d,cols", [(100, 8), (101, 16), (510, 24), (766, 8), (1001, 40), (2050, 8), (1001, 3)])
def test_layer_norm_strided_rows_that_begin_anywhere(d, cols):
    run(2, 700, d, "bf16", cols=cols, seed=d)
    run(2, 700, d, "bf16", cols=cols, seed=d, seq_lens=[650, 333], res=False)
    run(3, 450, d, "bf16", seed=d, seq_lens=[450, 0, 77], inplace="res")
    run(3, 450, d, "bf16", seed=d, seq_lens=[1, 450, 449], inplace="x")


@pytest.mark.parametrize("d", [1, 3, 101, 250, 511, 1530, 4001])
def test_layer_norm_a_row_of_nan_beside_rows_that_begin_anywhere(d):
    """What the pieces of a row hold of its neighbours counts for nothing, NaN and infinities among it."""
    T = 700
    shape = gbla.glr_shape(1, T, d)
    x, dy, ds = (torch.randn(T, d, generator=gen(d + k)).bfloat16().cuda() for k in range(3))
    w, b = torch.randn(d, generator=gen(9)).bfloat16().cuda(), torch.randn(d, generator=gen(8)).bfloat16().cuda()
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[1::3] = True
    want = {}
    for kind in (0.0, float("nan"), float("inf")):
        for t in (x, dy, ds):
            t[bad] = kind
        y, total, st = gbla.layer_norm_forward(shape, x, w, b, res=ds, stats=True)
        dx = gbla.layer_norm_backward(shape, total, w, st, dy, ds=ds)["dx"]
        for k, t in (("y", y), ("total", total), ("stats", st), ("dx", dx)):
            if kind == 0.0:
                want[k] = t[~bad].clone()
                assert torch.isfinite(want[k]).all(), k
            assert torch.equal(t[~bad], want[k]), (k, kind)


@pytest.mark.parametrize("d", [24, 32, 40, 88, 96, 104, 184, 192, 200, 320, 384, 392, 640, 768, 776, 1280, 1536, 1544, 2560, 4096, 4104, 5120, 6144, 6152, 8192])
def test_layer_norm_widths_of_every_group(d):
    run(1, 40 + 4000 // d, d, "bf16", seed=d)
    run(2, 1600000 // d // 8, d, "bf16", seed=d, res=False)


def test_layer_norm_padded_rows_may_hold_anything_and_nan_stays_in_its_row():
    B, L, d = 3, 16, 200
    lens = [16, 0, 5]
    valid = torch.as_tensor((np.arange(L)[None] < np.asarray(lens)[:, None]).reshape(-1))
    shape = gbla.glr_shape(B, L, d, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    g = gen(1)
    x, r, dy, ds = (torch.randn(B * L, d, generator=g).bfloat16() for _ in range(4))
    w, b = torch.randn(d, generator=g).bfloat16().cuda(), torch.randn(d, generator=g).bfloat16().cuda()

    def both(x, r, dy, ds):
        y, t, st = gbla.layer_norm_forward(shape, x.cuda(), w, b, res=r.cuda(), stats=True)
        return [y, t, st] + list(gbla.layer_norm_backward(shape, t, w, st, dy.cuda(), ds=ds.cuda()).values())
    a = both(x, r, dy, ds)
    wild = [torch.where(valid[:, None], t, torch.full_like(t, v)) for t, v in ((x, float("nan")), (r, float("inf")), (dy, float("nan")), (ds, float("-inf")))]
    for p, q in zip(a, both(*wild)):
        assert torch.equal(p, q)
    x[3] = float("nan")
    c = both(x, r, dy, ds)
    rows = torch.arange(B * L) != 3
    for p, q in zip(a[:4], c[:4]):
        assert torch.equal(p[rows], q[rows])
    assert c[0][3].isnan().all() and c[3][3].isnan().all() and torch.equal(a[5], c[5])


@pytest.mark.parametrize("dtype,T,d", [("bf16", 200000, 16), ("bf16", 90000, 33), ("bf16", 100001, 64), ("bf16", 60000, 512), ("bf16", 30000, 1000), ("bf16", 9000, 2048),
                                       ("bf16", 5000, 4095), ("bf16", 3001, 8192), ("bf16", 6000, 8190), ("bf16", 9001, 9000), ("f32", 100001, 24), ("f32", 60000, 200),
                                       ("f32", 30000, 511), ("f32", 9000, 2048), ("f32", 3000, 8192), ("f32", 4001, 8193)])
def test_layer_norm_column_sums_of_many_rows(dtype, T, d):
    """dw and db by the additions that a value goes through: a group's rows (of two CTAs an SM, 256 threads each), its CTA's groups,
    every 32nd CTA, a tree of 32; of rows that no group holds a 64th of the rows, two more partials, the tree."""
    f32 = dtype == "f32"
    wide = d if f32 else d + (0 if d % 8 == 0 else 4 if d % 4 == 0 else 6 if d % 2 == 0 else 7)
    if wide > 8192:
        chain = -(-T // 64) + 2 + 5
    else:
        threads = next(g for g in (4, 8, 16, 32, 64, 128, 256) if wide <= (32 if g == 256 else 8 if (f32 or wide <= 32) and g <= 32 else 16) * g)
        groups, sms = 256 // threads, torch.cuda.get_device_properties(0).multi_processor_count
        chain = -(-T // (2 * sms * groups)) + groups + -(-(2 * sms + 8) // 32) + 5
    dt = torch.float32 if f32 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(d)
    x, dy = ((torch.randn(T, d, generator=g, device="cuda") + 0.2).to(dt) for _ in range(2))
    shape = gbla.glr_shape(1, T, d, dtype=dtype)
    _, _, st = gbla.layer_norm_forward(shape, x, stats=True)
    got = gbla.layer_norm_backward(shape, x, None, st, dy)
    m, r = st[:, :1].double(), st[:, 1:].double()
    c = x.double() - m
    z, q = c * r, dy.double()
    bz = 4 * E * z.abs() + 2 * E * c.abs() * r
    for name, want, bound in (("dw", (q * z).sum(0), (chain + 2) * E * (q * z).abs().sum(0) + (q.abs() * bz).sum(0)),
                              ("db", q.sum(0), (chain + 2) * E * q.abs().sum(0))):
        err = (got[name].double() - want).abs()
        assert (err <= bound).all(), (name, (err / bound).max())


def test_layer_norm_bad_lengths_are_reported():
    for d in (64, 8300):
        for lens, bad in (([5, 9], 1), ([-1, 8], 0)):
            shape = gbla.glr_shape(2, 8, d, dtype="f32", seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
            x, dy = torch.randn(16, d, device="cuda"), torch.randn(16, d, device="cuda")
            ws = gbla.layer_norm_workspace(shape, True)
            y, _, st = gbla.layer_norm_forward(shape, x, stats=True, ws=ws)
            assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
            assert (y[8 * bad:8 * bad + 8] == 0).all() and (y[8 * (1 - bad):8 * (1 - bad) + 5] != 0).any()
            g = gbla.layer_norm_backward(shape, x, None, st, dy, ws=ws)
            assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
            assert (g["dx"][8 * bad:8 * bad + 8] == 0).all()
            good = gbla.glr_shape(2, 8, d, dtype="f32")
            gbla.layer_norm_forward(good, x, ws=ws)  # the next call's word is its own
            assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK


def test_layer_norm_of_many_slots():
    """More slots than one CTA checks: each reports its own length."""
    B, L, d = 9000, 2, 40
    ln = torch.randint(0, L + 1, (B,), generator=gen(4), dtype=torch.int32)
    for bad in (False, True):
        lens = ln.clone()
        if bad:
            lens[8999] = 3
        shape = gbla.glr_shape(B, L, d, dtype="f32", seq_lens=lens.cuda())
        x, dy = torch.randn(B * L, d, generator=gen(5)).cuda(), torch.randn(B * L, d, generator=gen(6)).cuda()
        ws = gbla.layer_norm_workspace(shape, True)
        ws.fill_(0xA5)
        y, _, st = gbla.layer_norm_forward(shape, x, stats=True, ws=ws)
        want = gbla.GBLA_ERR_DEVICE_CHECK if bad else gbla.GBLA_OK
        assert gbla.gbla_check_device_status(ws) == want
        g = gbla.layer_norm_backward(shape, x, None, st, dy, ws=ws)
        assert gbla.gbla_check_device_status(ws) == want
        valid = (torch.arange(L)[None] < torch.where(lens > L, 0, lens)[:, None]).view(-1)
        dense = gbla.glr_shape(1, B * L, d, dtype="f32")
        y2, _, st2 = gbla.layer_norm_forward(dense, x, stats=True)
        dy2 = torch.where(valid.cuda()[:, None], dy, 0.0)
        g2 = gbla.layer_norm_backward(dense, x, None, st2, dy2)
        assert torch.equal(y[valid], y2[valid]) and (y[~valid] == 0).all()
        assert torch.equal(g["dx"][valid], g2["dx"][valid]) and (g["dx"][~valid] == 0).all()
        # a row that counts for nothing adds exact zeros
        assert torch.equal(g["dw"], g2["dw"]) and torch.equal(g["db"], g2["db"])


def test_layer_norm_gradients_by_differences():
    T, d = 6, 20
    shape = gbla.glr_shape(1, T, d, dtype="f32")
    g = gen(9)
    x, r, dy, ds = (torch.randn(T, d, generator=g).cuda() for _ in range(4))
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    _, t, st = gbla.layer_norm_forward(shape, x, w, b, res=r, stats=True)
    got = gbla.layer_norm_backward(shape, t, w, st, dy, ds=ds)

    def f(x, w, b):
        y, t, _ = gbla.layer_norm_forward(shape, x, w, b, res=r)
        return float((y.double() * dy.double()).sum() + (t.double() * ds.double()).sum())
    h = 2.0 ** -6
    for name, t0, ref in (("dx", x, got["dx"]), ("dw", w, got["dw"]), ("db", b, got["db"])):
        for at in range(0, t0.numel(), 7):
            e = torch.zeros_like(t0).view(-1)
            e[at] = h
            e = e.view(t0.shape)
            p, m = [((x + k * e, w, b) if name == "dx" else (x, w + k * e, b) if name == "dw" else (x, w, b + k * e)) for k in (1, -1)]
            diff = (f(*p) - f(*m)) / (2 * h)
            # rounding 40 E of |f|'s terms (a few hundred) over 2 h; the second differences' h^2 / 6 times a third derivative below 60
            assert abs(diff - float(ref.view(-1)[at])) <= 40 * E * 300 / (2 * h) + h * h * 10, name


def test_layer_norm_offsets_beyond_32_bits():
    T, d = 1_100_000, 2048
    shape = gbla.glr_shape(1, T, d)
    x = torch.randn(4096, d, generator=gen(0)).bfloat16().cuda().repeat(-(-T // 4096), 1)[:T]
    st = torch.empty(T, 2, device="cuda")
    y, _, _ = gbla.layer_norm_forward(shape, x, stats=st)
    small = gbla.glr_shape(1, 4096, d)
    ys, _, ss = gbla.layer_norm_forward(small, x[:4096].contiguous(), stats=True)
    k = T // 4096
    assert torch.equal(y[(k - 1) * 4096:k * 4096], ys) and torch.equal(st[(k - 1) * 4096:k * 4096], ss) and torch.equal(y[:4096], ys)
    g = gbla.layer_norm_backward(shape, x, None, st, y, affine=False, out={"dx": torch.empty_like(x)})
    gs = gbla.layer_norm_backward(small, x[:4096].contiguous(), None, ss, ys, affine=False)
    assert torch.equal(g["dx"][(k - 1) * 4096:k * 4096], gs["dx"])


def test_layer_norm_on_streams_and_in_graphs():
    T, d = 3000, 512
    shape = gbla.glr_shape(1, T, d)
    g = gen(3)
    xs = [torch.randn(T, d, generator=g).bfloat16().cuda() for _ in range(2)]
    r, dy, ds = (torch.randn(T, d, generator=g).bfloat16().cuda() for _ in range(3))
    w, b = torch.randn(d, generator=g).bfloat16().cuda(), torch.randn(d, generator=g).bfloat16().cuda()
    ws = gbla.layer_norm_workspace(shape, True)

    def both(x, y=None, t=None, st=True, out=None):
        y, t, st = gbla.layer_norm_forward(shape, x, w, b, res=r, total=t, y=y, stats=st, ws=ws)
        return [y, t, st] + list(gbla.layer_norm_backward(shape, t, w, st, dy, ds=ds, ws=ws, out=out).values())
    want = [both(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(xs[0])
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(got, want[0]):
        assert torch.equal(p, q)  # the same bits again
    buf, mine = xs[0].clone(), [torch.empty_like(t) for t in want[0]]
    out = dict(zip(("dx", "dw", "db"), mine[3:]))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(buf, mine[0], mine[1], mine[2], out)
        graphs.append(graph)
    for k in (1, 0):
        buf.copy_(xs[k])
        for graph in graphs:
            for t in mine:
                t.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(mine, want[k]):
                assert torch.equal(p, q)
