"""beam_select and beam_reorder against their definition in 64 bits: both types,
odd and unaligned rows, masks (also over a whole row), ended, dead and identical
beams, ties, infinities and NaN, fewer candidates than beams, one to 1024 beams,
streams and graphs, states of every width moved in place and into others, a
decoding loop of embedding, norm, recurrence, selection and reordering, and a
training step of the same parts.

Order: the sum of a row's exponentials is off by 2^-27 at most (each by 2^-28.8; two
words, the lower of at most 0.011 of them through 7 additions on the mean), and so is its
logarithm.  So candidates of two beams may change places only where their scores
differ by less than 2 * 2^-27 (and 2^-46 of their size: two fp32 words); within a beam
never.  A score is rounded once: 2^-24 of its value beside that."""
import math

import numpy as np
import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
NEAR = 2.0 ** -26


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gbla.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def reference(logits, scores, V, n, allowed=None, done=None, eos=-1, over=False):
    """(B, K V) scores in 64 bits (-inf: no candidate) and each group's order of candidates, ties by place."""
    B, K = scores.shape
    x = logits.double().numpy().reshape(B, K, -1)[:, :, :V]
    ok = np.ones((B, K, V), bool) if allowed is None else allowed.reshape(B, K, V)
    s = np.where(ok, x, -np.inf) if over else x
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = np.max(np.where(np.isnan(s), -np.inf, s), axis=2, keepdims=True)
        base = np.where(np.isfinite(m), m, 0.0)
        log = np.log(np.exp(s - base).sum(2, keepdims=True))
        p = scores.double().numpy()[:, :, None] + ((x - base) - log)  # (of logits of 3e38 a sum with `base` would lose `log`)
    p = np.where(ok & (x > -np.inf), p, -np.inf)
    if done is not None:
        e = done.numpy()
        p[e] = -np.inf
        p[e, eos] = scores.double().numpy()[e]
    p = np.where(p > -np.inf, p, -np.inf).reshape(B, K * V)
    order = np.argsort(-p, axis=1, kind="stable")[:, :n]
    return p, order


def pack(ok):
    R, V = ok.shape
    bits = np.zeros((R, -(-V // 32) * 32), np.uint8)
    bits[:, :V] = ok
    w = np.packbits(bits.reshape(R, -1, 32), axis=2, bitorder="little").view(np.uint32).reshape(R, -1)
    return torch.from_numpy(w.astype(np.int64).astype(np.uint32).view(np.int32).copy())


def check(got, p, order, V, n, done=None, eos=-1, strict=True):
    sc, tok, par, dn = [None if t is None else t.cpu().numpy() for t in got]
    B = p.shape[0]
    for b in range(B):
        live = min(n, int((p[b] > -np.inf).sum()))
        assert (sc[b, live:] == -np.inf).all() and (tok[b, live:] == -1).all() and (par[b, live:] == 0).all()
        at = par[b, :live].astype(np.int64) * V + tok[b, :live]
        want = order[b, :live]
        assert len(set(at.tolist())) == live
        a, w = p[b, at], p[b, want]
        with np.errstate(invalid="ignore"):
            slack = NEAR + 2.0 ** -46 * np.abs(w)
            assert ((np.abs(a - w) <= slack) | (a == w)).all(), b
            assert ((np.abs(sc[b, :live] - a) <= NEAR + E * np.abs(a)) | (sc[b, :live] == a.astype(np.float32))).all()
        if strict:
            # (scores of -3e38, of logits of the type's lowest value: 64 bits hold no difference below 2^74 there, so -3e38 - 3 and
            # -3e38 - 6 tie in the reference; the second fp32 word holds it, and such candidates come in their true order)
            near = np.abs(w) < 2.0 ** 100
            assert (at == want)[near].all(), (b, np.flatnonzero(at != want)[:5])
        if dn is not None:
            old = np.zeros(par.shape[1], bool) if done is None else done[b].numpy()[par[b]]
            assert (dn[b, :live] == (old | (tok[b] == eos))[:live]).all() and not dn[b, live:].any()


def make(B, K, V, dtype="bf16", pad=0, offset=0, seed=0, std=2.0):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = gen(seed)
    x = (torch.randn(B * K, V + pad, generator=g) * std).to(dt)
    buf = torch.full((offset + x.numel() + 64,), float("nan"), dtype=dt, device="cuda")
    v = buf[offset:offset + x.numel()].view(B * K, V + pad)
    v.copy_(x)
    if pad:
        v[:, V:] = float("nan")  # the padding's columns are nobody's tokens
    scores = torch.sort(-5 * torch.rand(B, K, generator=g), dim=1, descending=True).values.contiguous()
    return v[:, :V], x[:, :V], scores


def run(B, K, V, n=None, dtype="bf16", mask=None, over=False, ends=0.0, eos=-1, strict=True, dead=(), **kw):
    n = K if n is None else n
    seed = B * 7 + K * 3 + V
    v, x, scores = make(B, K, V, dtype, seed=seed, **kw)
    for b, k in dead:
        scores[b, k] = -math.inf
    ok = None if mask is None else torch.rand(B * K, V, generator=gen(seed + 1)).numpy() < mask
    done = torch.rand(B, K, generator=gen(seed + 2)) < ends if ends else None
    beam = gbla.beam_shape(B, K, V, n, dtype=dtype, eos=eos, over_allowed=over)
    ws = gbla.beam_workspace(beam)
    ws.fill_(0xA5)
    got = gbla.beam_select(beam, v, scores.cuda(), allowed=None if ok is None else pack(ok).cuda(), done=None if done is None else done.cuda(), ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    p, order = reference(x, scores, V, n, ok, done, eos, over)
    check(got, p, order, V, n, done, eos, strict)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V,n", [(1, 1, 1, 1), (2, 1, 7, 3), (1, 8, 256, 8), (3, 5, 33, 5), (4, 1, 1000, 16), (2, 16, 2048, 16), (5, 7, 2049, 7), (2, 3, 40001, 20),
                                     (1, 256, 300, 256), (2, 50, 5000, 50), (1, 1024, 64, 1024), (1, 700, 90, 1000), (3, 2, 100, 1024), (1, 4, 130000, 512), (7, 4, 16384, 1)])
def test_beam_matches_definition(dtype, B, K, V, n):
    run(B, K, V, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V,n,pad,offset", [(1, 1, 131072, 1, 0, 0), (2, 4, 131072, 3, 0, 0), (2, 100, 20001, 2, 0, 0), (1, 64, 70000, 5, 3, 1), (3, 8, 100003, 16, 1, 0),
                                                (1, 300, 9000, 4, 8, 4), (1, 30, 65537, 60, 0, 3), (2, 2, 200000, 1, 7, 0)])
def test_beam_few_of_many(dtype, B, K, V, n, pad, offset):
    """Few beams of many candidates: runs of up to a warp's whole share of a row."""
    run(B, K, V, n, dtype, pad=pad, offset=offset)
    run(B, K, V, n, dtype, pad=pad, offset=offset, mask=0.01, over=K % 2 == 0, ends=0.2, eos=V - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (24, 7)])
@pytest.mark.parametrize("V", [5, 100, 4000])
def test_beam_rows_of_any_stride_and_alignment(dtype, pad, offset, V):
    run(2, 6, V, 6, dtype, pad=pad, offset=offset)
    run(2, 6, V, 6, dtype, pad=pad, offset=offset, mask=0.4, over=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("over", [False, True])
@pytest.mark.parametrize("K,V,mask", [(4, 100, 0.5), (16, 5000, 0.01), (256, 512, 0.02), (3, 31, 0.05), (5, 65, 0.0), (2, 20000, 0.001)])
def test_beam_masks(dtype, over, K, V, mask):
    run(3, K, V, K, dtype, mask=mask, over=over)
    run(3, K, V, K, dtype, mask=mask, over=over, ends=0.4, eos=V // 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beam_ended_and_dead_beams(dtype):
    run(4, 8, 500, 8, dtype, ends=0.5, eos=0)
    run(4, 8, 500, 8, dtype, ends=1.0, eos=499)           # every beam has ended: each goes on as itself
    run(4, 8, 500, 8, dtype, eos=3)                       # none has yet
    run(2, 6, 50, 6, dtype, dead=[(0, k) for k in range(1, 6)])  # a search that starts with copies of one beam
    run(2, 6, 50, 6, dtype, dead=[(1, k) for k in range(6)])     # a group without a live beam
    run(2, 6, 3, 6, dtype, dead=[(1, k) for k in range(5)], ends=0.2, eos=1)


def test_beam_ties_go_to_the_lowest_beam_and_token():
    for V, n in ((40, 16), (5000, 16), (300, 200)):
        beam = gbla.beam_shape(2, 16, V, n, dtype="f32")
        x = torch.zeros(32, V, device="cuda")
        sc, tok, par, _ = gbla.beam_select(beam, x, torch.zeros(2, 16, device="cuda"))
        want = torch.arange(n).repeat(2, 1)
        assert torch.equal(tok.cpu().long(), want % V) and torch.equal(par.cpu().long(), want // V)
        # three values, spread so that the equal ones lie in many runs and rows
        x = (torch.arange(32 * V).view(32, V) * 7919 % 3).float()
        x = torch.sort(x, dim=1).values[:, torch.randperm(V, generator=gen(V))]  # every row the same values: the same logarithm
        scores = torch.zeros(2, 16)
        got = gbla.beam_select(beam, x.cuda(), scores.cuda())
        p, order = reference(x, scores, V, n)
        top = p.max()
        flat = (got[2].long() * V + got[1]).cpu().numpy()
        for b in range(2):
            first = np.flatnonzero(np.abs(p[b] - top) < 1e-9)[:n]
            assert (flat[b, :len(first)] == first).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset", [(101, 0, 0), (255, 0, 0), (333, 1, 3), (1001, 0, 1), (2048, 1, 0), (5003, 0, 0), (5000, 3, 5), (40001, 0, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_beam_identical_beams_tie_wherever_their_rows_begin(dtype, V, pad, offset, masked):
    """Copies of one row with equal scores: the candidates of a token are exactly alike in all beams, and go by beam."""
    K, n = 24, 96
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for seed, std in ((1, 2.0), (2, 6.0), (3, 0.05)):
        row = (torch.randn(1, V, generator=gen(seed)) * std).to(dt)
        x = row.repeat(K, 1)
        buf = torch.full((offset + K * (V + pad) + 64,), float("nan"), dtype=dt, device="cuda")
        v = buf[offset:offset + K * (V + pad)].view(K, V + pad)[:, :V]
        v.copy_(x)
        ok = (torch.rand(1, V, generator=gen(seed + 9)).numpy() < 0.5).repeat(K, 0) if masked else None
        scores = torch.full((1, K), -1.25)
        for over in (False, True) if masked else (False,):
            beam = gbla.beam_shape(1, K, V, n, dtype=dtype, over_allowed=over)
            got = gbla.beam_select(beam, v, scores.cuda(), allowed=None if ok is None else pack(ok).cuda())
            p, _ = reference(x[:1], scores[:, :1], V, n, None if ok is None else ok[:1], over=over)
            p = np.tile(p, (1, K))  # exactly alike
            check(got, p, np.argsort(-p, axis=1, kind="stable")[:, :n], V, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beam_identical_beams_tie_beside_a_beam_far_from_zero(dtype):
    """Equal rows of which some share a warp with rows whose logits are far from 0."""
    V, K = 777, 48
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for seed in range(8):
        row = (torch.randn(1, V, generator=gen(seed)) * 2).to(dt)
        x = torch.cat([row.repeat(40, 1), (torch.randn(8, V, generator=gen(seed + 50)) * 2 - 2e4).to(dt)])
        scores = torch.cat([torch.full((1, 40), -0.75), torch.full((1, 8), -9.0)], 1)
        got = gbla.beam_select(gbla.beam_shape(1, K, V, K, dtype=dtype), x.cuda(), scores.cuda())
        p, _ = reference(x, scores, V, K)
        p = np.concatenate([np.tile(p[:, :V], (1, 40)), p[:, 40 * V:]], 1)  # exactly alike
        check(got, p, np.argsort(-p, axis=1, kind="stable")[:, :K], V, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 300, 5001])
@pytest.mark.parametrize("kind", ["allowed", "inf", "lowest"])
def test_beam_given_tokens_keep_their_scores(dtype, V, kind):
    """A beam with one token that may follow has log softmax 0, whatever the logit: its score stays, and beams of equal score, ended ones
    among them, go by number."""
    B, K = 3, 40
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for seed in range(6):
        g = gen(seed)
        x = (torch.randn(B * K, V, generator=g) * 9).to(dt)
        at = torch.randint(0, V, (B * K,), generator=g)
        ok = torch.zeros(B * K, V, dtype=torch.bool)
        ok[torch.arange(B * K), at] = True
        if kind != "allowed":
            x = torch.where(ok, x, torch.full_like(x, -math.inf if kind == "inf" else torch.finfo(dt).min))
        scores = (-torch.randint(0, 4, (B, K), generator=g) * 0.37 - (0.01 if seed % 2 else 0.0)).float()
        done = torch.rand(B, K, generator=g) < 0.3
        beam = gbla.beam_shape(B, K, V, dtype=dtype, eos=V // 2, over_allowed=True)
        sc, tok, par, dn = gbla.beam_select(beam, x.cuda(), scores.cuda(), allowed=pack(ok.numpy()).cuda() if kind == "allowed" else None, done=done.cuda())
        order = torch.sort(-scores, dim=1, stable=True).indices
        live = torch.gather(scores, 1, order)
        want = torch.gather(torch.where(done, V // 2, at.view(B, K)), 1, order)
        assert torch.equal(par.cpu().long(), order) and torch.equal(tok.cpu().long(), want) and torch.equal(sc.cpu(), live)
        assert torch.equal(dn.cpu(), torch.gather(done, 1, order) | (want == V // 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_ties_of_few_of_many(dtype):
    """Equal logits all over: more tokens of the best runs than the selection holds at once."""
    beam = gbla.beam_shape(1, 128, 131072, 8, dtype=dtype)
    sc, tok, par, _ = gbla.beam_select(beam, torch.ones(128, 131072, device="cuda", dtype=dtype), torch.zeros(1, 128, device="cuda"))
    assert torch.equal(tok.cpu().long(), torch.arange(8)[None]) and not par.any()
    assert ((sc.cpu().double() + math.log(131072)).abs() <= NEAR + E * math.log(131072)).all()


def test_beam_infinities_nan_and_far_logits():
    inf, nan = math.inf, math.nan
    V, K = 70, 6
    for dtype in ("bf16", "f32"):
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        low = torch.finfo(dt).min
        x = torch.randn(K, V, generator=gen(1)).to(dt)
        x[0, 5:] = -inf
        x[1] = -inf
        x[2, 7] = nan
        x[3, 9] = inf
        x[4, ::2] = low       # masks of the type's lowest value
        x[5] = low
        x[5, 11] = 0
        scores = torch.tensor([[-1.0, -0.5, 0.0, 0.0, -2.0, -3.0]])
        beam = gbla.beam_shape(1, K, V, 60, dtype=dtype)
        got = gbla.beam_select(beam, x.cuda(), scores.cuda())
        p, order = reference(x, scores, V, 60)
        assert set(got[2][0].tolist()) == {0, 4, 5}
        check(got, p, order, V, 60)
        # NaN and infinities where the mask lets nothing through: counted over all tokens, not counted over the allowed
        ok = np.ones((K, V), bool)
        ok[2, 7] = ok[3, 9] = False
        for over in (False, True):
            beam = gbla.beam_shape(1, K, V, 60, dtype=dtype, over_allowed=over)
            got = gbla.beam_select(beam, x.cuda(), scores.cuda(), allowed=pack(ok).cuda())
            p, order = reference(x, scores, V, 60, ok, over=over)
            check(got, p, order, V, 60)
            assert ({2, 3} <= set(got[2][0].tolist())) == over
        # logits far from 0, of whole rows and of parts of them, and the largest there are
        x = (torch.randn(K, 5000, generator=gen(2)) * 3).to(dt)
        x[1] += 1e4
        x[2] -= 1e5
        x[3, :100] = 5e3
        x[4] = torch.finfo(dt).max
        x[5, 2000:] = -3e4
        beam = gbla.beam_shape(1, K, 5000, 64, dtype=dtype)
        got = gbla.beam_select(beam, x.cuda(), scores.cuda())
        p, order = reference(x, scores, 5000, 64)
        check(got, p, order, 5000, 64, strict=False)
        # scores that are no numbers, infinite, and huge
        x = torch.randn(K, V, generator=gen(3)).to(dt)
        for s in ([nan, -1, -inf, -2, -3, -4], [inf, -1, -2, -3, nan, -5], [-1e30, -1e30, -2e30, -3e38, 1e30, 0]):
            scores = torch.tensor([s], dtype=torch.float32)
            got = gbla.beam_select(gbla.beam_shape(1, K, V, 20, dtype=dtype), x.cuda(), scores.cuda())
            p, order = reference(x, scores, V, 20)
            sc, tok, par, _ = got
            if inf in s:  # all of beam 0's are infinitely good: by token
                assert (par[0] == 0).all() and tok[0].tolist() == list(range(20)) and (sc[0] == inf).all()
            else:
                check(got, p, order, V, 20, strict=max(abs(v) for v in s if abs(v) < inf) < 100)


def test_beam_order_of_close_candidates():
    """Rows that differ in one far logit, so that their logarithms are some 2^-20 apart: fp32 would see ties."""
    V, K = 3000, 32
    x = (torch.randn(1, V, generator=gen(5)) * 2).repeat(K, 1)
    for k in range(K):  # a different mass in one token, the same best ones
        x[k, V - 1] = -9 + 0.01 * ((k * 11) % K)
    scores = torch.zeros(1, K)
    beam = gbla.beam_shape(1, K, V, K, dtype="f32")
    got = gbla.beam_select(beam, x.cuda(), scores.cuda())
    p, order = reference(x, scores, V, K)
    best = p[0].max()
    gaps = -np.diff(np.sort(-p[0])[:K] * -1)
    assert gaps.max() < 2.0 ** -20 and best > -20  # what fp32 could not tell apart
    check(got, p, order, V, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("std", [8.0, 300.0])
def test_beam_order_of_rows_that_one_logit_dominates(dtype, std):
    """1024 beams, in each one logit (another value each) so far above the rest that it has all the mass: score + logit - logarithm is
    the score, whatever the logit.  Scores are 2^-26 apart, the bound of two rows' logarithms: their order is the beams'."""
    K, V = 1024, 24
    x = torch.full((K, V), -math.inf)
    at = torch.randint(0, V, (K,), generator=gen(1))
    top = torch.randn(K, generator=gen(2)) * std
    x[torch.arange(K), (at + 3) % V] = top - 60
    x[torch.arange(K), at] = top
    x = x.bfloat16() if dtype == "bf16" else x
    for spread in (1, -1):
        scores = -(torch.arange(K)[None] * 2.0 ** -26).float()
        order = torch.arange(K) if spread > 0 else torch.arange(K).flip(0)
        scores = scores[:, order].contiguous()
        sc, tok, par, _ = gbla.beam_select(gbla.beam_shape(1, K, V, K, dtype=dtype), x.cuda(), scores.cuda())
        assert torch.equal(par[0].cpu().long(), order) and torch.equal(tok[0].cpu().long(), at[order])
        assert ((sc.cpu().double() - torch.sort(scores.double(), descending=True).values).abs() <= NEAR / 2).all()


def test_beam_every_bf16_top():
    """Rows whose largest logit is each bf16 value up to 4096 of either sign, with logits just below and far below it, -inf, and places
    past the row's end: none of them loses its row."""
    v = (torch.arange(65536, dtype=torch.int32) << 16).view(torch.float32)
    top = v[torch.isfinite(v) & (v.abs() <= 4096)]
    B, V = len(top), 300
    x = torch.full((B, V), -math.inf)
    x[:, 100:200] = top[:, None] - 2000
    x[:, 250] = top - 1
    x[:, 7] = top
    x = x.bfloat16()
    scores = torch.zeros(B, 1)
    got = gbla.beam_select(gbla.beam_shape(B, 1, V, 3), x.cuda(), scores.cuda())
    p, order = reference(x, scores, V, 3)
    check(got, p, order, V, 3, strict=False)


@pytest.mark.parametrize("far", [4090.0, -4090.0])
def test_beam_order_of_close_candidates_near_the_ends_of_the_fast_range(far):
    """Logits near +-4096, where the logarithm's power of two takes 13 bits; rows whose sums differ by some 2^-20."""
    V, K = 3000, 32
    x = (torch.randn(1, V, generator=gen(5)).clamp(-4, 4) + far).repeat(K, 1)
    for k in range(K):
        x[k, V - 1] = far - 4 + 0.25 * ((k * 11) % K) / K
        x[k] = x[k] + (k % 3) * 0.5  # the same row, moved: its candidates' scores stay
    x = torch.round(x * 1024) / 1024   # (moving a row is exact)
    scores = torch.zeros(1, K)
    got = gbla.beam_select(gbla.beam_shape(1, K, V, K, dtype="f32"), x.cuda(), scores.cuda())
    p, order = reference(x, scores, V, K)
    w = np.take_along_axis(p[0], order[0], 0)
    assert 0 < (-np.diff(w))[np.diff(w) != 0].min() < 2.0 ** -19
    check(got, p, order, V, K, strict=False)
    assert np.abs(got[0].cpu().double().numpy()[0] - w).max() <= NEAR + E * np.abs(w).max()


def test_beam_a_large_call_by_spot_checks():
    B, K, V = 64, 16, 32768
    v, x, scores = make(B, K, V, "bf16", seed=3)
    beam = gbla.beam_shape(B, K, V)
    ws = gbla.beam_workspace(beam)
    got = gbla.beam_select(beam, v, scores.cuda(), ws=ws)
    for b in (0, 31, 63):
        p, order = reference(x[b * K:(b + 1) * K], scores[b:b + 1], V, K)
        check([None if t is None else t[b:b + 1] for t in got], p, order, V, K)


def test_beam_offsets_beyond_32_bits():
    B, K, V = 2, 40, 1 << 24
    x = torch.full((B * K, V), -8.0, dtype=torch.bfloat16, device="cuda")
    want = {}
    for i, (b, k, t) in enumerate([(1, 39, V - 1), (1, 38, V - 2), (0, 39, 12345678), (1, 0, 0), (0, 0, V - 1)]):
        x[b * K + k, t] = 30 - i
        want.setdefault(b, []).append((k, t))
    scores = torch.zeros(B, K, device="cuda")
    sc, tok, par, _ = gbla.beam_select(gbla.beam_shape(B, K, V, 3), x, scores)
    for b, pairs in want.items():
        assert list(zip(par[b].tolist(), tok[b].tolist()))[:len(pairs)] == pairs or \
            set(list(zip(par[b].tolist(), tok[b].tolist()))[:len(pairs)]) == set(pairs)


def test_beam_logits_and_places_beyond_32_bits():
    """Logits of more than 2^32 values, and a group of more than 2^31 candidates whose best are in its last rows."""
    for B, K, V in ((2, 130, (1 << 24) + 1), (1, 150, 1 << 24)):
        assert K * V > 1 << 31 and (B == 1 or B * K * V > 1 << 32)
        x = torch.full((B * K, V), -8.0, dtype=torch.bfloat16, device="cuda")
        scores = torch.zeros(B, K)
        want = [[(K - 1, V - 1), (K - 2, 0), (0, 12345678), (K - 1, 3)], [(K - 1, V - 2), (K // 2, 5), (K - 3, V - 1), (1, 1)]][:B]
        for b, pairs in enumerate(want):
            for i, (k, t) in enumerate(pairs):
                x[b * K + k, t] = 30 - i / 4 if (k, t) != (K - 1, 3) else 24
                scores[b, k] -= i if k != K - 1 else 0
        sc, tok, par, _ = gbla.beam_select(gbla.beam_shape(B, K, V, 4), x, scores.cuda())
        for b, pairs in enumerate(want):
            assert list(zip(par[b].tolist(), tok[b].tolist())) == pairs, (K, b)
        del x


# ------------------------------------------------------------------ reorder
@pytest.mark.parametrize("dtype,width,offset", [(torch.float32, 512, 0), (torch.float32, 5, 0), (torch.float32, 64, 1), (torch.bfloat16, 33, 0), (torch.uint8, 1, 0),
                                                (torch.bfloat16, 8, 4), (torch.uint8, 100, 3), (torch.float32, 5000, 0), (torch.float64, 3, 0)])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 8), (2, 100), (1, 1024), (70, 16)])
def test_reorder_moves_rows(dtype, width, offset, B, K):
    n = max(1, K // 2 + 1)
    raw = torch.randint(0, 100, (B * K * width + offset + 16,), generator=gen(K), dtype=torch.uint8).to(dtype).cuda()
    src = raw[offset:offset + B * K * width].view(B * K, width)
    keep = raw.clone()
    beam = gbla.beam_shape(B, K, 50, n)
    parents = torch.randint(0, K, (B, n), generator=gen(7), dtype=torch.int32).cuda()
    out = torch.full((B * n * width + offset + 16,), 7, dtype=torch.uint8).to(dtype).cuda()
    dst = out[offset:offset + B * n * width].view(B * n, width)
    plan = gbla.beam_reorder_plan(beam, [src], [dst])
    gbla.beam_reorder(plan, parents)
    assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK
    rows = (parents.long() + torch.arange(B, device="cuda")[:, None] * K).view(-1)
    assert torch.equal(dst, src[rows]) and torch.equal(raw, keep)
    assert (out[:offset].float() == 7).all() and (out[offset + dst.numel():].float() == 7).all()
    # in place, with repeated, crossed and unmoved rows
    inplace = gbla.beam_shape(B, K, 50)
    parents = torch.randint(0, K, (B, K), generator=gen(8), dtype=torch.int32).cuda()
    parents[0] = torch.arange(K - 1, -1, -1)
    want = src[(parents.long() + torch.arange(B, device="cuda")[:, None] * K).view(-1)]
    gbla.beam_reorder(gbla.beam_reorder_plan(inplace, [src]), parents)
    assert torch.equal(src, want)
    assert torch.equal(raw[:offset], keep[:offset]) and torch.equal(raw[offset + src.numel():], keep[offset + src.numel():])


def test_reorder_to_more_beams_than_there_were():
    B, K, n = 5, 1, 700
    src = torch.randn(B, 96, generator=gen(1)).cuda()
    dst = torch.empty(B * n, 96, device="cuda")
    plan = gbla.beam_reorder_plan(gbla.beam_shape(B, K, 10, n), [src], [dst])
    gbla.beam_reorder(plan, torch.zeros(B, n, dtype=torch.int32, device="cuda"))
    assert torch.equal(dst, src.repeat_interleave(n, 0)) and gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK


def test_reorder_many_tensors_and_bad_parents():
    B, K = 3, 4
    beam = gbla.beam_shape(B, K, 10)
    states = [torch.randn(B * K, 1 + j % 7, generator=gen(j)).cuda() for j in range(150)] + [torch.empty(B * K, 0, device="cuda")]
    before = [s.clone() for s in states]
    parents = torch.tensor([[1, 0, 0, 3], [3, 3, 3, 3], [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    plan = gbla.beam_reorder_plan(beam, states)
    gbla.beam_reorder(plan, parents)
    assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_OK
    rows = (parents.long() + torch.arange(B, device="cuda")[:, None] * K).view(-1)
    for s, t in zip(states, before):
        assert torch.equal(s, t[rows])
    for bad in (-1, K, 2 ** 31 - 1):  # reported, and its row stays
        t = [s.clone() for s in states]
        parents[1, 2] = bad
        gbla.beam_reorder(plan, parents)
        assert gbla.gbla_check_device_status(plan.ws) == gbla.GBLA_ERR_DEVICE_CHECK
        good = torch.where(parents < 0, 2, torch.where(parents >= K, 2, parents))
        rows = (good.long() + torch.arange(B, device="cuda")[:, None] * K).view(-1)
        for s, u in zip(states, t):
            assert torch.equal(s, u[rows])
    empty = gbla.beam_reorder_plan(beam, [])
    gbla.beam_reorder(empty, parents.clamp(0, K - 1))
    assert gbla.gbla_check_device_status(empty.ws) == gbla.GBLA_OK


def test_beam_on_streams_and_in_graphs():
    B, K, V = 4, 8, 1000
    beam = gbla.beam_shape(B, K, V, eos=5)
    data = [make(B, K, V, seed=s) for s in (1, 2)]
    ws = gbla.beam_workspace(beam)
    state0 = torch.randn(B * K, 24, generator=gen(0)).cuda()
    want = []
    for v, _, sc in data:
        st = state0.clone()
        out = gbla.beam_select(beam, v, sc.cuda(), ws=ws)
        gbla.beam_reorder(gbla.beam_reorder_plan(beam, [st]), out[2])
        want.append((*out, st))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = gbla.beam_select(beam, data[0][0], data[0][2].cuda(), ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(other, want[0]):
        assert torch.equal(a, b)
    x, sc, st = data[0][0].contiguous().clone(), data[0][2].cuda(), state0.clone()
    out = tuple(torch.empty_like(t) for t in want[0][:4])
    plan = gbla.beam_reorder_plan(beam, [st])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gbla.beam_select(beam, x, sc, out=out, ws=ws)
        gbla.beam_reorder(plan, out[2])
    for k in (1, 0):
        x.copy_(data[k][0])
        sc.copy_(data[k][2])
        st.copy_(state0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, st), want[k]):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- together
def sigmoid(x):
    return 1 / (1 + np.exp(-x))


def test_decoding_loop():
    """Tokens in, best beams out, three steps: embedding, norm, one step of the recurrence with its state in place, norm, logits,
    selection among the allowed, states after their parents; against the same in numpy in 64 bits.  Scores by a bound: each
    step's logits are off by the roundings of fp32 (200 E of values up to 4, times the row sums of the products, below 60)."""
    B, K, V, d = 2, 5, 61, 24
    g = gen(11)
    f = lambda *s, k=1.0: torch.randn(*s, generator=g) * k  # noqa: E731
    table, W, head, lam = f(V, d), f(d, 3 * d, k=d ** -0.5), f(d, V, k=1.5 * d ** -0.5), f(d, k=0.5)
    w1, b1, w2, b2 = 1 + f(d, k=0.1), f(d, k=0.1), 1 + f(d, k=0.1), f(d, k=0.1)
    ok = torch.rand(B * K, V, generator=g).numpy() < 0.5
    cu = lambda t: t.float().cuda()  # noqa: E731
    shape, beam = gbla.glr_shape(B * K, 1, d, dtype="f32"), gbla.beam_shape(B, K, V, dtype="f32", eos=2)
    h = torch.zeros(B * K, d, device="cuda")
    tokens = torch.randint(0, V, (B, 1), generator=g, dtype=torch.int32).repeat(1, K).contiguous().cuda()
    scores = torch.full((B, K), -math.inf)
    scores[:, 0] = 0
    scores, done = scores.cuda(), torch.zeros(B, K, dtype=torch.bool, device="cuda")
    plan = gbla.beam_reorder_plan(beam, [h])
    allowed = pack(ok).cuda()
    # the same in 64 bits
    h64, t64 = np.zeros((B * K, d)), tokens.cpu().numpy().reshape(-1)
    s64, d64 = scores.cpu().double(), torch.zeros(B, K, dtype=torch.bool)
    n64 = lambda t: t.double().numpy()  # noqa: E731

    def norm(s, w, b):
        c = s - s.mean(1, keepdims=True)
        return c / np.sqrt((c ** 2).mean(1, keepdims=True) + 1e-5) * n64(w) + n64(b)
    for step in range(3):
        e = gbla.embed_forward(shape, tokens.view(-1), cu(table), scale=2.0)
        y, _, _ = gbla.layer_norm_forward(shape, e, cu(w1), cu(b1))
        xri = y @ cu(W)
        z, _, _ = gbla.glr_forward(shape, xri[:, :d], xri[:, d:2 * d], xri[:, 2 * d:], cu(lam), h0=h, hT=h)
        o, _, _ = gbla.layer_norm_forward(shape, z, cu(w2), cu(b2), res=e)
        scores, tok, parents, done = gbla.beam_select(beam, o @ cu(head), scores, allowed=allowed, done=done)
        gbla.beam_reorder(plan, parents)
        tokens = tok
        e6 = np.where(t64[:, None] >= 0, 2 * n64(table)[t64.clip(0)], 0)
        q = norm(e6, w1, b1) @ n64(W)
        a = np.exp(-8.0 * np.log1p(np.exp(n64(lam))) * sigmoid(q[:, d:2 * d]))
        h64 = a * h64 + np.sqrt(1 - a * a) * sigmoid(q[:, 2 * d:]) * q[:, :d]
        logits = norm(h64 + e6, w2, b2) @ n64(head)
        p, order = reference(torch.from_numpy(logits), s64, V, K, ok, d64, 2)
        live = np.sort(-p, axis=1)[:, :K + 1]
        assert (np.diff(live[np.isfinite(live).all(1)], axis=1) > 1e-4).all()  # the best are far enough apart to compare
        par, tk = order // V, order % V
        assert np.array_equal(parents.cpu().numpy(), par) and np.array_equal(tok.cpu().numpy(), tk)
        s64 = torch.from_numpy(np.take_along_axis(p, order, 1))
        d64 = torch.gather(d64, 1, torch.from_numpy(par)) | torch.from_numpy(tk == 2)
        assert torch.equal(done.cpu(), d64)
        assert (scores.cpu().double() - s64).abs().max() <= 200 * E * 4 * 60 * (step + 1)
        h64 = h64[(par + np.arange(B)[:, None] * K).reshape(-1)]
        t64 = tk.reshape(-1)
        assert np.abs(h.cpu().double().numpy() - h64).max() <= 200 * E * 4 * (step + 1) + 1e-4


def test_training_step_with_the_update():
    """ids -> embedding -> norm -> the layer -> norm with its residual, their gradients into one AdamW plan; the gradients of the
    embedding and the norms against differences of the whole's loss in the directions that they give.  The loss is summed in 64
    bits; the step of 2^-6 of each tensor's size leaves 0.05 of the derivative for the second differences and the layer's fp32."""
    B, L, d, H, dh, V = 2, 48, 64, 2, 32, 40
    n = H * dh
    g = gen(21)
    f = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).cuda()  # noqa: E731
    P = {"conv_w": f(d, 4, k=0.5), "conv_b": f(d, k=0.1), **{k: f(d, n, k=d ** -0.5) for k in ("W_q", "W_k", "W_v", "W_r")},
         "w_g": f(d, H, k=d ** -0.5), "b_g": f(H, k=0.1), "rms_w": 1 + f(dh, k=0.1),
         "table": f(V, d, k=0.2), "n1_w": 1 + f(d, k=0.1), "n1_b": f(d, k=0.1), "n2_w": 1 + f(d, k=0.1), "n2_b": f(d, k=0.1)}
    ids = torch.randint(0, V, (B * L,), generator=g, dtype=torch.int32).cuda()
    lens = torch.tensor([48, 31], dtype=torch.int32, device="cuda")
    shape = gbla.make_shape(B, L, d, H, dh, dtype="f32", seq_lens=lens)
    target = f(B * L, d)

    def forward(P):
        e = gbla.embed_forward(shape, ids, P["table"], scale=8.0)
        x, _, st1 = gbla.layer_norm_forward(shape, e, P["n1_w"], P["n1_b"], stats=True)
        y, saved = gbla.gbla_forward(shape, x, P, saved=True)
        o, s, st2 = gbla.layer_norm_forward(shape, y, P["n2_w"], P["n2_b"], res=e, stats=True)
        return float((o.double() * target.double()).sum()), (e, x, st1, saved, s, st2)
    loss, (e, x, st1, saved, s, st2) = forward(P)
    g2 = gbla.layer_norm_backward(shape, s, P["n2_w"], st2, target)
    grads = gbla.gbla_backward(shape, x, P, saved, g2["dx"])
    g1 = gbla.layer_norm_backward(shape, e, P["n1_w"], st1, grads["dx"], ds=g2["dx"])  # e goes on as the residual too
    grads.update(dtable=gbla.embed_backward(shape, ids, g1["dx"], V, scale=8.0), dn1_w=g1["dw"], dn1_b=g1["db"], dn2_w=g2["dw"], dn2_b=g2["db"])
    for k in ("table", "n1_w", "n1_b", "n2_w", "n2_b"):
        dirn = grads["d" + k] / grads["d" + k].norm()
        h = 2.0 ** -6 * float(P[k].norm()) / math.sqrt(P[k].numel())
        lo, hi = (forward({**P, k: P[k] + c * h * dirn})[0] for c in (-1, 1))
        want = float(grads["d" + k].norm())
        assert abs((hi - lo) / (2 * h) - want) <= 0.05 * want, k
    state = gbla.gbla_adamw_state(P)
    plan = gbla.gbla_adamw_plan(P, grads, state)
    before = {k: v.clone() for k, v in P.items()}
    gbla.gbla_adamw_step(plan, lr=1e-3, norm=gbla.gbla_grad_norm(plan), max_norm=1.0)
    torch.cuda.synchronize()
    assert int(state["step"]) == 1 and all(not torch.equal(before[k], P[k]) for k in P)
