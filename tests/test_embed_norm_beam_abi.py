"""Host-side statuses, sizes and the binding's refusals of the token embedding, the layer norm and the beam search (no GPU
needed)."""
import ctypes

import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla

FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)  # never dereferenced
OTHER = ctypes.c_void_p(1 << 21)
I, W, U = gbla.GBLA_ERR_INVALID_ARG, gbla.GBLA_ERR_WORKSPACE, gbla.GBLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return gbla.lib()


def _shapes_that_are_wrong():
    bad = gbla.glr_shape(2, 100, 48)
    bad.io_dtype = 9
    both = gbla.glr_shape(1, 100, 48)
    both.cu_seqlens, both.num_seqs, both.seq_lens = 256, 1, 512
    two = gbla.glr_shape(2, 100, 48)
    two.cu_seqlens, two.num_seqs = 256, 1
    return [(s, I) for s in (bad, both, two, gbla.glr_shape(0, 100, 48), gbla.glr_shape(2, 0, 48), gbla.glr_shape(2, 100, 0))] + \
        [(gbla.glr_shape(1 << 16, 1 << 16, 48), U), (gbla.glr_shape(2, 100, (1 << 20) + 1), U)]


def _embed(L, s, bwd, ids=FAKE, wide=0, k=1, t=FAKE, V=500, out=OTHER, ws=FAKE, n=1 << 40):
    return (L.embed_backward if bwd else L.embed_forward)(ctypes.byref(s), ids, wide, k, t, V, 1.0, out, ws, n, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embed_host_errors_launch_nothing(L, bwd, dtype):
    s = gbla.glr_shape(2, 100, 48, dtype=dtype)
    for bad in (dict(ids=None), dict(ids=ODD), dict(t=None), dict(t=ODD), dict(out=None), dict(out=ODD), dict(wide=2), dict(wide=-1),
                dict(k=0), dict(V=0), dict(V=-1), dict(wide=1, ids=ctypes.c_void_p((1 << 20) + 4))):
        assert _embed(L, s, bwd, **bad) == I, bad
    assert _embed(L, gbla.glr_shape(1 << 10, 1 << 18, 8192, dtype=dtype), bwd) == U  # rows k d
    for big in (dict(V=(1 << 30) + 1), dict(k=1 << 24), dict(k=(1 << 20) + 1)):
        assert _embed(L, s, bwd, **big) == U, big
    assert _embed(L, gbla.glr_shape(2, 100, 1 << 20, dtype=dtype), bwd, V=1 << 20) == U
    n = gbla.embed_workspace_size(s, 500, 1, bwd)
    assert n > 0
    for bad in (dict(n=n - 1), dict(ws=None), dict(ws=ctypes.c_void_p((1 << 20) + 16))):
        assert _embed(L, s, bwd, **bad) == W, bad
    for wrong, want in _shapes_that_are_wrong():
        assert _embed(L, wrong, bwd) == want and gbla.embed_workspace_size(wrong, 500, 1, bwd) == 0
    assert L.embed_workspace_size(ctypes.byref(s), 500, 1, 2) == 0
    with pytest.raises(gbla.GblaError):
        gbla.embed_workspace(s, 0)


def test_embed_sizes(L):
    s, big = gbla.glr_shape(2, 100, 48), gbla.glr_shape(32, 4096, 512)
    assert gbla.embed_workspace_size(s, 500) == 256
    assert 0 < gbla.embed_workspace_size(s, 500, 1, True) < gbla.embed_workspace_size(s, 500, 4, True) < gbla.embed_workspace_size(big, 500, 4, True)
    # keys and slots twice, the digits' counts of tiles of 1024 keys, two partial rows of 32 slots, a word an id: about
    # n (17 + d / 4) + 4 V bytes
    n, d, V = 32 * 4096, 512, 1 << 20
    assert gbla.embed_workspace_size(big, V, 1, True) < n * (18 + d // 4) + 4 * V + (1 << 16)


def _fwd(L, s, x=FAKE, ldx=48, res=OTHER, w=FAKE, b=FAKE, eps=1e-5, total=ctypes.c_void_p(3 << 20), y=ctypes.c_void_p(4 << 20),
         stats=ctypes.c_void_p(5 << 20), ws=FAKE, n=1 << 40):
    return L.layer_norm_forward(ctypes.byref(s), x, ldx, res, w, b, eps, total, y, stats, ws, n, None)


def _bwd(L, s, x=FAKE, ldx=48, w=FAKE, stats=FAKE, dy=OTHER, ds=OTHER, dx=ctypes.c_void_p(3 << 20), dw=FAKE, db=FAKE, ws=FAKE, n=1 << 40):
    return L.layer_norm_backward(ctypes.byref(s), x, ldx, w, stats, dy, ds, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_host_errors_launch_nothing(L, dtype):
    s = gbla.glr_shape(2, 100, 48, dtype=dtype)
    for bad in (dict(x=None), dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(b=ODD), dict(y=None), dict(y=ODD), dict(total=ODD), dict(stats=ODD),
                dict(stats=ctypes.c_void_p((5 << 20) + 4)), dict(ldx=47), dict(ldx=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(res=None), dict(total=FAKE, ldx=96), dict(y=FAKE), dict(y=OTHER), dict(y=ctypes.c_void_p(3 << 20))):
        assert _fwd(L, s, **bad) == I, bad
    for bad in (dict(x=None), dict(stats=None), dict(stats=ctypes.c_void_p((1 << 20) + 4)), dict(dy=None), dict(dy=ODD), dict(ds=ODD),
                dict(dx=None), dict(dx=ODD), dict(dw=ODD), dict(db=ODD), dict(w=ODD), dict(ldx=0), dict(dx=FAKE), dict(dx=OTHER)):
        assert _bwd(L, s, **bad) == I, bad
    n, m = gbla.layer_norm_workspace_size(s), gbla.layer_norm_workspace_size(s, True)
    assert 0 < n < m
    for bad in (dict(n=n - 1), dict(ws=None), dict(ws=ctypes.c_void_p((1 << 20) + 16))):
        assert _fwd(L, s, **bad) == W, bad
    assert _bwd(L, s, n=m - 1) == W and _bwd(L, s, ws=None) == W
    for wrong, want in _shapes_that_are_wrong():
        assert _fwd(L, wrong, ldx=1 << 21) == want and _bwd(L, wrong, ldx=1 << 21) == want and gbla.layer_norm_workspace_size(wrong, True) == 0
    assert L.layer_norm_workspace_size(ctypes.byref(s), 2) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_refuses_strides_that_pass_64_bits(L, dtype):
    s = gbla.glr_shape(2, 100, 48, dtype=dtype)
    for ldx in ((1 << 40) + 1, 1 << 60):
        assert _fwd(L, s, ldx=ldx) == I and _bwd(L, s, ldx=ldx) == I


def _select(L, g, logits=FAKE, ld=1000, scores=FAKE, allowed=None, done=None, out=(FAKE, FAKE, FAKE), new_done=None, ws=FAKE, n=1 << 40):
    return L.beam_select(ctypes.byref(g), logits, ld, scores, allowed, done, *out, new_done, ws, n, None)


def _wrong_beams():
    ok = dict(B=2, K=4, V=1000, n_out=4)
    for bad in (dict(B=0), dict(K=0), dict(V=0), dict(n_out=0), dict(eos=-2), dict(eos=1000)):
        yield gbla.beam_shape(**{**ok, **bad}), I
    g = gbla.beam_shape(**ok)
    g.io_dtype = 5
    yield g, I
    g = gbla.beam_shape(**ok)
    g.over_allowed = 2
    yield g, I
    for bad in (dict(K=1025), dict(n_out=1025), dict(K=1024, V=(1 << 22) + 1), dict(K=1, V=(1 << 30) + 1), dict(B=1 << 30)):
        yield gbla.beam_shape(**{**ok, **bad}), U


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beam_host_errors_launch_nothing(L, dtype):
    g = gbla.beam_shape(2, 4, 1000, dtype=dtype)
    for bad in (dict(logits=None), dict(logits=ODD), dict(ld=999), dict(ld=-1), dict(ld=1 << 41), dict(scores=None), dict(scores=ODD),
                dict(allowed=ODD), dict(out=(None, FAKE, FAKE)), dict(out=(FAKE, ODD, FAKE)), dict(out=(FAKE, FAKE, None)), dict(done=FAKE)):
        assert _select(L, g, **bad) == I, bad
    n = gbla.beam_workspace_size(g)
    assert _select(L, g, n=n - 1) == W and _select(L, g, ws=None) == W and _select(L, g, ws=ctypes.c_void_p((1 << 20) + 16)) == W
    for wrong, want in _wrong_beams():
        assert _select(L, wrong, ld=1 << 23) == want and gbla.beam_workspace_size(wrong) == 0
        assert L.beam_reorder(ctypes.byref(wrong), None, 0, FAKE, FAKE, 256, None) == want
    with pytest.raises(gbla.GblaError):
        gbla.beam_workspace(gbla.beam_shape(2, 4, 1000, eos=1000))
    assert 0 < n < gbla.beam_workspace_size(gbla.beam_shape(64, 16, 32768)) < 4 << 20


def test_reorder_host_errors_launch_nothing(L):
    g, h = gbla.beam_shape(2, 4, 1000), gbla.beam_shape(2, 4, 1000, n_out=3)

    def call(g, states, parents=FAKE, ws=FAKE, n=256, count=None):
        table = (gbla.BeamState * max(1, len(states)))(*states)
        return L.beam_reorder(ctypes.byref(g), table, len(states) if count is None else count, parents, ws, n, None)
    ok = gbla.BeamState(1 << 20, 1 << 21, 64)
    for states in ([gbla.BeamState(None, 1 << 21, 64)], [gbla.BeamState(1 << 20, None, 64)], [gbla.BeamState(1 << 20, 1 << 21, -1)]):
        assert call(g, states) == I
    assert call(h, [gbla.BeamState(1 << 20, 1 << 20, 64)]) == I  # in place, but not as many beams out as in
    assert call(g, [ok], parents=None) == I and call(g, [ok], parents=ODD) == I and call(g, [ok], count=-1) == I
    assert L.beam_reorder(ctypes.byref(g), None, 1, FAKE, FAKE, 256, None) == I
    assert call(g, [ok], n=255) == W and call(g, [ok], ws=None) == W
    assert call(gbla.beam_shape(1 << 20, 4, 1000), [gbla.BeamState(1 << 20, 1 << 21, 1 << 30)]) == U


def test_reorder_refuses_what_31_bits_of_tasks_cannot_count(L):
    def call(B, n, row, dst):
        table = (gbla.BeamState * 1)(gbla.BeamState(dst, 1 << 21, row))
        return L.beam_reorder(ctypes.byref(gbla.beam_shape(B, 4, 1000, n_out=n)), table, 1, FAKE, FAKE, 256, None)
    for dst in (1 << 20, 1 << 21):  # into another tensor, within one
        assert call(1 << 20, 4, 1 << 18, dst) == U and call(1 << 9, 4, (1 << 28) + 1, dst) == U
        assert call(1, 4, (1 << 30) + 1, dst) == U
    assert call(1 << 9, 1024, (1 << 20) + 1, 1 << 20) == U


def test_binding_refuses_wrong_tensors(L):
    """Host tensors, wrong types, sizes and strides, before anything reaches the library."""
    s = gbla.glr_shape(2, 8, 16, dtype="f32")
    t = torch.zeros(16, 16)
    ids = torch.zeros(16, dtype=torch.int32)
    for call in (lambda: gbla.embed_forward(s, ids, t), lambda: gbla.embed_backward(s, ids, t, 16), lambda: gbla.layer_norm_forward(s, t),
                 lambda: gbla.layer_norm_backward(s, t, None, torch.zeros(16, 2), t),
                 lambda: gbla.beam_select(gbla.beam_shape(2, 8, 16, dtype="f32"), t, torch.zeros(2, 8)),
                 lambda: gbla.beam_reorder_plan(gbla.beam_shape(2, 8, 16), [t])):
        with pytest.raises(ValueError):
            call()

    class Fake:  # what the binding asks of a tensor
        is_cuda, device = True, torch.device("cuda", 0)

        def __init__(self, shape, dtype, strides=None):
            self.shape, self.dtype, self.at = torch.Size(shape), dtype, 1 << 20
            self.strides = strides or tuple(torch.empty(shape, device="meta").stride())

        def dim(self):
            return len(self.shape)

        def stride(self, k=None):
            return self.strides if k is None else self.strides[k]

        def is_contiguous(self):
            return self.strides == tuple(torch.empty(self.shape, device="meta").stride())

        def numel(self):
            return self.shape.numel()

        def element_size(self):
            return self.dtype.itemsize

        def data_ptr(self):
            return self.at

    f, i32 = torch.float32, torch.int32
    for ids, table in ((Fake((16,), torch.int16), Fake((9, 16), f)), (Fake((15,), i32), Fake((9, 16), f)), (Fake((16, 2, 2), i32), Fake((9, 16), f)),
                       (Fake((16, 2), i32, (4, 2)), Fake((9, 16), f)), (Fake((16,), i32), Fake((9, 15), f)), (Fake((16,), i32), Fake((9, 16), torch.bfloat16)),
                       (Fake((16,), i32), Fake((9, 16), f, (32, 1))), (Fake((16,), i32), Fake((144,), f))):
        with pytest.raises(ValueError):
            gbla.embed_forward(s, ids, table, y=Fake((16, 16), f), ws=Fake((256,), torch.uint8))
    x = Fake((16, 16), f)
    for kw in (dict(x=Fake((16, 15), f)), dict(x=Fake((16, 16), f, (1, 16))), dict(x=x, w=Fake((15,), f)), dict(x=x, b=Fake((16,), torch.bfloat16)),
               dict(x=x, res=Fake((16, 16), f, (32, 1))), dict(x=x, y=Fake((15, 16), f)), dict(x=x, stats=Fake((16,), f))):
        with pytest.raises(ValueError):
            gbla.layer_norm_forward(s, **{**dict(y=x, total=False, ws=Fake((256,), torch.uint8)), **kw})
    g = gbla.beam_shape(2, 8, 100, dtype="f32", eos=3)
    out = (Fake((2, 8), f), Fake((2, 8), i32), Fake((2, 8), i32), Fake((2, 8), torch.bool))
    lg, sc = Fake((16, 100), f), Fake((2, 8), f)
    for kw in (dict(logits=Fake((16, 99), f)), dict(logits=Fake((16, 100), torch.bfloat16)), dict(scores=Fake((16,), f)),
               dict(allowed=Fake((16, 3), i32)), dict(allowed=Fake((16, 4), torch.int64)), dict(done=Fake((2, 8), torch.uint8)),
               dict(out=out[:1] + (Fake((2, 8), torch.int64),) + out[2:]), dict(out=out[:3] + (Fake((2, 7), torch.bool),))):
        with pytest.raises(ValueError):
            gbla.beam_select(g, **{**dict(logits=lg, scores=sc, out=out, ws=Fake((1 << 20,), torch.uint8)), **kw})
    # reordering: shapes, an overlap, in place with another number of beams
    for states, to, beam in (([Fake((15, 4), f)], None, g), ([Fake((16, 4), f)], [Fake((16, 4), i32)], g), ([Fake((16, 4), f)], [], g),
                             ([Fake((16, 4), f)], [Fake((16, 4), f)], g), ([Fake((16, 4), f)], None, gbla.beam_shape(2, 8, 100, n_out=4))):
        with pytest.raises(ValueError):
            gbla.BeamReorderPlan(beam, states, to)
