"""Host-side statuses and sizes of the gated linear recurrence's entry points (no GPU needed)."""
import ctypes

import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla

FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)  # never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return gbla.lib()


def _fwd(L, s, x=FAKE, r=FAKE, i=FAKE, ld=48, lam=FAKE, c=8.0, reverse=0, h0=None, y=FAKE, hT=None, saved=None, ws=FAKE, n=1 << 30):
    return L.glr_forward(ctypes.byref(s), x, r, i, ld, lam, c, reverse, h0, y, hT, saved, ws, n, None)


def _bwd(L, s, saved=FAKE, dy=FAKE, dhT=None, dx=FAKE, dr=FAKE, di=FAKE, ldd=48, dlam=FAKE, dh0=None, ws=FAKE, n=1 << 30, ld=48):
    return L.glr_backward(ctypes.byref(s), FAKE, FAKE, FAKE, ld, FAKE, 8.0, 0, None, saved, dy, dhT, dx, dr, di, ldd, dlam, dh0, ws, n, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_host_errors_launch_nothing(L, dtype):
    s = gbla.glr_shape(2, 100, 48, dtype=dtype)
    I, W, U = gbla.GBLA_ERR_INVALID_ARG, gbla.GBLA_ERR_WORKSPACE, gbla.GBLA_ERR_UNSUPPORTED
    for bad in (dict(x=None), dict(r=None), dict(i=ODD), dict(x=ODD), dict(lam=None), dict(lam=ODD), dict(y=None), dict(y=ODD), dict(h0=ODD),
                dict(hT=ODD), dict(ld=47), dict(ld=-48), dict(c=0.0), dict(c=-1.0), dict(c=float("nan")), dict(c=float("inf")),
                dict(reverse=2), dict(saved=ctypes.c_void_p((1 << 20) + 16))):
        assert _fwd(L, s, **bad) == I, bad
    for bad in (dict(saved=None), dict(saved=ODD), dict(dy=None), dict(dx=None), dict(dr=ODD), dict(di=None), dict(ldd=47), dict(dlam=ODD),
                dict(dhT=ODD), dict(dh0=ODD), dict(ld=0)):
        assert _bwd(L, s, **bad) == I, bad
    n = gbla.gbla_workspace_size(s, gbla.GBLA_OP_GLR_FORWARD)
    m = gbla.gbla_workspace_size(s, gbla.GBLA_OP_GLR_BACKWARD)
    assert _fwd(L, s, n=n - 1) == W and _fwd(L, s, ws=None) == W and _fwd(L, s, ws=ctypes.c_void_p((1 << 20) + 16)) == W
    assert _bwd(L, s, n=m - 1) == W and _bwd(L, s, ws=None) == W
    assert L.glr_forward(None, *[FAKE] * 3, 48, FAKE, 8.0, 0, None, FAKE, None, None, FAKE, 1 << 30, None) == I
    for B, T, d, want in ((1 << 16, 1 << 16, 48, U), (2, 100, (1 << 20) + 1, U), (0, 100, 48, I), (2, 0, 48, I), (2, 100, 0, I)):
        assert _fwd(L, gbla.glr_shape(B, T, d, dtype=dtype), ld=1 << 21) == want


def test_shapes_and_sizes(L):
    small, big = gbla.glr_shape(2, 100, 48), gbla.glr_shape(32, 4096, 512)
    for op in (gbla.GBLA_OP_GLR_FORWARD, gbla.GBLA_OP_GLR_BACKWARD):
        assert 0 < gbla.gbla_workspace_size(small, op) <= gbla.gbla_workspace_size(big, op)
    assert gbla.glr_saved_size(big) == 32 * 512 * 512 * 4  # a state per 8 rows
    assert 0 < gbla.glr_saved_size(small) < gbla.glr_saved_size(big)
    bad = gbla.glr_shape(2, 100, 48)
    bad.io_dtype = 9
    both = gbla.glr_shape(1, 100, 48)
    both.cu_seqlens, both.num_seqs, both.seq_lens = 256, 1, 512
    two = gbla.glr_shape(2, 100, 48)
    two.cu_seqlens, two.num_seqs = 256, 1
    for s in (bad, both, two):
        assert gbla.glr_saved_size(s) == 0 and gbla.gbla_workspace_size(s, gbla.GBLA_OP_GLR_FORWARD) == 0
        assert _fwd(L, s) == gbla.GBLA_ERR_INVALID_ARG
        with pytest.raises(gbla.GblaError):
            gbla.workspace(s, gbla.GBLA_OP_GLR_FORWARD)


def test_binding_refuses_host_tensors(L):
    import torch
    t = torch.zeros(200, 48)
    with pytest.raises(ValueError):
        gbla.glr_forward(gbla.glr_shape(2, 100, 48, dtype="f32"), t, t, t, torch.zeros(48))
    with pytest.raises(ValueError):
        gbla.glr_shape(1, 100, 48, cu_seqlens=torch.zeros(2, dtype=torch.int32))


def test_checks_follow_a_changed_shape(L):
    """A shape's fields are plain values: after a change the binding's checks are those of the new sizes."""
    sh = gbla.glr_shape(2, 16, 8)
    seen = []

    class Fake:  # what the binding asks of a tensor
        is_cuda, dtype, device = True, torch.bfloat16, torch.device("cuda", 0)

        def __init__(self, *shape):
            self.shape = shape

        def dim(self):
            return 2

        def stride(self, k=None):
            return (8, 1) if k is None else (8, 1)[k]

        def data_ptr(self):
            seen.append(self.shape)
            return 256

    sh.L = 32
    with pytest.raises(ValueError, match="64, 8"):
        gbla._glr_inputs(sh, Fake(32, 8), Fake(32, 8), Fake(32, 8), None, None)
    assert not seen


def test_which_calls_are_cut_one_by_one(L):
    """By the size of what a forward saves: a state per 8 rows of each slot (or sequence), or of all rows as one stream."""
    def pieces(d, B, rows, n=0):
        s = gbla.glr_shape(B, rows, d)
        if n:
            s.cu_seqlens, s.num_seqs = 256, n
        return gbla.glr_saved_size(s) // (4 * d)
    for B, rows, one in ((2621, 100, True), (504, 65, True), (40, 100, False), (4096, 63, False), (2, 513, True), (8, 511, False), (64, 511, True)):
        assert pieces(512, B, rows) == (B * -(-rows // 8) if one else -(-B * rows // 8)), (B, rows)
    for d, T, n, one in ((512, 131076, 929, True), (512, 524311, 9714, True), (512, 524291, 35195, False), (512, 8266, 56, False),
                         (512, 32771, 600, False), (1024, 32770, 600, True), (512, 33158, 27, True), (1024, 8653, 8, False), (1024, 262144, 1, False)):
        assert pieces(d, 1, T, n) == (T // 8 + n if one else -(-T // 8)), (d, T, n)


def test_workspace_of_short_slots(L):
    """Slots of one tile exchange no words: the forward's workspace holds none, the backward's (smaller tiles) little."""
    rows, d = 4096 * 100, 512
    s = gbla.glr_shape(4096, 100, d)
    assert gbla.gbla_workspace_size(s, gbla.GBLA_OP_GLR_FORWARD) < 1 << 16
    # two chunks of 64 rows a slot: a word of 8 bytes and a partial sum of 4 for each and channel, one slot more in either
    assert gbla.gbla_workspace_size(s, gbla.GBLA_OP_GLR_BACKWARD) < (rows // 64 + 2 * 4096) * d * 8 + 2 * 4097 * d * 4 + (1 << 16)
