"""embed_forward and embed_backward against their formulas: every type, odd and
unaligned rows, several ids a token, padded slots, ids of none, one and very many
tokens, sizes around the sort's tiles and digits, offsets beyond 32 bits, bad
ids, streams and graphs.

Bounds: y is one fp32 product and one rounding, so it equals the same operations
in torch bit for bit.  A gradient sums at most 32 rows in fp32 in a row (31
additions, each off by 2^-24 of at most the sum of magnitudes S), such sums in
two fp32 words, and is multiplied and rounded: 34 * 2^-24 scale S.  Tests that say
66 were written for chains of 64 rows and allow more than that."""
import numpy as np
import pytest
import torch

from generative_retrieval_encoder_gb300 import build, gbla

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gbla.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def place(t, offset=0, guard=8):
    """t on the GPU, `offset` values into a larger buffer (so of the element's alignment alone); the buffer too."""
    b = torch.full((t.numel() + offset + guard,), 77, dtype=t.dtype, device="cuda")
    v = b[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    return v, b


def valid_rows(B, L, seq_lens):
    if seq_lens is None:
        return np.ones(B * L, bool)
    return (np.arange(L)[None, :] < np.asarray(seq_lens)[:, None]).reshape(-1)


def reference(ids, valid, dy, V, scale):
    """(dtable, bound) in 64 bits."""
    T, k = ids.shape
    d = dy.shape[1] // k
    ids = np.where(valid[:, None], ids, -1).reshape(-1)
    rows = dy.reshape(T * k, d)
    g, s = np.zeros((V, d)), np.zeros((V, d))
    keep = ids >= 0
    np.add.at(g, ids[keep], rows[keep])
    np.add.at(s, ids[keep], np.abs(rows[keep]))
    return g * scale, 66 * E * abs(scale) * s + 1e-40


def check_case(ids, V, d, dtype="bf16", B=None, L=None, seq_lens=None, scale=1.5, wide=False, offset=0, seed=0, varlen=False):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ids = torch.as_tensor(ids)
    ids = ids[:, None] if ids.dim() == 1 else ids
    T, k = ids.shape
    B, L = (1, T) if B is None else (B, L)
    table, _ = place(torch.randn(V, d, generator=gen(seed)).to(dt), offset)
    dy, _ = place(torch.randn(T, k * d, generator=gen(seed + 1)).to(dt), offset)
    y, yb = place(torch.zeros(T, k * d, dtype=dt), offset)
    dtable, gb = place(torch.zeros(V, d), offset)
    y.fill_(9)
    dtable.fill_(9)
    id_dev = ids.to(torch.int64 if wide else torch.int32).cuda()
    lens = None if seq_lens is None else torch.tensor(seq_lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda") if varlen else None
    shape = gbla.glr_shape(B, L, d, dtype=dtype, seq_lens=lens, cu_seqlens=cu)
    ws = gbla.embed_workspace(shape, V, k, True)
    ws.fill_(0xA5)
    one = id_dev[:, 0].contiguous() if k == 1 else id_dev
    assert gbla.embed_forward(shape, one, table, scale=scale, y=y, ws=ws) is y
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    gbla.embed_backward(shape, one, dy, V, scale=scale, dtable=dtable, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    has = torch.as_tensor(valid_rows(B, L, seq_lens))[:, None] & (ids >= 0)
    want = (table.float()[ids.clamp(min=0).view(-1).cuda()] * scale).to(dt)
    want = torch.where(has.view(-1, 1).cuda(), want, torch.zeros((), dtype=dt, device="cuda")).view(T, k * d)
    assert torch.equal(y, want)
    g, bound = reference(ids.numpy(), valid_rows(B, L, seq_lens), dy.double().cpu().numpy(), V, scale)
    err = np.abs(dtable.double().cpu().numpy() - g)
    assert (err <= bound).all(), (err - bound).max()
    assert (yb[:offset] == 77).all() and (yb[offset + y.numel():] == 77).all()
    assert (gb[:offset] == 77).all() and (gb[offset + dtable.numel():] == 77).all()
    # again: the same bits
    again = gbla.embed_backward(shape, one, dy, V, scale=scale, ws=ws)
    assert torch.equal(again, dtable)


def ids_of(kind, n, V, seed):
    g = gen(seed + 100)
    if kind == "uniform":
        return torch.randint(0, V, (n,), generator=g)
    if kind == "one":
        return torch.full((n,), V - 1)
    if kind == "none":
        return torch.full((n,), -1)
    if kind == "hot":  # a power law, some of none
        t = (torch.exp(np.log(V + 1) * torch.rand(n, generator=g)).long() - 1).clamp(0, V - 1)
        return torch.where(torch.rand(n, generator=g) < 0.05, -1, t)
    if kind == "two":  # two ids of many tokens side by side in the sorted order
        return torch.where(torch.rand(n, generator=g) < 0.5, V // 2, V // 2 - 1)
    return torch.arange(n) % V


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,d,kind", [
    (1, 1, 1, "uniform"), (1, 5, 8, "none"), (3, 2, 3, "one"), (63, 9, 64, "one"), (64, 9, 64, "one"), (65, 9, 64, "one"), (129, 3, 16, "two"),
    (2047, 300, 72, "hot"), (2048, 2047, 8, "hot"), (2049, 2048, 8, "hot"), (5000, 2049, 40, "hot"), (4096, 100, 257, "two"),
    (65536 + 1, 7, 8, "uniform"), (70000, 40000, 16, "hot"), (140000, 5, 4, "hot"), (6000, 6000, 512, "range"), (3000, 4200000, 2, "hot"),
    (9000, 64, 1030, "one"), (300, 50, 8200, "hot")])
def test_embed_matches_formulas(dtype, n, V, d, kind):
    check_case(ids_of(kind, n, V, n), V, d, dtype, wide=n % 2 == 0, seed=n)


@pytest.mark.parametrize("dtype,d,offset", [("bf16", 64, 1), ("bf16", 33, 0), ("bf16", 1, 3), ("f32", 64, 1), ("f32", 6, 0), ("bf16", 520, 4), ("f32", 300, 2)])
def test_embed_rows_of_any_alignment(dtype, d, offset):
    check_case(ids_of("hot", 3000, 50, d), 50, d, dtype, offset=offset, seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(20001, 1), (20001, 2), (9001, 5), (9001, 6), (5003, 7), (5003, 10), (3001, 12), (3001, 60), (3001, 100), (2500, 201), (700, 453),
                                 (2500, 510), (2500, 1001), (90, 8198), (40, 30001)])
def test_embed_rows_that_are_not_whole_pieces(dtype, n, d):
    """Pieces of y that hold the ends of rows, or several of them; sums by pairs and by single values."""
    check_case(ids_of("hot", n, 300, d), 300, d, dtype, seed=d)
    check_case(ids_of("hot", n, n // 2, d), n // 2, d, dtype, offset=8 if dtype == "bf16" else 4, seed=d + 1)


@pytest.mark.parametrize("d,offset", [(10, 2), (100, 1), (7, 1), (510, 6)])
def test_embed_tables_of_other_alignment_than_the_output(d, offset):
    table, _ = place(torch.randn(70, d, generator=gen(d)).bfloat16(), offset)
    ids = ids_of("hot", 4001, 70, d).int().cuda()
    shape = gbla.glr_shape(1, 4001, d)
    want = (table.float()[ids.clamp(min=0).long()] * 0.5).bfloat16()
    want[ids < 0] = 0
    for y_off in (0, 3):
        y, buf = place(torch.zeros(4001, d).bfloat16(), y_off)
        gbla.embed_forward(shape, ids, table, scale=0.5, y=y)
        assert torch.equal(y, want) and (buf[:y_off] == 77).all() and (buf[y_off + y.numel():] == 77).all()


@pytest.mark.parametrize("k,d", [(2, 64), (3, 5), (4, 128)])
@pytest.mark.parametrize("form", ["dense", "padded", "varlen"])
def test_embed_several_ids_and_forms(k, d, form):
    B, L = 5, 211
    ids = ids_of("hot", B * L * k, 90, d).view(B * L, k)
    lens = [211, 0, 1, 64, 210] if form == "padded" else None
    if form == "varlen":
        check_case(ids, 90, d, seed=d, varlen=True, wide=True)
    else:
        check_case(ids, 90, d, B=B, L=L, seq_lens=lens, seed=d, scale=-0.3)


def test_embed_padded_rows_may_hold_anything():
    """Ids past a sequence's end are not looked at: out of range or not, they change nothing and report nothing."""
    B, L, V, d = 3, 20, 30, 24
    lens = torch.tensor([20, 0, 7], dtype=torch.int32, device="cuda")
    shape = gbla.glr_shape(B, L, d, seq_lens=lens)
    ids = torch.randint(0, V, (B * L,), generator=gen(0), dtype=torch.int32).cuda()
    inside = torch.as_tensor(valid_rows(B, L, lens.tolist())).cuda()
    table = torch.randn(V, d, generator=gen(1)).bfloat16().cuda()
    dy = torch.randn(B * L, d, generator=gen(2)).bfloat16().cuda()
    ws = gbla.embed_workspace(shape, V, 1, True)
    a, g = gbla.embed_forward(shape, ids, table, ws=ws), gbla.embed_backward(shape, ids, dy, V, ws=ws)
    wild = torch.where(inside, ids, torch.full_like(ids, 2 ** 31 - 1))
    dy2 = torch.where(inside[:, None], dy, torch.full_like(dy, float("nan")))
    b = gbla.embed_forward(shape, wild, table, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    h = gbla.embed_backward(shape, wild, dy2, V, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    assert torch.equal(a, b) and torch.equal(g, h) and (a[~inside] == 0).all()


@pytest.mark.parametrize("n", [5, 3000, 9000])
@pytest.mark.parametrize("wide", [False, True])
def test_embed_bad_ids_and_lengths_are_reported(n, wide):
    V, d = 100, 32
    shape = gbla.glr_shape(1, n, d)
    ids = torch.randint(0, V, (n,), generator=gen(n)).to(torch.int64 if wide else torch.int32).cuda()
    table, dy = torch.randn(V, d, generator=gen(1)).bfloat16().cuda(), torch.randn(n, d, generator=gen(2)).bfloat16().cuda()
    ws = gbla.embed_workspace(shape, V, 1, True)
    bad = ids.clone()
    bad[n // 2] = 2 ** 40 if wide else V
    clean = ids.clone()
    clean[n // 2] = -(2 ** 40) if wide else -2 ** 31
    want_y, want_g = gbla.embed_forward(shape, clean, table, ws=ws), gbla.embed_backward(shape, clean, dy, V, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    y = gbla.embed_forward(shape, bad, table, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
    g = gbla.embed_backward(shape, bad, dy, V, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK
    assert torch.equal(y, want_y) and torch.equal(g, want_g)
    for lens in ([n + 1], [-1]):  # counts as an empty sequence
        s = gbla.glr_shape(1, n, d, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        y = gbla.embed_forward(s, ids, table, ws=ws)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK and (y == 0).all()
        g = gbla.embed_backward(s, ids, dy, V, ws=ws)
        assert gbla.gbla_check_device_status(ws) == gbla.GBLA_ERR_DEVICE_CHECK and (g == 0).all()


def test_embed_nonfinite_rows_stay_theirs():
    V, d, n = 12, 64, 400
    table = torch.randn(V, d, generator=gen(0)).bfloat16()
    table[3] = float("nan")
    table[4] = float("inf")
    ids = torch.randint(0, V, (n,), generator=gen(1), dtype=torch.int32)
    shape = gbla.glr_shape(1, n, d)
    y = gbla.embed_forward(shape, ids.cuda(), table.cuda()).cpu()
    assert y[ids == 3].isnan().all() and (y[ids == 4] == float("inf")).all() and y[(ids != 3) & (ids != 4)].isfinite().all()
    dy = torch.randn(n, d, generator=gen(2)).bfloat16()
    dy[ids == 7] = float("nan")
    g = gbla.embed_backward(shape, ids.cuda(), dy.cuda(), V).cpu()
    assert g[7].isnan().all() and g[[v for v in range(V) if v != 7]].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count", [33, 100, 3000])
def test_embed_infinite_gradients_of_frequent_ids(dtype, count):
    """An infinity among an id's gradients makes its sum infinite, two of different sign NaN; an fp32 sum past the range is infinite."""
    V, d, inf = 5, 16, float("inf")
    ids = torch.arange(V).repeat_interleave(count).to(torch.int32)
    dy = torch.randn(V * count, d, generator=gen(1)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    dy[count // 2, 3] = inf                # id 0
    dy[2 * count - 1, 4] = -inf            # id 1
    dy[2 * count, 5], dy[3 * count - 1, 5] = inf, -inf
    dy[3 * count:4 * count, 6] = 3e38      # id 3: every partial sum of two and more is past the range
    dy[3 * count:4 * count, 7] = 1e37      # one of 32 is in it, the whole is not, or only the whole of many
    shape = gbla.glr_shape(1, V * count, d, dtype=dtype)
    g = gbla.embed_backward(shape, ids.cuda(), dy.cuda(), V).cpu()
    want = dy.double().view(V, count, d).sum(1)
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, torch.sign(want) * inf, want)
    size = dy.double().abs().view(V, count, d).sum(1)
    assert want[0, 3] == inf and want[1, 4] == -inf and want[2, 5].isnan() and want[3, 6] == inf
    same = (g.double() == want) | (g.isnan() & want.isnan()) | ((g.double() - want).abs() <= 34 * E * size)
    assert same.all(), (~same).nonzero()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 10), ("bf16", 7), ("f32", 64), ("f32", 7)])
@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan")])
def test_embed_rows_of_no_token_are_zeros_whatever_the_scale(dtype, d, scale):
    V, n = 9, 300
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ids = torch.randint(-1, V, (n,), generator=gen(1), dtype=torch.int32).cuda()
    table, dy = torch.randn(V, d, generator=gen(2)).to(dt).cuda(), torch.randn(n, d, generator=gen(3)).to(dt).cuda()
    lens = torch.tensor([90, 0, 100], dtype=torch.int32, device="cuda")
    shape = gbla.glr_shape(3, 100, d, dtype=dtype, seq_lens=lens)
    has = (ids >= 0) & torch.as_tensor(valid_rows(3, 100, lens.tolist())).cuda()
    y = gbla.embed_forward(shape, ids, table, scale=scale)
    assert torch.equal(y[~has], torch.zeros_like(y[~has]))
    assert torch.equal(y[has].nan_to_num(nan=7.0), (table[ids[has].long()].float() * scale).to(dt).nan_to_num(nan=7.0))
    g = gbla.embed_backward(shape, torch.where(ids == 5, -1, ids), dy, V, scale=scale)
    assert (g[5] == 0).all() and not g[4].isfinite().any()


def test_embed_gradient_by_differences():
    V, d, n = 7, 5, 300
    shape = gbla.glr_shape(1, n, d, dtype="f32")
    ids = torch.randint(-1, V, (n,), generator=gen(3), dtype=torch.int32).cuda()
    table, dy = torch.randn(V, d, generator=gen(4)).cuda(), torch.randn(n, d, generator=gen(5)).cuda()
    g = gbla.embed_backward(shape, ids, dy, V, scale=0.7)
    f = lambda t: float((gbla.embed_forward(shape, ids, t, scale=0.7).double() * dy.double()).sum())  # noqa: E731
    for v in range(V):
        for c in range(d):
            e = torch.zeros_like(table)
            e[v, c] = 2.0 ** -3
            diff = (f(table + e) - f(table - e)) / 2.0 ** -2
            # table +- e and its products are rounded: 4 E of |table| + |e| a term, over the step
            terms = float((dy[ids == v, c].double().abs()).sum()) * 0.7 * (abs(float(table[v, c])) + 1)
            assert abs(diff - float(g[v, c])) <= 8 * 4 * E * terms + 66 * E * terms


def test_embed_offsets_beyond_32_bits():
    """A table and outputs of more than 2^32 bytes: the far rows are the right ones."""
    V, d, n = 2_300_000, 1024, 40
    table = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1 - 3 * i for i in range(n)], dtype=torch.int64)
    rows = torch.randn(n, d, generator=gen(0)).bfloat16().cuda()
    table[ids.cuda()] = rows
    shape = gbla.glr_shape(1, n, d)
    assert torch.equal(gbla.embed_forward(shape, ids.cuda(), table), rows)
    del table
    g = gbla.embed_backward(shape, ids.cuda(), rows, V)
    assert torch.equal(g[ids.cuda()], rows.float())
    assert int((g != 0).sum()) == int((rows != 0).sum())
    del g
    torch.cuda.empty_cache()
    # many tokens: y of 2^32 bytes and more
    n, d, V = 1_100_000, 2048, 37
    table = torch.randn(V, d, generator=gen(1)).bfloat16().cuda()
    ids = (torch.arange(n) * 5 % V).to(torch.int32).cuda()
    shape = gbla.glr_shape(1, n, d)
    y = gbla.embed_forward(shape, ids, table)
    at = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
    assert torch.equal(y[at], table[ids[at].long()])
    g = gbla.embed_backward(shape, ids, y, V)
    count = torch.bincount(ids.long(), minlength=V).double()[:, None]
    want = table.double() * count
    assert ((g.double() - want).abs() <= 66 * E * want.abs()).all()


def test_embed_on_streams_in_graphs_and_with_shared_workspaces():
    """A captured forward and backward follow the ids that their buffers hold at replay; two graphs may share a workspace
    where they run in order; a call on a side stream gives the same."""
    n, V, d = 5000, 700, 64
    shape = gbla.glr_shape(1, n, d)
    ids = [ids_of("hot", n, V, s).to(torch.int32).cuda() for s in (1, 2)]
    table, dy = torch.randn(V, d, generator=gen(1)).bfloat16().cuda(), torch.randn(n, d, generator=gen(2)).bfloat16().cuda()
    ws = gbla.embed_workspace(shape, V, 1, True)
    want = [(gbla.embed_forward(shape, i, table, ws=ws), gbla.embed_backward(shape, i, dy, V, ws=ws)) for i in ids]
    buf, y, g = ids[0].clone(), torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = gbla.embed_forward(shape, ids[1], table, ws=ws)
        b = gbla.embed_backward(shape, ids[1], dy, V, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want[1][0]) and torch.equal(b, want[1][1])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gbla.embed_forward(shape, buf, table, y=y, ws=ws)
            gbla.embed_backward(shape, buf, dy, V, dtable=g, ws=ws)
        graphs.append(graph)
    for k in (1, 0, 1):
        buf.copy_(ids[k])
        for graph in graphs:
            y.zero_()
            g.fill_(5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[k][0]) and torch.equal(g, want[k][1])


def torch_gradient(ids, dy, V, scale):
    """(dtable, sum of magnitudes) in 64 bits, on the GPU."""
    keep = ids >= 0
    at, rows = ids[keep].long(), dy[keep].double()
    zero = torch.zeros(V, dy.shape[1], dtype=torch.float64, device="cuda")
    return zero.index_add(0, at, rows) * scale, zero.index_add(0, at, rows.abs()) * abs(scale)


@pytest.mark.parametrize("dtype,d", [("bf16", 2048), ("f32", 2044), ("bf16", 515)])
def test_embed_frequent_ids_in_every_turn_of_the_join(dtype, d):
    """More columns of repeated ids than the join's CTAs take at once (32 tasks an SM), every tenth id so frequent that a whole CTA
    sums it.  Bound: up to 31 additions in fp32, two words after that, their sum and the scale: 34 E of the magnitudes."""
    V, rare, often = 900, 40, 1000
    blocks = -(-d // (128 if d % 4 == 0 else 32))
    assert V * blocks > 2 * 32 * torch.cuda.get_device_properties(0).multi_processor_count
    ids = torch.cat([torch.arange(V).repeat_interleave(rare), torch.arange(0, V, 10).repeat_interleave(often)])
    ids = ids[torch.randperm(len(ids), generator=gen(1))].to(torch.int32).cuda()
    dy = torch.randn(len(ids), d, generator=gen(2)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    shape = gbla.glr_shape(1, len(ids), d, dtype=dtype)
    ws = gbla.embed_workspace(shape, V, 1, True)
    got = gbla.embed_backward(shape, ids, dy, V, scale=1.5, ws=ws)
    want, size = torch_gradient(ids, dy, V, 1.5)
    assert ((got.double() - want).abs() <= 34 * E * size).all()
    for _ in range(5):
        assert torch.equal(gbla.embed_backward(shape, ids, dy, V, scale=1.5, ws=ws), got)


@pytest.mark.parametrize("dtype,n,V,d", [("bf16", 655361, 70000, 3), ("f32", 700001, 2_000_000, 4), ("bf16", 3_300_000, 70000, 2), ("bf16", 2_500_001, 1_500_000, 8),
                                         ("bf16", 4_194_304, 200, 1)])
def test_embed_gradient_of_millions_of_slots(dtype, n, V, d):
    """More tiles than whose counts a tile reads itself.  Bound: up to 31 additions in fp32, two words after that, their sum and the
    scale: 34 E of the magnitudes."""
    ids = ids_of("hot", n, V, d).to(torch.int32).cuda()
    dy = torch.randn(n, d, generator=gen(d)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    shape = gbla.glr_shape(1, n, d, dtype=dtype)
    ws = gbla.embed_workspace(shape, V, 1, True)
    ws.fill_(0xA5)
    got = gbla.embed_backward(shape, ids, dy, V, scale=0.5, ws=ws)
    assert gbla.gbla_check_device_status(ws) == gbla.GBLA_OK
    want, size = torch_gradient(ids, dy, V, 0.5)
    assert ((got.double() - want).abs() <= 34 * E * size).all()
    assert torch.equal(gbla.embed_backward(shape, ids, dy, V, scale=0.5, ws=ws), got)


def test_embed_gradient_takes_time_by_the_slots_not_their_square():
    """Eight times the slots: some 7 times the time, where reading all counts in every tile takes 20."""
    V, d, best = 32768, 8, []
    for n in (1 << 21, 1 << 24):
        ids = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda")
        dy, out = torch.ones(n, d, dtype=torch.bfloat16, device="cuda"), torch.empty(V, d, device="cuda")
        shape = gbla.glr_shape(1, n, d)
        ws = gbla.embed_workspace(shape, V, 1, True)
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            gbla.embed_backward(shape, ids, dy, V, dtable=out, ws=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    assert best[1] < 12 * best[0], best
