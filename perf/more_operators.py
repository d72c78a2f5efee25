"""The ends and the joints of a model around the layer: token embedding, layer norm and beam search, as a training or
serving program calls them.

Four families of cases:

* ``embed``: rows of a shared table by token ids times a scale, k ids a token (their rows side by side; k > 1 for
      items named by several hashes), alone or with the table's gradient: the sum of the gradients of every token that
      has the id.  Ids follow a power law; some are -1 (no token: a row of zeros).
* ``norm``: s = x + residual, y = (s - mean s) / sqrt(var s + eps) w + b per token, alone or with the gradients of x
      (where the residual's gradient joins), w and b.
* ``beam``: of each group's K beams x V next tokens the n_out of highest score + log softmax(logits), ties to the lowest
      beam and token, with or without a mask of the valid tokens and with beams that have ended; then the beams' states
      follow their parents, in place or into other tensors.

``own`` false computes them with elementary torch operations, true with this repository's kernels.
"""
import math
import random

import torch

own = False

EPS = 1e-5
EOS = 1           # the token that ends a beam, in cases with ended beams


# ----------------------------------------------------------------- cases
def _embed(name, B, L, d, V, dtype="bf16", train=False, form="dense", lo=1, k=1, wide=False):
    c = {"op": "embed", "B": B, "L": L, "d": d, "V": V, "dtype": dtype, "train": train, "form": form, "lo": lo, "k": k, "wide": wide}
    return dict(c, name=name) if name else c


def _norm(name, B, L, d, dtype="bf16", train=False, form="dense", lo=1, res=True, affine=True, cols=False):
    c = {"op": "norm", "B": B, "L": L, "d": d, "dtype": dtype, "train": train, "form": form, "lo": lo, "res": res, "affine": affine,
         "cols": cols}
    return dict(c, name=name) if name else c


def _beam(name, B, K, V, n, dtype="bf16", mask=0.0, renorm=False, ends=False, layers=2, d=512, inplace=True, pad=0):
    c = {"op": "beam", "B": B, "K": K, "V": V, "n": n, "dtype": dtype, "mask": mask, "renorm": renorm, "ends": ends, "layers": layers,
         "d": d, "inplace": inplace and n == K, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the newest token of each of 16 sequences: latency counts
        _embed("embed step B16 d512", 16, 1, 512, 32768),
        # the encoder's ordinary batch over a large catalogue
        _embed("embed fwd B32 L2048 d512", 32, 2048, 512, 262144),
        # the training step's batch, a vocabulary of which most rows occur, some of them thousands of times
        _embed("embed train B16 L8192 d512", 16, 8192, 512, 32768, train=True),
        # items named by four hashes into one shared table of a million short rows, most of which a batch has none of
        _embed("embed train 4 hashes d128", 32, 2048, 128, 1048576, train=True, k=4, form="varlen", lo=64),
        # a small odd fp32 table, padded, 64-bit ids: latency and ragged edges
        _embed("embed train f32 B3 L341 d73", 3, 341, 73, 1000, dtype="f32", train=True, form="padded", lo=0, wide=True),
        # one token of 16 sequences between two layers
        _norm("norm step B16 d512", 16, 1, 512),
        # a block's entry in the encoder's ordinary batch: residual stream and norm
        _norm("norm fwd B32 L2048 d512", 32, 2048, 512),
        # the training step's batch
        _norm("norm train B16 L8192 d512", 16, 8192, 512, train=True),
        # an odd fp32 layer, padded
        _norm("norm train f32 B5 L401 d201", 5, 401, 201, dtype="f32", train=True, form="padded", lo=0),
        # one user's next code out of a codebook: latency
        _beam("beam B1 K8 V256", 1, 8, 256, 8),
        # an ordinary decoding batch, 12 layers' states
        _beam("beam B64 K16 V32768", 64, 16, 32768, 16, layers=12),
        # wide beams over a codebook, only codes that continue a known item, some beams at their end
        _beam("beam B32 K256 V2048 valid", 32, 256, 2048, 256, dtype="f32", mask=0.1, renorm=True, ends=True, layers=6, inplace=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["embed", "norm", "beam"])
    if kind == "beam":
        while True:
            B, K, V = _log_int(rng, 1, 256), _log_int(rng, 1, 256), _log_int(rng, 16, 131072)
            d, layers = _log_int(rng, 8, 1024), _log_int(rng, 1, 24)
            if B * K * V <= 30_000_000 and B * K * d * layers <= 25_000_000:
                break
        n = K if rng.random() < 0.75 else min(256, V, _log_int(rng, 1, 256))
        return _beam(None, B, K, V, n, dtype=rng.choice(["bf16", "f32"]), mask=rng.choice([0.0, 0.0, 0.01, 0.3]), renorm=rng.random() < 0.5,
                     ends=rng.random() < 0.4, layers=layers, d=d, inplace=rng.random() < 0.6, pad=rng.choice([0, 0, 1, 8]))
    step = rng.random() < 0.15
    form = "dense" if step else rng.choice(["dense", "padded", "varlen"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = not step and rng.random() < 0.6
    while True:
        d = rng.choice([64, 128, 256, 512, 1024, _log_int(rng, 8, 2048)])
        L = 1 if step else _log_int(rng, 2, 32768)
        B = _log_int(rng, 1, 512)
        k = rng.choice([1, 1, 2, 4]) if kind == "embed" else 1
        V = _log_int(rng, 64, 1048576)
        if B * L * d * k <= 50_000_000 and (kind == "norm" or V * d <= 130_000_000):
            break
    lo = rng.randint(0, min(L, 64))
    if kind == "embed":
        return _embed(None, B, L, d, V, dtype=dtype, train=train, form=form, lo=lo, k=k, wide=rng.random() < 0.3)
    return _norm(None, B, L, d, dtype=dtype, train=train, form=form, lo=lo, res=rng.random() < 0.7, affine=rng.random() < 0.85,
                 cols=rng.random() < 0.2)


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


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    es, d = _es(case), case.get("d")
    if case["op"] == "beam":
        rows, out = case["B"] * case["K"], case["B"] * case["n"]
        b = rows * (case["V"] * es + 4 + (1 if case["ends"] else 0)) + out * 13
        if case["mask"]:
            b += rows * -(-case["V"] // 32) * 4
        # a state is read and written once for each beam that goes on
        return {"bytes": b + out * d * 4 * 2 * case["layers"], "flops": 4 * rows * case["V"]}
    n = sum(_lengths(case))
    if case["op"] == "embed":
        ids = n * case["k"]
        seen = min(ids, case["V"])  # each row of the table is read once at most
        b = ids * (8 if case["wide"] else 4) + seen * d * es + ids * d * es
        if case["train"]:  # after the rest of the net: ids and dy in, the whole gradient out
            b += ids * (8 if case["wide"] else 4) + ids * d * es + case["V"] * d * 4
        return {"bytes": b, "flops": (2 if case["train"] else 1) * ids * d}
    b = n * d * es * (4 if case["res"] else 2) + (2 * d * es if case["affine"] else 0)
    if case["train"]:  # s, dy (and the residual's gradient) in, dx, dw and db out
        b += n * d * es * (4 if case["res"] else 3) + (d * es + 8 * d if case["affine"] else 0)
    return {"bytes": b, "flops": (20 if case["train"] else 8) * n * d}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _gen(seed)
    f = dict(generator=g, device="cuda", dtype=torch.float32)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = {"case": case}
    if case["op"] == "beam":
        B, K, V, n = case["B"], case["K"], case["V"], case["n"]
        # a language model's logits: a few tokens far above the rest, rows of a matrix product's padded output
        logits = torch.randn(B * K, V + case["pad"], **f) * 2
        logits += (torch.rand(B * K, V + case["pad"], **f) < 8 / V) * 6
        s["logits"] = logits.to(dt)[:, :V]
        s["scores"] = torch.sort(-4 * torch.rand(B, K, **f), dim=1, descending=True).values.contiguous()
        if case["mask"]:
            words = -(-V // 32)
            ok = torch.rand(B * K, words * 32, **f) < case["mask"]
            ok = ok.view(B * K, words, 32).long()
            bits = (ok << torch.arange(32, device="cuda")).sum(2)
            s["allowed"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
        if case["ends"]:
            s["done"] = torch.rand(B, K, **f) < 0.1
        s["states"] = [torch.randn(B * K, case["d"], **f) for _ in range(case["layers"])]
        if not case["inplace"]:
            s["next"] = [torch.empty(B * n, case["d"], device="cuda") for _ in range(case["layers"])]
        return s
    ln, B, d = _lengths(case), case["B"], case["d"]
    rows = sum(ln) if case["form"] == "varlen" else B * case["L"]
    s["rows"] = rows
    if case["form"] == "varlen":
        s["cu"] = torch.tensor([0] + ln, device="cuda").cumsum(0).to(torch.int32)
    elif case["form"] == "padded":
        s["seq_lens"] = torch.tensor(ln, dtype=torch.int32, device="cuda")
    if case["op"] == "embed":
        V, k = case["V"], case["k"]
        ids = torch.exp(math.log(V + 1) * torch.rand(rows, k, **f)).long() - 1
        ids = (ids.clamp(0, V - 1) * 7919 + 13) % V  # frequent ids anywhere in the table
        ids = torch.where(torch.rand(rows, k, **f) < 0.01, -1, ids)
        s["ids"] = ids if case["wide"] else ids.to(torch.int32)
        s["table"] = (torch.randn(V, d, **f) * 0.05).to(dt)
        s["scale"] = math.sqrt(d)
        if case["train"]:
            s["dy"] = torch.randn(rows, k * d, **f).to(dt)
        return s
    x = torch.randn(rows, d * (2 if case["cols"] else 1), **f) * (0.5 + torch.rand(1, **f)) + 0.3
    s["x"] = x.to(dt)[:, :d]  # the first columns of a wider projection, or a tensor of its own
    if case["res"]:
        s["res"] = (torch.randn(rows, d, **f) * 2).to(dt)
    if case["affine"]:
        s["w"] = (1 + 0.1 * torch.randn(d, **f)).to(dt)
        s["b"] = (0.1 * torch.randn(d, **f)).to(dt)
    if case["train"]:
        s["dy"] = torch.randn(rows, d, **f).to(dt)
        if case["res"]:
            s["ds"] = torch.randn(rows, d, **f).to(dt)
    return s


# ------------------------------------------------------------- plain forms
def _valid(st):
    """[rows, 1], true in rows that belong to a sequence."""
    case = st["case"]
    if case["form"] != "padded":
        return torch.ones(st["rows"], 1, dtype=torch.bool, device="cuda")
    return (torch.arange(case["L"], device="cuda")[None, :] < st["seq_lens"][:, None].long()).view(-1, 1)


def _plain_embed(st):
    case = st["case"]
    d, V, k = case["d"], case["V"], case["k"]
    ids = st["ids"].long()
    has = (ids >= 0) & _valid(st)
    at = torch.where(has, ids, 0).view(-1)
    y = st["table"][at].float() * st["scale"]
    y = torch.where(has.view(-1, 1), y, 0.0).to(st["table"].dtype).view(-1, k * d)
    if not case["train"]:
        return {"y": y}
    dy = torch.where(has.view(-1, 1), st["dy"].view(-1, d).double(), 0.0)  # a frequent id's sum is long
    grad = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, at, dy)
    return {"y": y, "dtable": (grad * st["scale"]).float()}


def _plain_norm(st):
    case = st["case"]
    dt, v = st["x"].dtype, _valid(st)
    s = st["x"].float()
    out = {}
    if case["res"]:
        out["s"] = torch.where(v, s + st["res"].float(), 0.0).to(dt)
        s = out["s"].float()
    m = s.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((s - m) * (s - m)).mean(1, keepdim=True) + EPS)
    z = (s - m) * r
    w, b = (st["w"].float(), st["b"].float()) if case["affine"] else (1.0, 0.0)
    out["y"] = torch.where(v, z * w + b, 0.0).to(dt)
    if not case["train"]:
        return out
    dy = torch.where(v, st["dy"].float(), 0.0)
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True))
    if case["res"]:
        dx = dx + st["ds"].float()
    out["dx"] = torch.where(v, dx, 0.0).to(dt)
    if case["affine"]:
        out["dw"] = (dy * z).sum(0, dtype=torch.float64).float()
        out["db"] = dy.sum(0, dtype=torch.float64).float()
    return out


def _bits(st):
    """The mask's bits as [B K, V] truth values."""
    w = st["allowed"].long() & 0xFFFFFFFF
    return ((w[:, :, None] >> torch.arange(32, device="cuda")) & 1).bool().view(w.shape[0], -1)[:, :st["case"]["V"]]


def _plain_beam(st):
    case = st["case"]
    B, K, V, n = case["B"], case["K"], case["V"], case["n"]
    x = st["logits"].double()  # which of two beams is ahead is a matter of far digits
    if case["mask"]:
        ok = _bits(st)
        if case["renorm"]:
            x = torch.where(ok, x, -math.inf)
    top = x.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    score = st["scores"].double().view(-1, 1) + (x - lse)
    if case["mask"]:
        score = torch.where(ok, score, -math.inf)
    if case["ends"]:  # an ended beam goes on as itself
        done = st["done"].view(-1, 1)
        is_eos = torch.arange(V, device="cuda") == EOS
        score = torch.where(done, torch.where(is_eos, st["scores"].double().view(-1, 1), -math.inf), score)
    score = torch.where(score > -math.inf, score, -math.inf)  # NaN: no candidate
    best, at = torch.sort(score.view(B, K * V), dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    if best.shape[1] < n:
        more = n - best.shape[1]
        best = torch.cat([best, torch.full((B, more), -math.inf, dtype=best.dtype, device="cuda")], 1)
        at = torch.cat([at, torch.zeros(B, more, dtype=at.dtype, device="cuda")], 1)
    live = best > -math.inf
    parent = torch.where(live, at // V, 0)
    token = torch.where(live, at % V, -1)
    out = {"scores": best.float(), "tokens": token.to(torch.int32), "parents": parent.to(torch.int32)}
    if case["ends"]:
        out["done"] = live & (torch.gather(st["done"], 1, parent) | (token == EOS))
    rows = (parent + torch.arange(B, device="cuda")[:, None] * K).view(-1)
    moved = [s[rows] for s in st["states"]]
    for a, b in zip(st["states"] if case["inplace"] else st["next"], moved):
        a.copy_(b)
    out["states"] = st["states"] if case["inplace"] else st["next"]
    return out


# ----------------------------------------------------- the framework's calls
def _shape(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    n = case["B"] if case["form"] != "varlen" else 1
    rows = case["L"] if case["form"] != "varlen" else st["rows"]
    return gbla.glr_shape(n, rows, case["d"], dtype=case["dtype"], cu_seqlens=st.get("cu"), seq_lens=st.get("seq_lens"))


def _own_embed(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    if "shape" not in st:  # what a program keeps: the shape and its workspace
        st["shape"] = _shape(st)
        st["ws"] = gbla.embed_workspace(st["shape"], case["V"], case["k"], backward=case["train"])
    y = gbla.embed_forward(st["shape"], st["ids"], st["table"], scale=st["scale"], ws=st["ws"])
    if not case["train"]:
        return {"y": y}
    return {"y": y, "dtable": gbla.embed_backward(st["shape"], st["ids"], st["dy"], case["V"], scale=st["scale"], ws=st["ws"])}


def _own_norm(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    if "shape" not in st:
        st["shape"] = _shape(st)
        st["ws"] = gbla.layer_norm_workspace(st["shape"], backward=case["train"])
    w, b = st.get("w"), st.get("b")
    y, total, stats = gbla.layer_norm_forward(st["shape"], st["x"], w, b, eps=EPS, res=st.get("res"), stats=case["train"] or None,
                                              ws=st["ws"])
    out = {"y": y}
    if case["res"]:
        out["s"] = total
    if case["train"]:
        g = gbla.layer_norm_backward(st["shape"], total if case["res"] else st["x"], w, stats, st["dy"], ds=st.get("ds"),
                                     affine=case["affine"], ws=st["ws"])
        out.update(g)
    return out


def _own_beam(st):
    from generative_retrieval_encoder_gb300 import gbla
    case = st["case"]
    if "beam" not in st:
        st["beam"] = gbla.beam_shape(case["B"], case["K"], case["V"], case["n"], dtype=case["dtype"], eos=EOS if case["ends"] else -1,
                                     over_allowed=case["renorm"])
        st["ws"] = gbla.beam_workspace(st["beam"])
        st["plan"] = gbla.beam_reorder_plan(st["beam"], st["states"], None if case["inplace"] else st["next"])
    scores, tokens, parents, done = gbla.beam_select(st["beam"], st["logits"], st["scores"], allowed=st.get("allowed"), done=st.get("done"),
                                                     ws=st["ws"])
    gbla.beam_reorder(st["plan"], parents)
    out = {"scores": scores, "tokens": tokens, "parents": parents, "states": st["states"] if case["inplace"] else st["next"]}
    if case["ends"]:
        out["done"] = done
    return out


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# --------------------------------------------------------- in 64 bits
def _rows_of(case):
    """The rows that belong to a sequence."""
    if case["form"] != "padded":
        return None
    return torch.tensor([b * case["L"] + t for b, n in enumerate(_lengths(case)) for t in range(n)], dtype=torch.long, device="cuda")


def _exact_embed(st):
    case, T = st["case"], st["table"].double()
    d, k = case["d"], case["k"]
    ids = st["ids"].long().clone()
    rows = _rows_of(case)
    if rows is not None:
        keep = torch.zeros(ids.shape[0], dtype=torch.bool, device="cuda")
        keep[rows] = True
        ids[~keep] = -1
    ids = ids.view(-1)
    y = torch.zeros(ids.numel(), d, dtype=torch.float64, device="cuda")
    there = (ids >= 0).nonzero()[:, 0]
    y[there] = T[ids[there]] * st["scale"]
    out = {"y": y.view(-1, k * d)}
    if case["train"]:  # tokens by id, each id's run from the running sums of its gradients
        order = there[torch.argsort(ids[there], stable=True)]
        key, count = torch.unique_consecutive(ids[order], return_counts=True)
        grad = torch.zeros(case["V"], d, dtype=torch.float64, device="cuda")
        dy = st["dy"].view(-1, d)
        end = count.cumsum(0)
        width = max(1, (1 << 26) // max(1, order.numel()))
        for c in range(0, d, width):  # columns at a time: the running sums are large
            part = dy[order, c:c + width].double()
            run = torch.cat([torch.zeros_like(part[:1]), part.cumsum(0)])
            grad[key, c:c + width] = run[end] - run[end - count]
        out["dtable"] = grad * st["scale"]
    return out


def _exact_norm(st):
    case, dt = st["case"], st["x"].dtype
    rows = _rows_of(case)
    pick = (lambda t: t) if rows is None else (lambda t: t[rows])

    def put(t):
        if rows is None:
            return t
        o = torch.zeros(st["rows"], t.shape[1], dtype=t.dtype, device="cuda")
        o[rows] = t
        return o
    s = pick(st["x"]).double()
    out = {}
    if case["res"]:  # what is normed is the sum as it is stored
        s = s + pick(st["res"]).double()
        out["s"] = put(s)
        s = s.to(dt).double()
    var, mean = torch.var_mean(s, dim=1, unbiased=False, keepdim=True)
    r = (var + EPS).rsqrt()
    z = (s - mean) * r
    w = st["w"].double() if case["affine"] else torch.ones(case["d"], dtype=torch.float64, device="cuda")
    out["y"] = put(z * w + st["b"].double() if case["affine"] else z)
    if case["train"]:
        dy = pick(st["dy"]).double()
        g = dy * w
        D = case["d"]
        dx = r / D * (D * g - g.sum(1, keepdim=True) - z * (g * z).sum(1, keepdim=True))
        out["dx"] = put(dx + pick(st["ds"]).double() if case["res"] else dx)
        if case["affine"]:
            out["dw"], out["db"] = (dy * z).sum(0), dy.sum(0)
    return out


def _exact_beam(st):
    """Group by group: every beam's best n tokens, then the best n of those."""
    case = st["case"]
    B, K, V, n = case["B"], case["K"], case["V"], case["n"]
    dev = "cuda"
    scores, tokens, parents = [], [], []
    lanes = torch.arange(V, device=dev)
    for g in range(B):
        x = st["logits"][g * K:(g + 1) * K].double()
        ok = torch.ones(K, V, dtype=torch.bool, device=dev)
        if case["mask"]:
            w = st["allowed"][g * K:(g + 1) * K].long()
            ok = ((w[:, lanes // 32] >> (lanes % 32)) & 1) == 1
        base = st["scores"][g].double()
        p = torch.log_softmax(x.masked_fill(~ok, -math.inf) if case["renorm"] else x, dim=1) + base[:, None]
        p = p.masked_fill(~ok, -math.inf)
        if case["ends"]:
            e = st["done"][g]
            p[e] = -math.inf
            p[e, EOS] = base[e]
        p = torch.nan_to_num(p, nan=-math.inf)
        m = min(n, V)
        v, t = torch.sort(p, dim=1, descending=True, stable=True)
        v, t = v[:, :m].reshape(-1), t[:, :m].reshape(-1)
        b = torch.arange(K, device=dev).repeat_interleave(m)
        v, o = torch.sort(v, descending=True, stable=True)
        v, t, b = v[:n], t[o][:n], b[o][:n]
        gone = ~(v > -math.inf)
        t, b = t.masked_fill(gone, -1), b.masked_fill(gone, 0)
        fill = n - v.numel()
        pad = lambda q, c: torch.cat([q, torch.full((fill,), c, dtype=q.dtype, device=dev)])  # noqa: E731
        scores.append(pad(v, -math.inf))
        tokens.append(pad(t, -1))
        parents.append(pad(b, 0))
    tokens, parents = torch.stack(tokens), torch.stack(parents)
    out = {"scores": torch.stack(scores), "tokens": tokens, "parents": parents}
    if case["ends"]:
        out["done"] = (torch.gather(st["done"], 1, parents) | (tokens == EOS)) & (tokens >= 0)
    out["states"] = [s.view(B, K, -1)[torch.arange(B, device=dev)[:, None], parents].reshape(B * n, -1).double() for s in st["states"]]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](st)
