"""The gated linear recurrence in 64 bits, token by token from its formulas,
with the bound that fp32 gates and states and one rounding of each output keep
to (no constant of it is fitted to a result):

* a gate's relative error is at most K = 5e-6 (for logits up to 8; in
  proportion beyond): the exponent's argument |r| 2^-24 * 1.5, ex2 2^-22, rcp
  2^-23, the series or 1 - e^-s 1.2e-6, rsqrt 2^-22, and the products' 2^-24;
* the decay's absolute error is at most K q + 2^-24 with q = 1 - a, so an error
  E of the state obeys E_t <= a E_{t-1} + (K q + 2^-24) |h_{t-1}| + K |u| + 2^-24 |h_t|
  (twice the state's two roundings: the kernels may regroup the products);
* w obeys the same recurrence backwards, and each gradient is a product of
  these with first-order bounds; a sum of n terms adds 2^-24 * 200 times the
  sum of magnitudes (the longest chain of additions of the reductions);
* an output is rounded once: 2^-8 (bf16) or 2^-24 (fp32) of its value.
"""
from __future__ import annotations

import numpy as np
import torch

from generative_retrieval_encoder_gb300 import gbla

K, E32 = 5e-6, 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 1e-30


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def gates(x, r, i, lam, c):
    sr, gi = sigmoid(r), sigmoid(i)
    s = c * softplus(lam) * sr
    a, q = np.exp(-s), -np.expm1(-s)
    m = np.sqrt(q * (2 - q))
    with np.errstate(divide="ignore", invalid="ignore"):
        sm = np.where(m > 0, s / m, 0.0)
    return sr, gi, s, a, q, m, sm


def reference(x, r, i, lam, c, starts, lens, reverse=False, h0=None, dy=None, dhT=None, io="bf16"):
    """{name: (value, bound)} of y, hT and, given dy, dx, dr, di, dlam, dh0 (64-bit arrays of the rows of [T, d])."""
    T, d = x.shape
    n = len(starts)
    with np.errstate(over="ignore", invalid="ignore"):
        sr, gi, s, a, q, m, sm = gates(x, r, i, lam, c)
        k = K * np.maximum(1, np.maximum(np.abs(r), np.abs(i)).clip(max=200) / 8)
        u = m * gi * x
    H, EH, P, EP = (np.zeros((T, d)) for _ in range(4))
    hT, ET = np.zeros((n, d)), np.zeros((n, d))
    W, EW = np.zeros((T, d)), np.zeros((T, d))
    dh0, E0 = np.zeros((n, d)), np.zeros((n, d))
    for b in range(n):
        rows = list(range(starts[b], starts[b] + lens[b]))
        if reverse:
            rows.reverse()
        h, e = (h0[b].copy() if h0 is not None else np.zeros(d)), np.zeros(d)
        for t in rows:
            P[t], EP[t] = h, e
            e = a[t] * e + (k[t] * q[t] + E32) * np.abs(h) + k[t] * np.abs(u[t])
            h = a[t] * h + u[t]
            e = e + E32 * np.abs(h)
            H[t], EH[t] = h, e
        hT[b], ET[b] = h, e
        if dy is not None:
            w, e = (dhT[b].copy() if dhT is not None else np.zeros(d)), np.zeros(d)
            for t in reversed(rows):
                w = w + dy[t]
                e = e + E32 * np.abs(w)
                W[t], EW[t] = w, e
                e = a[t] * e + (k[t] * q[t] + E32) * np.abs(w)
                w = a[t] * w
            dh0[b], E0[b] = w, e
    hs = HALF_STEP[io]
    out = {"y": (H, EH + hs * np.abs(H)), "hT": (hT, ET + E32 * np.abs(hT))}
    if dy is None:
        return out
    valid = np.zeros((T, 1), bool)
    for b in range(n):
        valid[starts[b]:starts[b] + lens[b]] = True
    z = lambda v: np.where(valid, v, 0.0)  # noqa: E731
    G = z(a * s * P - gi * x * a * a * sm)
    BG = z(a * s * EP + k * (np.abs(a * s * P) + 3 * np.abs(gi * x * a * a * sm)))
    e, Be = -W * G, EW * np.abs(G) + np.abs(W) * BG + 4 * E32 * np.abs(W * G)
    dx, di, dr = z(W * m * gi), z(W * m * x * gi * (1 - gi)), e * (1 - sr)
    Bd = lambda v, f: (EW * np.abs(f) + 3 * k * np.abs(v))  # noqa: E731
    # 1 - sigmoid is formed by a subtraction: an absolute error of 2^-24 and the sigmoid's relative one
    lost = 2 * E32 + k * gi
    out["dx"] = dx, z(Bd(dx, m * gi)) * (1 + hs) + hs * np.abs(dx)
    out["di"] = di, z(Bd(di, m * x * gi * (1 - gi)) + lost * np.abs(W * m * x * gi)) + hs * np.abs(di)
    out["dr"] = dr, z(Be * (1 - sr) + (2 * E32 + k * sr) * np.abs(e)) + hs * np.abs(dr)
    ratio = sigmoid(lam) / np.maximum(softplus(lam), TINY)
    ratio = np.where(lam < -30, 1.0, ratio)
    dlam = e.sum(0) * ratio
    out["dlam"] = dlam, (Be.sum(0) + (200 * E32 + 4 * E32) * np.abs(e).sum(0)) * ratio + K * np.abs(dlam)
    out["dh0"] = dh0, E0 + E32 * np.abs(dh0)
    return out


def check(got: dict, want: dict, floor=1e-30):
    for n, t in got.items():
        if t is None:
            continue
        v, bound = want[n]
        g = t.detach().double().cpu().numpy()
        assert g.shape == v.shape, (n, g.shape, v.shape)
        assert np.isfinite(g).all(), f"{n}: {np.count_nonzero(~np.isfinite(g))} values are not finite"
        off = np.abs(g - v) - bound
        assert (off <= floor).all(), f"{n}: off by up to {np.abs(g - v).max():.3g}, {off.max():.3g} over its bound"


class Case:
    """Seeded inputs on the GPU and their exact 64-bit values."""

    def __init__(self, dtype, d, L=None, B=1, seq_lens=None, lengths=None, reverse=False, state=True, packed=False, seed=0,
                 c=8.0, lam=None):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.dtype, self.d, self.c, self.reverse, self.packed = dtype, d, c, reverse, packed
        if lengths is not None:
            self.lens, self.n = list(lengths), len(lengths)
            self.starts = np.concatenate([[0], np.cumsum(self.lens)[:-1]]).astype(int).tolist()
            self.T = sum(self.lens)
            cu = torch.tensor([0] + np.cumsum(self.lens).tolist(), dtype=torch.int32).cuda()
            self.shape = gbla.glr_shape(1, self.T, d, dtype=dtype, cu_seqlens=cu)
        else:
            self.n, self.T = B, B * L
            self.lens = list(seq_lens) if seq_lens is not None else [L] * B
            self.starts = [b * L for b in range(B)]
            sl = None if seq_lens is None else torch.tensor(seq_lens, dtype=torch.int32).cuda()
            self.shape = gbla.glr_shape(B, L, d, dtype=dtype, seq_lens=sl)
        T, n = self.T, self.n
        xri = [rn(T, d).to(dt) for _ in range(3)]
        if packed:
            buf = torch.cat(xri, 1).cuda()
            self.x, self.r, self.i = buf[:, :d], buf[:, d:2 * d], buf[:, 2 * d:]
        else:
            self.x, self.r, self.i = (t.cuda() for t in xri)
        if lam is None:  # decays at r = +inf from 0.9 to 0.999
            lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(d, generator=gen)) / 8.0))
        self.lam = lam.float().cuda()
        self.dy = rn(T, d).to(dt).cuda()
        self.h0 = rn(n, d).cuda() if state else None
        self.dhT = rn(n, d).cuda() if state else None

    def reference(self, backward=True):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return reference(f(self.x), f(self.r), f(self.i), f(self.lam), self.c, self.starts, self.lens, self.reverse, f(self.h0),
                         f(self.dy) if backward else None, f(self.dhT), self.dtype)

    def forward(self, **kw):
        return gbla.glr_forward(self.shape, self.x, self.r, self.i, self.lam, c=self.c, reverse=self.reverse, h0=self.h0, **kw)

    def backward(self, saved, **kw):
        return gbla.glr_backward(self.shape, self.x, self.r, self.i, self.lam, saved, self.dy, c=self.c, reverse=self.reverse,
                                 h0=self.h0, dhT=self.dhT, **kw)
