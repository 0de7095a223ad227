"""fp64 oracle of attention whose scores are capped, biased by distance and masked by a range of keys a row, from its definition,
on the CPU, and of the same over a paged cache.

x_ij = cap tanh(scale q_i.k_j / cap) (or scale q_i.k_j) - slope_h |i - j| over lo_i <= j < hi_i, O = softmax(x) V.  Plain loops over
batch and heads; shares no code with the GPU path.  Beside each value comes its magnitude sum (the same sum over absolute
terms), from which the tests derive elementwise error bounds.
"""
from __future__ import annotations

import math

import torch


def scores(q, k, far, keep, scale, cap, slope):
    """(x, t) of one head: masked scores [S, T] and the cap's tanh (zeros without one)."""
    x = scale * (q @ k.T)
    t = torch.zeros_like(x)
    if cap:
        t = torch.tanh(x / cap)
        x = cap * t
    x = x - slope * far.abs().double()
    return x.masked_fill(~keep, -math.inf), t


def softmax(x):
    """(P, LSE) of rows, zeros and -inf for a row without a key."""
    if x.shape[1] == 0:
        return x, torch.full((x.shape[0],), -math.inf, dtype=x.dtype)
    m = x.max(-1).values
    ms = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - ms[:, None])
    l = e.sum(-1)
    safe = torch.where(l > 0, l, torch.ones_like(l))
    return e / safe[:, None], torch.where(l > 0, ms + torch.log(safe), torch.full_like(l, -math.inf))


def visible(lo, hi, S):
    j = torch.arange(S)
    return (j >= lo.long()[:, None]) & (j < hi.long()[:, None])


def _ranges_of(lo, b):
    return lo if lo.dim() == 1 else lo[min(b, lo.shape[0] - 1)]


def forward(q, k, v, lo, hi, scale=None, cap=0.0, slopes=None):
    """(O, LSE [B, Hq, S], magnitude sums of O)."""
    q, k, v = (t.double() for t in (q, k, v))
    B, Hq, S, d = q.shape
    g = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    far = torch.arange(S)[:, None] - torch.arange(S)
    O, mag, L = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(B, Hq, S, dtype=torch.float64)
    for b in range(B):
        keep = visible(_ranges_of(lo, b), _ranges_of(hi, b), S)
        for h in range(Hq):
            x, _ = scores(q[b, h], k[b, h // g], far, keep, scale, cap, 0.0 if slopes is None else float(slopes[h]))
            P, L[b, h] = softmax(x)
            O[b, h], mag[b, h] = P @ v[b, h // g], P @ v[b, h // g].abs()
    return O, L, mag


def backward(q, k, v, g_out, lo, hi, scale=None, cap=0.0, slopes=None):
    """{name: (gradient, magnitude sums)} of q, k, v."""
    q, k, v, go = (t.double() for t in (q, k, v, g_out))
    B, Hq, S, d = q.shape
    g = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    far = torch.arange(S)[:, None] - torch.arange(S)
    out = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in (("q", q), ("k", k), ("v", v))}
    for b in range(B):
        keep = visible(_ranges_of(lo, b), _ranges_of(hi, b), S)
        for h in range(Hq):
            j = h // g
            x, t = scores(q[b, h], k[b, j], far, keep, scale, cap, 0.0 if slopes is None else float(slopes[h]))
            P, _ = softmax(x)
            O = P @ v[b, j]
            dP = go[b, h] @ v[b, j].T
            f = P * (1.0 - t * t)
            dS = f * (dP - (go[b, h] * O).sum(-1, keepdim=True))
            # what a rounding of O in D, or of P and dS, is relative to
            dmag = (go[b, h].abs() * (O.abs() + P @ v[b, j].abs())).sum(-1, keepdim=True)
            smag = dS.abs() + dmag * f
            out["q"][0][b, h] = scale * (dS @ k[b, j])
            out["q"][1][b, h] = scale * (smag @ k[b, j].abs())
            out["k"][0][b, j] += scale * (dS.T @ q[b, h])
            out["k"][1][b, j] += scale * (smag.T @ q[b, h].abs())
            out["v"][0][b, j] += P.T @ go[b, h]
            out["v"][1][b, j] += P.T @ go[b, h].abs()
    return out


def gather(pages, table, b, length):
    """The first `length` tokens of sequence b: [Hkv, length, d] of pages [n_pages, Hkv, page, d]."""
    page = pages.shape[2]
    rows = [pages[int(table[b, i // page]), :, i % page] for i in range(length)]
    return torch.stack(rows, 1) if rows else pages.new_zeros(pages.shape[1], 0, pages.shape[3])


def paged(q, k_pages, v_pages, table, offsets, lens, scale=None, cap=0.0, slopes=None, window=0):
    """(O [N, Hq, d], LSE [N, Hq], magnitude sums) of the new tokens; rows of no sequence stay zero."""
    N, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    O, mag, L = (torch.zeros(N, Hq, d, dtype=torch.float64), torch.zeros(N, Hq, d, dtype=torch.float64),
                 torch.zeros(N, Hq, dtype=torch.float64))
    for b in range(len(lens)):
        o0, o1, T = int(offsets[b]), int(offsets[b + 1]), int(lens[b])
        if o0 == o1:
            continue
        k, v = (gather(p, table, b, T).double() for p in (k_pages, v_pages))
        far = torch.arange(T - (o1 - o0), T)[:, None] - torch.arange(T)
        keep = far >= 0
        if window:
            keep = keep & (far < window)
        for h in range(Hq):
            x, _ = scores(q[o0:o1, h].double(), k[h // g], far, keep, scale, cap, 0.0 if slopes is None else float(slopes[h]))
            P, L[o0:o1, h] = softmax(x)
            O[o0:o1, h], mag[o0:o1, h] = P @ v[h // g], P @ v[h // g].abs()
    return O, L, mag
