"""fp64 oracle of differential attention and of rotary positions, from their definitions, on the CPU.

O = P1 V - lam P2 V with P_m = softmax(scale q_m k_m^T) over the visible keys, q = [q1 | q2] and
k = [k1 | k2] by columns.  Plain loops over batch and heads, two-pass softmax; shares no code with
the GPU path.  Beside each value comes its magnitude sum (the same sum over absolute terms), from
which the tests derive elementwise error bounds.
"""
from __future__ import annotations

import math

import torch


def _maps(q, k, keep, scale):
    """P and LSE of both maps for one head: q [S, d], k [T, d], keep [S, T]."""
    h = q.shape[-1] // 2
    P, L = [], []
    for part in (slice(0, h), slice(h, 2 * h)):
        s = scale * (q[:, part] @ k[:, part].T)
        s = s.masked_fill(~keep, -math.inf)
        m = s.max(-1).values if s.shape[1] else torch.full((s.shape[0],), -math.inf, dtype=s.dtype)
        ms = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        e = torch.exp(s - ms[:, None])
        l = e.sum(-1)
        P.append(e / torch.where(l > 0, l, torch.ones_like(l))[:, None])
        L.append(torch.where(l > 0, ms + torch.log(torch.where(l > 0, l, torch.ones_like(l))), torch.full_like(l, -math.inf)))
    return P, L


def visible(S, T, causal, length=None):
    keep = torch.ones(S, T, dtype=torch.bool)
    if causal:
        keep = keep.tril()
    if length is not None:
        keep = keep & (torch.arange(T) < length)[None, :]
    return keep


def forward(q, k, v, lam, causal, scale=None, lens=None):
    """(O, LSE [B, Hq, 2, S], O2, magnitude sums of O) in fp64."""
    q, k, v, lam = (t.double() for t in (q, k, v, lam))
    B, Hq, S, d = q.shape
    T, g = k.shape[2], Hq // k.shape[1]
    scale = 1.0 / math.sqrt(d // 2) if scale is None else scale
    O, O2, mag = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    L = torch.zeros(B, Hq, 2, S, dtype=torch.float64)
    for b in range(B):
        keep = visible(S, T, causal, None if lens is None else int(lens[b]))
        seen = keep.any(0)
        for h in range(Hq):
            vb = torch.where(seen[:, None], v[b, h // g], torch.zeros(()).double())
            kb = torch.where(seen[:, None], k[b, h // g], torch.zeros(()).double())
            P, l = _maps(q[b, h], kb, keep, scale)
            w = lam[h if lam.numel() > 1 else 0]
            O2[b, h] = P[1] @ vb
            O[b, h] = P[0] @ vb - w * O2[b, h]
            mag[b, h] = P[0] @ vb.abs() + w.abs() * (P[1] @ vb.abs())
            L[b, h, 0], L[b, h, 1] = l
    return O, L, O2, mag


def backward(q, k, v, lam, dO, causal, scale=None):
    """{name: (gradient, magnitude sums)} for q, k, v and lam.  The magnitude sums of dQ and dK take
    |dS| + P * (the magnitude sum of D), those of dV take P1 + |lam| P2."""
    dtype_lam = lam
    q, k, v, lam, dO = (t.double() for t in (q, k, v, lam, dO))
    B, Hq, S, d = q.shape
    Hkv, h2 = k.shape[1], d // 2
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(h2) if scale is None else scale
    out = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in (("q", q), ("k", k), ("v", v), ("lam", dtype_lam.double()))}
    keep = visible(S, S, causal)
    for b in range(B):
        for h in range(Hq):
            j, i = h // g, h if lam.numel() > 1 else 0
            P, _ = _maps(q[b, h], k[b, j], keep, scale)
            w, G, V = lam[i], dO[b, h], v[b, j]
            out["v"][0][b, j] += (P[0] - w * P[1]).T @ G
            out["v"][1][b, j] += (P[0] + w.abs() * P[1]).T @ G.abs()
            dP = G @ V.T
            o = [P[0] @ V, P[1] @ V]
            # D of the first map is computed from O + lam O2
            dmag = [(G * (o[0] - w * o[1])).abs().sum(-1) + (w * G * o[1]).abs().sum(-1), (G * o[1]).abs().sum(-1)]
            for m, part in enumerate((slice(0, h2), slice(h2, d))):
                c = 1.0 if m == 0 else -w
                dS = c * P[m] * (dP - (G * o[m]).sum(-1, keepdim=True))
                dSm = dS.abs() + abs(c) * P[m] * dmag[m][:, None]
                out["q"][0][b, h][:, part] += scale * dS @ k[b, j][:, part]
                out["q"][1][b, h][:, part] += scale * dSm @ k[b, j][:, part].abs()
                out["k"][0][b, j][:, part] += scale * dS.T @ q[b, h][:, part]
                out["k"][1][b, j][:, part] += scale * dSm.T @ q[b, h][:, part].abs()
            out["lam"][0][i] -= (G * o[1]).sum()
            out["lam"][1][i] += (P[1] * dP.abs()).sum()
    return out


def rope(x, positions, freq, axis, groups=1, adjacent=False, inverse=False):
    """Rotated x [B, H, S, d] in fp64 and the magnitude |a| + |b| of each element's pair; positions
    [axes, B, S] integers."""
    x = x.double()
    n, dh = len(freq), x.shape[-1] // groups
    y, mag = x.clone(), x.abs().clone()
    for i in range(n):
        phi = positions[axis[i]].double() * freq[i] * (-1.0 if inverse else 1.0)
        c, s = torch.cos(phi)[:, None, :], torch.sin(phi)[:, None, :]
        for g in range(groups):
            a, b = (g * dh + 2 * i, g * dh + 2 * i + 1) if adjacent else (g * dh + i, g * dh + n + i)
            xa, xb = x[..., a], x[..., b]
            y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
            mag[..., a] = mag[..., b] = xa.abs() + xb.abs()
    return y, mag
