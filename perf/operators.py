"""Measured cases of the rotary positions and of differential attention: each operator in a plain form (elementary torch
operations in 32 bits) and as a user's program calls it, over the range of sizes, types and directions that it serves.

Operators (`op` of a case):
  rope    rotary positions with several axes on q and k [B, H, S, d], which arrive as the projection wrote them
          ([B, S, H, d] in memory); `dir` "bwd" takes gradients in the attention's layout back to the projection's
  diff    differential attention, O = (softmax(q1 k1^T s) - lam softmax(q2 k2^T s)) v with q = [q1 | q2], k = [k1 | k2]
          by columns and one lam a head; `dir` "fwd" is a prefill, "train" a forward and a backward pass
  decode  the same for one new token a sequence over a cache with lengths of its own
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one decoding step of a batch of 64: positions anywhere in a long context, differential heads
        {"name": "rope_step_b64", "op": "rope", "dir": "fwd", "B": 64, "S": 1, "Hq": 32, "Hkv": 8, "d": 128, "groups": 2,
         "axes": 3, "pairs": 32, "style": "half", "freq": "global", "dtype": BF16},
        # a long video and text sequence before its attention
        {"name": "rope_video_64k", "op": "rope", "dir": "fwd", "B": 1, "S": 65536, "Hq": 16, "Hkv": 4, "d": 128, "groups": 2,
         "axes": 3, "pairs": 32, "style": "half", "freq": "global", "dtype": BF16},
        # the gradient of rotated q and k of an image batch: rows and columns, part of the head rotated
        {"name": "rope_image_bwd", "op": "rope", "dir": "bwd", "B": 3, "S": 4107, "Hq": 12, "Hkv": 12, "d": 64, "groups": 1,
         "axes": 2, "pairs": 28, "style": "adjacent", "freq": "axial", "dtype": F32},
        # the tiny exact configuration: latency
        {"name": "diff_tiny_f32", "op": "diff", "dir": "fwd", "B": 1, "S": 512, "Hq": 2, "Hkv": 2, "d": 64, "P": 4,
         "causal": False, "dtype": F32},
        # the 16K causal configuration
        {"name": "diff_causal_16k", "op": "diff", "dir": "fwd", "B": 1, "S": 16384, "Hq": 16, "Hkv": 16, "d": 128, "P": 1,
         "causal": True, "dtype": BF16},
        # a batch of ragged length without a mask, shared KV heads
        {"name": "diff_ragged_gqa", "op": "diff", "dir": "fwd", "B": 2, "S": 2500, "Hq": 8, "Hkv": 2, "d": 128, "P": 4,
         "causal": False, "dtype": BF16},
        # training at 8K with shared KV heads
        {"name": "diff_train_8k", "op": "diff", "dir": "train", "B": 1, "S": 8192, "Hq": 16, "Hkv": 4, "d": 128, "P": 1,
         "causal": True, "dtype": BF16},
        # training of a small model with short ragged sequences
        {"name": "diff_train_small", "op": "diff", "dir": "train", "B": 2, "S": 1000, "Hq": 4, "Hkv": 4, "d": 64, "P": 1,
         "causal": True, "dtype": BF16},
        # training in fp32
        {"name": "diff_train_f32", "op": "diff", "dir": "train", "B": 1, "S": 777, "Hq": 4, "Hkv": 2, "d": 64, "P": 1,
         "causal": True, "dtype": F32},
        # one sequence with a context of 256K
        {"name": "decode_256k", "op": "decode", "B": 1, "T": 262144, "Hq": 16, "Hkv": 4, "d": 128, "dtype": BF16},
        # a served batch: lengths from none and one to the cache's end
        {"name": "decode_b64_ragged", "op": "decode", "B": 64, "T": 8192, "Hq": 32, "Hkv": 8, "d": 128, "dtype": BF16},
        # a few short sequences in fp32: latency
        {"name": "decode_f32_short", "op": "decode", "B": 4, "T": 1000, "Hq": 8, "Hkv": 4, "d": 64, "dtype": F32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "diff", "diff", "decode"])
    d = rng.choice([64, 128])
    dtype = rng.choice([BF16, BF16, F32])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4])
    if op == "rope":
        groups = rng.choice([1, 2])
        half = d // groups // 2
        B = rng.choice([1, 2, 3, 16])
        S = _log(rng, 1, 65536 // B)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "B": B, "S": S, "Hq": min(hq, 16), "Hkv": min(hkv, 4), "d": d,
                "groups": groups, "axes": rng.choice([1, 2, 3]), "pairs": rng.choice([half, half, half - 4, half - 3]),
                "style": rng.choice(["half", "adjacent"]), "freq": rng.choice(["global", "axial"]), "dtype": dtype}
    if op == "decode":
        T = _log(rng, 1, 65536)
        B = min(64, _log(rng, 1, max(1, 262144 // T)))
        return {"op": op, "B": B, "T": T, "Hq": hq, "Hkv": hkv, "d": d, "dtype": dtype}
    way = rng.choice(["fwd", "train"])
    P = rng.choice([1, 1, 4, 9])
    top = 1024 if dtype == F32 and way == "train" else 2048 if dtype == F32 else 4096 if way == "train" else 8192
    L = _log(rng, max(8, 64 // P), top // P)
    B = rng.choice([1, 1, 2])
    return {"op": op, "dir": way, "B": B, "S": L * P, "Hq": min(hq, 16 // B), "Hkv": hkv if hq <= 16 // B else 1, "d": d, "P": P,
            "causal": rng.choice([True, True, False]), "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _sections(case):
    """Pairs of each axis: even shares, what is left over to the first."""
    n, a = case["pairs"], case["axes"]
    return [n // a + n % a] + [n // a] * (a - 1)


_FREQ_BASE = 10000.0


def _pairs(case):
    """(axis of a pair, its frequency) for the pairs of a column group, on the host in 64 bits."""
    sec = _sections(case)
    axis = [a for a, n in enumerate(sec) for _ in range(n)]
    if case["freq"] == "global":  # one ladder of frequencies over all pairs, the axes take stretches of it
        freq = [_FREQ_BASE ** (-i / case["pairs"]) for i in range(case["pairs"])]
    else:  # a ladder of its own for each axis
        freq = [_FREQ_BASE ** (-j / n) for n in sec for j in range(n)]
    return axis, freq


def _lengths(case):
    """Cached tokens of each sequence: the whole cache, none, one, and spread in between."""
    T = case["T"]
    return [(T, 0, 1)[b] if b < 3 else int(T * ((b + 1) * 0.6180339887498949 % 1.0)) for b in range(case["B"])]


def prepare(case, seed):
    dev, t = "cuda", _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(t)

    s = {"case": dict(case)}
    if case["op"] == "rope":
        B, S, d = case["B"], case["S"], case["d"]
        if case["dir"] == "fwd":  # as the projections write them
            s["q"] = normal(B, S, case["Hq"], d).transpose(1, 2)
            s["k"] = normal(B, S, case["Hkv"], d).transpose(1, 2)
        else:  # as the attention's backward writes them
            s["q"] = normal(B, case["Hq"], S, d)
            s["k"] = normal(B, case["Hkv"], S, d)
        # text before, then frames of rows and columns; each sequence starts somewhere in a long context
        i = torch.arange(S, device=dev)
        w = max(1, math.isqrt(max(1, S // 16)))
        start = torch.randint(0, 1 << 20, (B, 1), generator=gen, device=dev)
        axes = [start + i // (w * w), start + i // w % w, start + i % w] if case["axes"] == 3 else [start + i // w, start + i % w]
        s["pos"] = torch.stack(axes if case["axes"] > 1 else [start + i])  # [axes, B, S]
        return s
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    # lam: exp(a.b) - exp(c.d) + 0.8 of small learned vectors lies around 0.8
    s["lam"] = (0.8 + 0.1 * torch.randn(Hq, generator=gen, device=dev)).to(t)
    if case["op"] == "diff":
        S = case["S"]
        s["q"], s["k"], s["v"] = normal(B, Hq, S, d), normal(B, Hkv, S, d), normal(B, Hkv, S, d)
        if case["dir"] == "train":
            s["g"] = normal(B, Hq, S, d)
        return s
    T = case["T"]
    s["q"], s["k"], s["v"] = normal(B, Hq, 1, d), normal(B, Hkv, T, d), normal(B, Hkv, T, d)
    order = torch.randperm(B, generator=gen, device=dev)
    s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
    return s


# ------------------------------------------------------------------ the framework's calls

_kept = {}  # what a user's program makes once for its sizes: plans, rotary tables, workspaces


def _once(key, make):
    if key not in _kept:
        _kept[key] = make()
    return _kept[key]


def _run_own(s):
    import tiled_distributed_attention_gb300 as mesh
    c = s["case"]
    if c["op"] == "rope":
        key = ("rope", c["d"], c["groups"], c["axes"], c["pairs"], c["style"], c["freq"])
        rope = _once(key, lambda: mesh.MeshRope(c["d"], _sections(c), base=_FREQ_BASE, groups=c["groups"], style=c["style"],
                                                freq=c["freq"]))
        if c["dir"] == "fwd":
            return mesh.mesh_rope(s["q"], s["k"], s["pos"], rope)
        dq, dk = (torch.empty_like(x.transpose(1, 2), memory_format=torch.contiguous_format).transpose(1, 2)
                  for x in (s["q"], s["k"]))
        return mesh.mesh_rope_backward(s["q"], s["k"], s["pos"], rope, dq_out=dq, dk_out=dk)
    status = _once("status", lambda: mesh.new_status())
    if c["op"] == "decode":
        key = ("decode", c["B"], c["T"], c["Hq"], c["Hkv"], c["d"])
        ws = _once(key, lambda: mesh.new_diff_decode_workspace(c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]))
        return mesh.mesh_diff_decode(s["q"], s["k"], s["v"], s["lens"], s["lam"], workspace=ws, status=status,
                                     check_status=False)
    plan = _once(("plan", c["S"], c["P"], c["causal"]), lambda: mesh.mesh_attn_plan_create(c["S"], c["P"], c["causal"]))
    key = ("diff", c["dir"], c["S"], c["P"], c["causal"], c["B"], c["Hq"], c["Hkv"], c["d"], c["dtype"])
    ws = _once(key, lambda: mesh.new_diff_workspace(plan, s["q"], s["k"], backward=c["dir"] == "train"))
    keep = dict(plan=plan, workspace=ws, status=status, check_status=False)
    if c["dir"] == "fwd":
        return mesh.mesh_diff_attention(s["q"], s["k"], s["v"], s["lam"], c["P"], c["causal"], **keep)
    O, O2, LSE = mesh.mesh_diff_attention(s["q"], s["k"], s["v"], s["lam"], c["P"], c["causal"], return_saved=True, **keep)
    grads = mesh.mesh_diff_attention_backward(s["q"], s["k"], s["v"], s["lam"], O, O2, LSE, s["g"], c["P"], c["causal"], **keep)
    return (O, LSE) + tuple(grads)


# ------------------------------------------------------------------ the plain forms

def _plain_rope(s):
    c = s["case"]
    axis, freq = _pairs(c)
    n, g, dh = c["pairs"], c["groups"], c["d"] // c["groups"]
    dev = s["q"].device
    # 64 bits: an angle of a far position keeps none of its digits after the point in 32
    ang = s["pos"].double()[torch.tensor(axis, device=dev)] * torch.tensor(freq, dtype=torch.float64, device=dev)[:, None, None]
    ang = ang.permute(1, 2, 0)[:, None, :, None, :]  # [B, 1, S, 1, n]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if c["dir"] == "bwd":
        sin = -sin

    def turn(x):
        y = x.float().reshape(x.shape[0], x.shape[1], x.shape[2], g, dh)
        rot, rest = y[..., : 2 * n], y[..., 2 * n:]
        if c["style"] == "half":
            a, b = rot[..., :n], rot[..., n:]
            rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([rot, rest], -1).reshape(x.shape).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _maps(q, k, scale, keep):
    """The two score maps [B, Hkv, g S, T] of q [B, Hq, S, d] and k [B, Hkv, T, d], masked, and their LSE and softmax."""
    B, Hq, S, d = q.shape
    Hkv, h = k.shape[1], d // 2
    rows = q.reshape(B, Hkv, Hq // Hkv * S, d)
    both = []
    for part in (slice(0, h), slice(h, d)):
        x = torch.matmul(rows[..., part], k[..., part].transpose(-1, -2)).mul_(scale)
        if keep is not None:
            x = x.view(B, Hkv, Hq // Hkv, S, -1).masked_fill_(~keep, float("-inf")).view(x.shape)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
        x = x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        both += [x.div_(torch.where(l == 0, torch.ones_like(l), l)), (m + torch.log(l)).view(B, Hq, S)]
    return both


def _plain_diff(s):
    c = s["case"]
    q, k, v, lam = (s[n].float() for n in ("q", "k", "v", "lam"))
    B, Hq, S, d = q.shape
    Hkv, T, h, t = k.shape[1], k.shape[2], d // 2, s["q"].dtype
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(h)
    keep = None
    if c["op"] == "decode":
        keep = (torch.arange(T, device=q.device) < s["lens"][:, None])[:, None, None, None, :]
    elif c["causal"]:
        keep = torch.ones(S, T, dtype=torch.bool, device=q.device).tril_()
    p1, l1, p2, l2 = _maps(q, k, scale, keep)
    lse = torch.stack([l1, l2], 2)  # [B, Hq, 2, S]
    w = lam.view(Hkv, g, 1).expand(Hkv, g, S).reshape(1, Hkv, g * S, 1)
    if c["op"] == "decode" or c["dir"] == "fwd":
        o = torch.matmul(p1.sub_(p2.mul_(w)), v).view(B, Hq, S, d)
        return o.to(t), lse
    go = s["g"].float().reshape(B, Hkv, g * S, d)
    o1, o2 = torch.matmul(p1, v), torch.matmul(p2, v)
    o = (o1 - w * o2).view(B, Hq, S, d)
    dv = torch.matmul((p1 - w * p2).transpose(-1, -2), go)
    dp = torch.matmul(go, v.transpose(-1, -2))
    d1, d2 = (go * o1).sum(-1, keepdim=True), (go * o2).sum(-1, keepdim=True)
    dlam = -d2.double().view(B, Hq, S).sum((0, 2)).float()  # a sum over every row of the batch
    ds1 = (dp - d1).mul_(p1).mul_(scale)
    ds2 = dp.sub_(d2).mul_(p2).mul_(-scale * w)
    rows = q.reshape(B, Hkv, g * S, d)
    dq = torch.cat([torch.matmul(ds1, k[..., :h]), torch.matmul(ds2, k[..., h:])], -1).view(q.shape)
    dk = torch.cat([torch.matmul(ds1.transpose(-1, -2), rows[..., :h]), torch.matmul(ds2.transpose(-1, -2), rows[..., h:])], -1)
    return o.to(t), lse, dq.to(t), dk.to(t), dv.to(t), dlam.to(t)


def run(state):
    if own:
        return _run_own(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_diff(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        n = B * case["S"] * (Hq + Hkv)
        return {"bytes": 2 * n * d * es + 8 * case["axes"] * B * case["S"], "flops": 6 * n * case["groups"] * case["pairs"]}
    if case["op"] == "decode":
        keys = sum(_lengths(case))
        return {"bytes": 2 * keys * Hkv * d * es + 2 * B * Hq * d * es + 8 * B * Hq + 4 * B, "flops": 6 * d * Hq * keys}
    S = case["S"]
    pairs = B * Hq * (S * (S + 1) // 2 if case["causal"] else S * S)
    q, kv = B * Hq * S * d * es, B * Hkv * S * d * es
    out = {"bytes": 2 * q + 2 * kv + 8 * B * Hq * S, "flops": 6 * d * pairs}
    if case["dir"] == "train":  # the gradient is read, and those of q, k and v are written
        out = {"bytes": out["bytes"] + 2 * q + 2 * kv, "flops": out["flops"] + 10 * d * pairs}
    return out


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_rope(s):
    c = s["case"]
    axis, freq = _pairs(c)
    dh, n = c["d"] // c["groups"], c["pairs"]
    sign = -1.0 if c["dir"] == "bwd" else 1.0
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for i in range(n):
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(s["pos"].shape[1:]),
                               sign * s["pos"][axis[i]].double() * freq[i])[:, None, :]
            for at in range(0, c["d"], dh):
                a, b = (at + i, at + n + i) if c["style"] == "half" else (at + 2 * i, at + 2 * i + 1)
                z = torch.complex(y[..., a], y[..., b]) * turn
                y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_head(q, k, v, lam, g, keep, scale):
    """One query head: q [S, d], k, v [T, d], keep [S, T] or None; with its gradients where g is given."""
    h = q.shape[-1] // 2
    probs, lses, outs = [], [], []
    for part in (slice(0, h), slice(h, 2 * h)):
        x = (q[:, part] * scale) @ k[:, part].T
        if keep is not None:
            x = torch.where(keep, x, torch.full((), -math.inf, dtype=x.dtype, device=x.device))
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
        probs.append(p)
        lses.append(lse)
        outs.append(p @ v)
    o = outs[0] - lam * outs[1]
    if g is None:
        return o, torch.stack(lses), None
    dq, dk, dlam = [], [], -(g * outs[1]).sum()
    dv = (probs[0] - lam * probs[1]).T @ g
    da = g @ v.T
    for m, part in enumerate((slice(0, h), slice(h, 2 * h))):
        w = 1.0 if m == 0 else -lam
        ds = w * probs[m] * (da - (g * outs[m]).sum(-1, keepdim=True))
        dq.append(scale * (ds @ k[:, part]))
        dk.append(scale * (ds.T @ q[:, part]))
    return o, torch.stack(lses), (torch.cat(dq, -1), torch.cat(dk, -1), dv, dlam)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if work(case)["flops"] > 6e12:  # 64-bit products of this size take too long
        return None
    q, k, v, lam = (s[n].double() for n in ("q", "k", "v", "lam"))
    B, Hq, S, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    train = case["op"] == "diff" and case["dir"] == "train"
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 2, S, dtype=torch.float64, device=q.device)
    dq, dk, dv, dlam = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(lam)
    for b in range(B):
        keep = None
        if case["op"] == "decode":
            keep = (torch.arange(T, device=q.device) < s["lens"][b])[None, :]
        elif case["causal"]:
            i = torch.arange(S, device=q.device)
            keep = i[None, :] <= i[:, None]
        for h in range(Hq):
            j = h * Hkv // Hq
            o[b, h], lse[b, h], got = _exact_head(q[b, h], k[b, j], v[b, j], lam[h], s["g"][b, h].double() if train else None,
                                                  keep, 1.0 / math.sqrt(d // 2))
            if train:
                dq[b, h] = got[0]
                dk[b, j] += got[1]
                dv[b, j] += got[2]
                dlam[h] += got[3]
    return (o, lse, dq, dk, dv, dlam) if train else (o, lse)
