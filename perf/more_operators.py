"""Measured cases of the paged cache's append, of attention over a paged cache, and of attention whose scores are capped, biased
by distance and masked by a range of keys a row: each operator in a plain form (elementary torch operations in 32 bits) and as a
user's program calls it, over the range of sizes, types and directions that it serves.

Operators (`op` of a case):
  append  keys and values of new tokens into their sequences' pages, queries and keys rotated on the way; q, k and v
          are slices of one projection [N, (Hq + 2 Hkv) d], the tokens of all sequences one after another
  paged   attention of each sequence's new tokens (one: a decoding step; many: a chunk of a prompt) over its pages, the new
          tokens' own keys among them; causal, with a cap, slopes or a window where the case has them
  range   attention of a dense batch where query i sees the keys [lo_i, hi_i): documents packed into one row, prefixes that see
          one another; with a cap and slopes where the case has them; `dir` "fwd", or "train" for a forward and a backward pass
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one decoding step of a served batch of 64
        {"name": "append_step_b64", "op": "append", "B": 64, "new": "one", "N": 64, "T": 8192, "page": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "groups": 1, "pairs": 64, "style": "half", "dtype": BF16},
        # eight prompts of ragged length at once
        {"name": "append_prompts_16k", "op": "append", "B": 8, "new": "ragged", "N": 16384, "T": 8192, "page": 64, "Hq": 32, "Hkv": 8,
         "d": 128, "groups": 1, "pairs": 64, "style": "half", "dtype": BF16},
        # one new token for each of 64 sequences, lengths from one to the table's end
        {"name": "step_b64_ragged", "op": "paged", "B": 64, "new": "one", "N": 64, "T": 8192, "page": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "cap": 0.0, "slopes": False, "window": 0, "dtype": BF16},
        # one new token of one sequence with a context of 128K
        {"name": "step_128k", "op": "paged", "B": 1, "new": "one", "N": 1, "T": 131072, "page": 64, "Hq": 16, "Hkv": 4, "d": 128,
         "cap": 0.0, "slopes": False, "window": 0, "dtype": BF16},
        # a chunk of a long prompt
        {"name": "chunk_1k_over_64k", "op": "paged", "B": 1, "new": "ragged", "N": 1024, "T": 65536, "page": 64, "Hq": 32, "Hkv": 8,
         "d": 128, "cap": 0.0, "slopes": False, "window": 0, "dtype": BF16},
        # a mixed batch: single tokens beside chunks of prompts, small pages, capped scores
        {"name": "mixed_b16_capped", "op": "paged", "B": 16, "new": "mixed", "N": 2048, "T": 4096, "page": 16, "Hq": 16, "Hkv": 4,
         "d": 128, "cap": 50.0, "slopes": False, "window": 0, "dtype": BF16},
        # a few short sequences in fp32, biased by distance, with a window
        {"name": "chunk_f32_window", "op": "paged", "B": 3, "new": "ragged", "N": 111, "T": 1000, "page": 32, "Hq": 8, "Hkv": 4, "d": 64,
         "cap": 0.0, "slopes": True, "window": 257, "dtype": F32},
        # documents packed into the 16K causal configuration
        {"name": "docs_16k", "op": "range", "dir": "fwd", "B": 1, "S": 16384, "Hq": 16, "Hkv": 16, "d": 128, "mask": "docs", "docs": 6,
         "cap": 0.0, "slopes": False, "dtype": BF16},
        # prefixes that see one another, ragged length, shared KV heads, capped scores
        {"name": "prefix_ragged_capped", "op": "range", "dir": "fwd", "B": 2, "S": 2500, "Hq": 8, "Hkv": 2, "d": 128, "mask": "prefix",
         "docs": 2, "cap": 50.0, "slopes": False, "dtype": BF16},
        # training on packed documents at 8K with shared KV heads, capped scores
        {"name": "docs_train_8k_capped", "op": "range", "dir": "train", "B": 1, "S": 8192, "Hq": 16, "Hkv": 4, "d": 128, "mask": "docs",
         "docs": 5, "cap": 30.0, "slopes": False, "dtype": BF16},
        # training of a small model whose scores are biased by distance
        {"name": "causal_train_slopes", "op": "range", "dir": "train", "B": 2, "S": 1000, "Hq": 4, "Hkv": 4, "d": 64, "mask": "docs",
         "docs": 1, "cap": 0.0, "slopes": True, "dtype": BF16},
        # training in fp32: documents, cap and slopes
        {"name": "docs_train_f32", "op": "range", "dir": "train", "B": 1, "S": 777, "Hq": 4, "Hkv": 2, "d": 64, "mask": "docs", "docs": 3,
         "cap": 20.0, "slopes": True, "dtype": F32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "range", "range"])
    d = rng.choice([64, 128])
    dtype = rng.choice([BF16, BF16, F32])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = min(32, hkv * rng.choice([1, 2, 3, 4, 5, 8]) // hkv * hkv)
    if hq % hkv:
        hq = hkv
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "append":
        new = rng.choice(["one", "ragged", "mixed"])
        B = _log(rng, 1, 64)
        N = B if new == "one" else max(B, _log(rng, 1, 12288 if dtype == BF16 else 6144))
        groups = rng.choice([1, 1, 2])
        half = d // groups // 2
        return {"op": op, "B": B, "new": new, "N": N, "T": max(N, _log(rng, 64, max(64, 131072 // B))), "page": page, "Hq": hq, "Hkv": hkv, "d": d,
                "groups": groups, "pairs": rng.choice([half, half, half - 4, half - 3]), "style": rng.choice(["half", "adjacent"]),
                "dtype": dtype}
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    slopes = rng.choice([False, False, True])
    if op == "paged":
        new = rng.choice(["one", "one", "ragged", "mixed"])
        T = _log(rng, 1, 16384 if dtype == BF16 else 4096)
        B = min(64, _log(rng, 1, max(1, 131072 // T)))
        top = min(T * B, max(B, (1 << 24) // (T * max(1, hq // 8)))) if dtype == BF16 else min(T * B, max(B, (1 << 21) // T))
        N = B if new == "one" else max(B, _log(rng, B, max(B + 1, min(4096, top))))
        N = min(N, B * T)
        return {"op": op, "B": B, "new": "one" if N == B else new, "N": N, "T": T, "page": page, "Hq": hq, "Hkv": hkv, "d": d, "cap": cap,
                "slopes": slopes, "window": rng.choice([0, 0, 1, _log(rng, 2, 2048)]), "dtype": dtype}
    way = rng.choice(["fwd", "train"])
    top = 1024 if dtype == F32 and way == "train" else 2048 if dtype == F32 else 4096 if way == "train" else 8192
    S = _log(rng, 16, top)
    B = rng.choice([1, 1, 2, 3])
    return {"op": op, "dir": way, "B": B, "S": S, "Hq": hq if hq * B <= 16 else hkv, "Hkv": hkv, "d": d, "mask": rng.choice(["docs", "docs", "prefix", "both"]),
            "docs": min(rng.choice([1, 2, 5, 17]), S // 8), "cap": cap, "slopes": slopes, "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _new_tokens(case):
    """New tokens of each sequence: one each, uneven shares, or a few chunks among single tokens."""
    B, N, T = case["B"], case["N"], case["T"]
    if case["new"] == "one":
        return [1] * B
    some = list(range(B)) if case["new"] == "ragged" else list(range(0, B, 4))
    n = [1] * B
    left = N - B
    weight = [1 + (i * 7 + 3) % 5 for i in range(len(some))]
    for i, b in enumerate(some):
        n[b] += left * weight[i] // sum(weight)
    n[some[-1]] += N - sum(n)
    over = 0  # no more than the table holds
    for b in range(B):
        over += max(0, n[b] - T)
        n[b] = min(n[b], T)
    for b in range(B):
        more = min(over, T - n[b])
        n[b] += more
        over -= more
    return n


def _lengths(case, n):
    """Cached tokens of each sequence after the append: a full table, nothing before, and spread in between."""
    T = case["T"]
    out = []
    for b, m in enumerate(n):
        f = 1.0 if b == 0 else 0.0 if b == 1 else (b + 1) * 0.6180339887498949 % 1.0
        out.append(m + int((T - m) * f))
    return out


def _ranges(case):
    """lo and hi of each query, on the host: documents of uneven length, causal within; "prefix": the first third of each sees
    itself both ways; "both": everything within a document, and the last tenth of the batch's rows is padding."""
    S, B = case["S"], case["B"]
    lo, hi = torch.zeros(B, S, dtype=torch.int32), torch.zeros(B, S, dtype=torch.int32)
    for b in range(B):
        weight = [2 + (i * 5 + b * 3) % 7 for i in range(case["docs"])]
        edge = [S * sum(weight[:i]) // sum(weight) for i in range(case["docs"] + 1)]
        for x, y in zip(edge, edge[1:]):
            i = torch.arange(x, y, dtype=torch.int32)
            lo[b, x:y] = x
            hi[b, x:y] = y if case["mask"] == "both" else torch.clamp(i + 1, min=x + (y - x) // 3 if case["mask"] == "prefix" else 0)
        if case["mask"] == "both":  # padding: rows that see nothing and keys that nobody sees
            end = S - S // 10
            lo[b, end:] = hi[b, end:] = 0
            hi[b].clamp_(max=end)
    return lo, hi


def prepare(case, seed):
    dev, t = "cuda", _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(t)

    s = {"case": dict(case)}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case.get("slopes"):
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev)
    if case["op"] == "range":
        B, S = case["B"], case["S"]
        s["q"], s["k"], s["v"] = normal(B, Hq, S, d) * 2, normal(B, Hkv, S, d), normal(B, Hkv, S, d)
        if case["dir"] == "train":
            s["g"] = normal(B, Hq, S, d)
        lo, hi = _ranges(case)
        s["lo"], s["hi"] = lo.to(dev), hi.to(dev)
        return s
    B, N, T, page = case["B"], case["N"], case["T"], case["page"]
    n = _new_tokens(case)
    lens = _lengths(case, n)
    order = torch.randperm(B, generator=gen, device=dev).tolist()
    n, lens = [n[i] for i in order], [lens[i] for i in order]
    off = [0]
    for m in n:
        off.append(off[-1] + m)
    s["max_new"] = max(n)
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # pages in no order, a few of other sequences among them
    pages = [(x + page - 1) // page for x in lens]
    total = sum(pages) + 5
    perm = torch.randperm(total, generator=gen, device=dev, dtype=torch.int32)
    table = torch.zeros(B, (T + page - 1) // page, dtype=torch.int32, device=dev)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = perm[at:at + m]
        at += m
    s["table"] = table
    s["k_pages"], s["v_pages"] = normal(total, Hkv, page, d), normal(total, Hkv, page, d)
    if case["op"] == "append":
        qkv = normal(N, (Hq + 2 * Hkv) * d).view(N, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"] = normal(N, Hq, d) * 2
    return s


# ------------------------------------------------------------------ the framework's calls

_BASE = 10000.0
_kept = {}  # what a user's program makes once for its sizes: rotations, workspaces, the status block


def _once(key, make):
    if key not in _kept:
        _kept[key] = make()
    return _kept[key]


def _run_own(s):
    import tiled_distributed_attention_gb300 as mesh
    c = s["case"]
    status = _once("status", lambda: mesh.new_status())
    keep = dict(status=status, check_status=False)
    if c["op"] == "append":
        rope = _once((c["d"], c["groups"], c["pairs"], c["style"]),
                     lambda: mesh.MeshRope(c["d"], [c["pairs"]], base=_BASE, groups=c["groups"], style=c["style"]))
        q = mesh.mesh_paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["offsets"], s["lens"], rope=rope,
                                   **keep)
        return q, s["k_pages"], s["v_pages"]
    more = dict(cap=c["cap"], slopes=s.get("slopes"), **keep)
    if c["op"] == "paged":
        ws = _once(("paged", c["B"], c["N"], s["max_new"], c["Hq"], c["Hkv"], c["d"], c["dtype"]),
                   lambda: mesh.new_paged_workspace(s["q"], s["k_pages"], s["table"], s["max_new"]))
        return mesh.mesh_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["offsets"], s["lens"], s["max_new"],
                                         window=c["window"], workspace=ws, **more)
    ws = _once(("range", c["dir"], c["B"], c["S"], c["Hq"], c["Hkv"], c["d"], c["dtype"]),
               lambda: mesh.new_range_workspace(s["q"], s["k"], backward=c["dir"] == "train"))
    o, lse = mesh.mesh_range_attention(s["q"], s["k"], s["v"], s["lo"], s["hi"], workspace=ws, **more)
    if c["dir"] == "fwd":
        return o, lse
    return (o, lse) + tuple(mesh.mesh_range_attention_backward(s["q"], s["k"], s["v"], s["lo"], s["hi"], o, lse, s["g"], workspace=ws,
                                                               **more))


# ------------------------------------------------------------------ the plain forms

def _token_places(s):
    """Sequence of each new token, its number within the call, its place in the sequence."""
    off = s["offsets"].long()
    i = torch.arange(s["case"]["N"], device=off.device)
    b = torch.searchsorted(off[1:].contiguous(), i, right=True)
    t = i - off[b]
    return b, t, s["lens"].long()[b] - (off[b + 1] - off[b]) + t


def _plain_append(s):
    c = s["case"]
    b, _, place = _token_places(s)
    n, g, dh = c["pairs"], c["groups"], c["d"] // c["groups"]
    # 64 bits: an angle of a far position keeps none of its digits after the point in 32
    freq = torch.tensor([_BASE ** (-i / n) for i in range(n)], dtype=torch.float64, device=place.device)
    ang = (place.double()[:, None] * freq)[:, None, None, :]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def turn(x):
        y = x.float().reshape(x.shape[0], x.shape[1], g, dh)
        rot, rest = y[..., : 2 * n], y[..., 2 * n:]
        if c["style"] == "half":
            u, w = rot[..., :n], rot[..., n:]
            rot = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
        else:
            u, w = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
        return torch.cat([rot, rest], -1).reshape(x.shape).to(x.dtype)

    at, row = s["table"].long()[b, place // c["page"]], place % c["page"]
    s["k_pages"][at, :, row] = turn(s["k"])
    s["v_pages"][at, :, row] = s["v"]
    return turn(s["q"]), s["k_pages"], s["v_pages"]


def _softmax(x, keep):
    x = x.masked_fill_(~keep, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    return x.div_(torch.where(l == 0, torch.ones_like(l), l)), (m + torch.log(l)).squeeze(-1)


def _plain_paged(s):
    c = s["case"]
    B, Hkv, d, g, m = c["B"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"], s["max_new"]
    t = s["q"].dtype
    off, lens = s["offsets"].long(), s["lens"].long()
    n = off[1:] - off[:-1]
    j = torch.arange(m, device=off.device)
    which = (off[:-1, None] + j).clamp_(max=c["N"] - 1)
    q = s["q"].float()[which].view(B, m, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * m, d)
    k, v = (s[x].float()[s["table"].long()].transpose(1, 2).reshape(B, Hkv, -1, d) for x in ("k_pages", "v_pages"))
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, g, m, -1)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    place = (lens - n)[:, None] + j  # [B, m]
    far = place[:, :, None] - torch.arange(k.shape[2], device=off.device)  # [B, m, T]
    if c["slopes"]:
        x = x.sub_(s["slopes"].view(Hkv, g, 1, 1) * far[:, None, None].abs().float())
    keep = (far >= 0) & (j < n[:, None])[:, :, None]
    if c["window"]:
        keep &= far < c["window"]
    p, lse = _softmax(x, keep[:, None, None])
    o = torch.matmul(p.view(B, Hkv, g * m, -1), v).view(B, Hkv, g, m, d)
    b, at, _ = _token_places(s)
    return o.permute(0, 3, 1, 2, 4)[b, at].reshape(c["N"], c["Hq"], d).to(t), lse.permute(0, 3, 1, 2)[b, at].reshape(c["N"], c["Hq"])


def _plain_range(s):
    c = s["case"]
    B, S, Hq, Hkv, d = c["B"], c["S"], c["Hq"], c["Hkv"], c["d"]
    g, t, scale = Hq // Hkv, s["q"].dtype, 1.0 / math.sqrt(d)
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    rows = q.view(B, Hkv, g * S, d)
    i = torch.arange(S, device=q.device)
    keep = ((i >= s["lo"][:, :, None]) & (i < s["hi"][:, :, None]))[:, None, None]  # [B, 1, 1, S, S]
    x = torch.matmul(rows, k.transpose(-1, -2)).mul_(scale).view(B, Hkv, g, S, S)
    th = None
    if c["cap"]:
        th = x.div_(c["cap"]).tanh_()
        x = th * c["cap"]
    if c["slopes"]:
        x = x - s["slopes"].view(Hkv, g, 1, 1) * (i[:, None] - i).abs().float()
    p, lse = _softmax(x, keep)
    p = p.view(B, Hkv, g * S, S)
    o = torch.matmul(p, v)
    out = (o.view(B, Hq, S, d).to(t), lse.view(B, Hq, S))
    if c["dir"] == "fwd":
        return out
    go = s["g"].float().view(B, Hkv, g * S, d)
    dv = torch.matmul(p.transpose(-1, -2), go)
    ds = torch.matmul(go, v.transpose(-1, -2)).sub_((go * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    if th is not None:
        ds = ds.mul_(1 - th.view(B, Hkv, g * S, S).square_())
    dq = torch.matmul(ds, k).view(B, Hq, S, d)
    dk = torch.matmul(ds.transpose(-1, -2), rows)
    return out + (dq.to(t), dk.to(t), dv.to(t))


def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "paged": _plain_paged, "range": _plain_range}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "range":
        lo, hi = _ranges(case)
        S = case["S"]
        pairs = Hq * int((hi.long() - lo.long()).clamp_(min=0).sum())
        q, kv = B * Hq * S * d * es, B * Hkv * S * d * es
        out = {"bytes": 2 * q + 2 * kv + 4 * B * Hq * S + 8 * B * S, "flops": 4 * d * pairs}
        if case["dir"] == "train":  # the gradient is read, and those of q, k and v are written
            out = {"bytes": out["bytes"] + 2 * q + 2 * kv, "flops": out["flops"] + 10 * d * pairs}
        return out
    n = _new_tokens(case)
    lens = _lengths(case, n)
    N, page = case["N"], case["page"]
    if case["op"] == "append":
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * d * es + 4 * sum((m + page - 1) // page for m in n) + 8 * B,
                "flops": 6 * N * (Hq + Hkv) * case["groups"] * case["pairs"]}
    w = case["window"] or case["T"]
    keys = sum(min(x, m - 1 + w) for x, m in zip(lens, n))  # that some new token sees
    pairs = 0
    for x, m in zip(lens, n):  # token t of m sees min(x - m + t + 1, w) keys
        first = x - m + 1
        short = max(0, min(m, w - first))  # tokens that see less than the window
        pairs += short * first + short * (short - 1) // 2 + (m - short) * min(w, x)
    return {"bytes": 2 * keys * Hkv * d * es + 2 * N * Hq * d * es + 4 * N * Hq + 4 * (keys // page + 2 * B), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_append(s):
    c = s["case"]
    b, _, place = _token_places(s)
    dh, n = c["d"] // c["groups"], c["pairs"]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for i in range(n):
            turn = torch.polar(torch.ones_like(place, dtype=torch.float64), place.double() * _BASE ** (-i / n))[:, None]
            for at in range(0, c["d"], dh):
                u, w = (at + i, at + n + i) if c["style"] == "half" else (at + 2 * i, at + 2 * i + 1)
                z = torch.complex(y[..., u], y[..., w]) * turn
                y[..., u], y[..., w] = z.real, z.imag
        out.append(y)
    at = s["table"].long()[b, place // c["page"]] * c["page"] + place % c["page"]
    for pages, x in ((s["k_pages"], out[1]), (s["v_pages"], s["v"])):
        flat = pages.double().transpose(1, 2).reshape(-1, c["Hkv"], c["d"]).clone()  # [tokens of all pages, Hkv, d]
        flat[at] = x.double()
        out.append(flat.view(-1, c["page"], c["Hkv"], c["d"]).transpose(1, 2).contiguous())
    return out[0], out[2], out[3]


def _exact_scores(q, k, cap, slope, far, keep):
    """Masked scores of one head, q [m, d], k [T, d], far and keep [m, T], and the slope of the cap."""
    x = (q / math.sqrt(q.shape[-1])) @ k.T
    turn = None
    if cap:
        e = torch.exp(-2.0 * (x / cap).abs())
        th = torch.sign(x) * (1.0 - e) / (1.0 + e)
        x, turn = cap * th, 1.0 - th * th
    if slope is not None:
        x = x - slope * far.abs().double()
    return torch.where(keep, x, torch.full((), -math.inf, dtype=x.dtype, device=x.device)), turn


def _exact_probs(x):
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]), lse


def _exact_paged(s):
    c = s["case"]
    q, slopes, g = s["q"].double(), s.get("slopes"), c["Hq"] // c["Hkv"]
    o, lse = torch.empty_like(q), torch.empty(c["N"], c["Hq"], dtype=torch.float64, device=q.device)
    off, lens, page = s["offsets"].tolist(), s["lens"].tolist(), c["page"]
    for b in range(c["B"]):
        m, T = off[b + 1] - off[b], lens[b]
        if m == 0:
            continue
        at = s["table"][b, : (T + page - 1) // page].long()
        k, v = (s[x][at].transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[:T].double() for x in ("k_pages", "v_pages"))
        far = torch.arange(T - m, T, device=q.device)[:, None] - torch.arange(T, device=q.device)
        keep = far >= 0
        if c["window"]:
            keep &= far < c["window"]
        for h in range(c["Hq"]):
            x, _ = _exact_scores(q[off[b]:off[b + 1], h], k[:, h // g], c["cap"], None if slopes is None else slopes[h].double(), far,
                                 keep)
            p, lse[off[b]:off[b + 1], h] = _exact_probs(x)
            o[off[b]:off[b + 1], h] = p @ v[:, h // g]
    return o, lse


def _exact_range(s):
    c = s["case"]
    q, k, v, slopes = s["q"].double(), s["k"].double(), s["v"].double(), s.get("slopes")
    B, Hq, S, d = q.shape
    g, train, scale = Hq // c["Hkv"], c["dir"] == "train", 1.0 / math.sqrt(d)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, S, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    i = torch.arange(S, device=q.device)
    far = i[:, None] - i
    for b in range(B):
        keep = (i >= s["lo"][b, :, None]) & (i < s["hi"][b, :, None])
        for h in range(Hq):
            j = h // g
            x, turn = _exact_scores(q[b, h], k[b, j], c["cap"], None if slopes is None else slopes[h].double(), far, keep)
            p, lse[b, h] = _exact_probs(x)
            o[b, h] = p @ v[b, j]
            if train:
                go = s["g"][b, h].double()
                ds = p * (go @ v[b, j].T - (go * o[b, h]).sum(-1, keepdim=True))
                if turn is not None:
                    ds = ds * turn
                dq[b, h] = scale * (ds @ k[b, j])
                dk[b, j] += scale * (ds.T @ q[b, h])
                dv[b, j] += p.T @ go
    return (o, lse, dq, dk, dv) if train else (o, lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "paged":
        n = _new_tokens(case)
        if sum(4.0 * m * x for m, x in zip(n, _lengths(case, n))) * case["Hq"] * case["d"] > 6e12:  # too long in 64 bits
            return None
        return _exact_paged(s)
    if 4.0 * case["B"] * case["Hq"] * case["S"] ** 2 * case["d"] * (3.5 if case["dir"] == "train" else 1) > 6e12:
        return None
    return _exact_range(s)
