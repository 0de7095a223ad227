"""The paged cache: append with rotation, attention of new tokens over pages, and both as a serving loop uses them, against the fp64
oracles.

Bounds as in test_gpu_range.py; with few rows P goes in two bf16 pieces (2^-17), so O has u |O| + (2^-12 + n 2^-23) mag.  Rotations are
off by u |x| for their rounding and 2^-20 (|x| + |y|) for sines, cosines and the two products in fp32.
"""
import math

import pytest
import torch

from oracle import range_attention as OR
from tests.test_gpu_range import DT, slopes_of, within

pytestmark = pytest.mark.gpu


def cache(new, lens, page, Hq, Hkv, d, dtype, seed, spare=3, layout="pages", fill=None):
    """A batch over a paged cache on the host: q, k, v of the new tokens, full pages, table, offsets, lens."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])  # noqa: E731
    N = sum(new)
    q, k, v = n(N, Hq, d), n(N, Hkv, d), n(N, Hkv, d)
    need = [(x + page - 1) // page for x in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), total + 100, dtype=torch.int32)  # entries behind a sequence's pages: nonsense
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    kp, vp = n(total, Hkv, page, d), n(total, Hkv, page, d)
    off = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    return q, k, v, kp, vp, table, off, torch.tensor(lens, dtype=torch.int32)


def place_of(new, lens):
    return [(b, lens[b] - new[b] + t) for b in range(len(new)) for t in range(new[b])]


def turned(x, pos, rope):
    """x [N, H, d] turned by rope at the places pos [axes][N], and the magnitudes of the sums, in fp64."""
    y, mag = x.double().clone(), x.double().abs()
    dh, n = rope.d // rope.groups, rope.n_pairs
    for i in range(n):
        phi = torch.tensor([p * rope.freq[i] for p in pos[rope.axis[i]]], dtype=torch.float64)[:, None]
        c, s = torch.cos(phi), torch.sin(phi)
        for at in range(0, rope.d, dh):
            a, b = (at + i, at + n + i) if rope.style == "half" else (at + 2 * i, at + 2 * i + 1)
            u, w = x[..., a].double(), x[..., b].double()
            y[..., a], y[..., b] = u * c - w * s, w * c + u * s
            mag[..., a] = mag[..., b] = u.abs() + w.abs()
    return y, mag


# new, lens, page, Hq, Hkv, d, rope (pairs, groups, style) or None
APPENDS = [
    ([1], [1], 16, 1, 1, 64, (32, 1, "half")),
    ([1, 1, 1], [1, 17, 40], 16, 8, 2, 128, (64, 1, "half")),
    ([5, 0, 1, 33], [5, 9, 100, 64], 16, 4, 2, 128, (64, 1, "adjacent")),
    ([40, 7], [1000, 7], 48, 3, 1, 64, (13, 2, "half")),
    ([300], [300], 128, 2, 2, 128, (28, 2, "adjacent")),
    ([17, 3], [20, 3], 5, 2, 1, 64, (29, 1, "half")),
    ([9, 9, 9], [30, 9, 12], 32, 4, 4, 96, None),
    ([1] * 70, list(range(1, 71)), 16, 4, 1, 64, (32, 1, "half")),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{len(c[0])}x{c[2:]}")
def test_append(lib, case, dtype):
    new, lens, page, Hq, Hkv, d, r = case
    q, k, v, kp, vp, table, off, ln = cache(new, lens, page, Hq, Hkv, d, dtype, 40)
    rope = None if r is None else lib.MeshRope(d, (r[0],), groups=r[1], style=r[2])
    qkv = torch.cat([q, k, v], 1).cuda()  # slices of one projection
    kd, vd = kp.cuda(), vp.cuda()
    out = lib.mesh_paged_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kd, vd, table.cuda(), off.cuda(), ln.cuda(), rope=rope)
    where = place_of(new, lens)
    pos = [[p for _, p in where]]
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    if rope:
        qr, qm = turned(q, pos, rope)
        kr, km = turned(k, pos, rope)
        within(out, qr, u * qr.abs() + 2.0 ** -20 * qm + 1e-30, "q")
    else:
        assert torch.equal(out.cpu(), q)
    got_k, got_v = kd.cpu(), vd.cpu()
    for i, (b, p) in enumerate(where):
        at = int(table[b, p // page])
        assert torch.equal(got_v[at, :, p % page], v[i])
        if rope:
            within(got_k[at, :, p % page], kr[i], u * kr[i].abs() + 2.0 ** -20 * km[i] + 1e-30, "k")
        else:
            assert torch.equal(got_k[at, :, p % page], k[i])
        got_k[at, :, p % page], got_v[at, :, p % page] = kp[at, :, p % page], vp[at, :, p % page]
    assert torch.equal(got_k, kp) and torch.equal(got_v, vp)  # nothing else was written


def test_append_with_positions_views_and_no_q(lib):
    new, lens = [4, 6], [9, 6]
    q, k, v, kp, vp, table, off, ln = cache(new, lens, 16, 4, 2, 128, "bf16", 41)
    rope = lib.MeshRope(128, (20, 12, 8))
    pos = torch.randint(-1000, 1 << 20, (3, 10), generator=torch.Generator().manual_seed(3))
    tok = lambda t: t.cuda().transpose(1, 2).contiguous().transpose(1, 2)  # [n_pages, page, Hkv, d] in memory  # noqa: E731
    kd, vd = tok(kp), tok(vp)
    qo = torch.zeros(10, 6, 128, dtype=torch.bfloat16, device="cuda")[:, 1:5]
    got = lib.mesh_paged_append(q.cuda(), k.cuda(), v.cuda(), kd, vd, table.cuda(), off.cuda(), ln.cuda(), rope=rope, positions=pos.cuda(),
                                q_out=qo)
    assert got.data_ptr() == qo.data_ptr()
    qr, qm = turned(q, pos.tolist(), rope)
    kr, km = turned(k, pos.tolist(), rope)
    within(qo, qr, 2.0 ** -8 * qr.abs() + 2.0 ** -20 * qm + 1e-30, "q")
    ke, ve = tok(kp), tok(vp)
    assert lib.mesh_paged_append(None, k.cuda(), v.cuda(), ke, ve, table.cuda(), off.cuda(), ln.cuda(), rope=rope,
                                 positions=pos.cuda().int()) is None
    assert torch.equal(kd, ke) and torch.equal(vd, ve)
    for i, (b, p) in enumerate(place_of(new, lens)):
        at = int(table[b, p // 16])
        within(kd[at, :, p % 16], kr[i], 2.0 ** -8 * kr[i].abs() + 2.0 ** -20 * km[i] + 1e-30, "k")
        assert torch.equal(vd[at, :, p % 16].cpu(), v[i])
    # in place, and the same by mesh_rope on dense heads
    qi = q.cuda()
    lib.mesh_paged_append(qi, k.cuda(), v.cuda(), ke, ve, table.cuda(), off.cuda(), ln.cuda(), rope=rope, positions=pos.cuda(), q_out=qi)
    dense, _ = lib.mesh_rope(q.cuda().transpose(0, 1)[None], None, pos.cuda(), rope)
    assert torch.equal(qi, qo) and torch.equal(dense[0].transpose(0, 1), qo)


def test_append_leaves_out_what_does_not_exist(lib):
    """A page or place that does not exist is recorded; the other tokens are written, rows behind the last sequence are not."""
    new, lens = [2, 2, 2], [20, 20, 20]
    q, k, v, kp, vp, table, off, ln = cache(new, lens, 16, 2, 1, 64, "bf16", 42)
    for spoil, bad_b in (("page", 1), ("negative", 1), ("long", 2), ("short", 0)):
        t, l = table.clone(), ln.clone()
        if spoil == "page":
            t[1, 1] = kp.shape[0]
        elif spoil == "negative":
            t[1, 1] = -1
        elif spoil == "long":
            l[2] = 16 * t.shape[1] + 2
        else:
            l[0] = 0
        kd, vd, st = kp.cuda(), vp.cuda(), lib.new_status()
        qo = torch.full((8, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        pad = lambda x: torch.cat([x, x[:2]]).cuda()  # two rows of no sequence  # noqa: E731
        lib.mesh_paged_append(pad(q), pad(k), pad(v), kd, vd, t.cuda(), off.cuda(), l.cuda(), q_out=qo, status=st, check_status=False)
        assert lib.mesh_attn_read_status(st) == 6 and st.tolist()[2] == bad_b
        for i, (b, p) in enumerate(place_of(new, lens)):
            assert torch.equal(qo[i].cpu(), q[i]) == (b != bad_b)
            if b != bad_b:
                assert torch.equal(kd[int(table[b, p // 16]), :, p % 16].cpu(), k[i])
        assert (qo[6:] == 7).all()
    with pytest.raises(lib.MeshAttnError):
        lib.mesh_paged_append(q.cuda(), k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), t.cuda(), off.cuda(), l.cuda())


# new, lens, page, Hq, Hkv, d, cap, slopes, window
ATTENDS = [
    ([1], [1], 16, 1, 1, 128, 0.0, False, 0),
    ([1, 1, 1, 1], [1, 16, 129, 500], 16, 8, 2, 128, 0.0, False, 0),
    ([1] * 9, [3, 700, 1, 128, 127, 256, 40, 41, 42], 64, 4, 4, 64, 0.0, True, 0),
    ([1, 1], [300, 1100], 48, 16, 1, 128, 20.0, False, 100),
    ([1, 1], [300, 70], 32, 40, 1, 64, 0.0, False, 0),
    ([3, 1, 0, 4], [3, 260, 10, 400], 16, 4, 1, 128, 0.0, True, 37),
    ([2, 5], [90, 5], 16, 6, 2, 64, 1.0, False, 1),
    ([40], [40], 16, 4, 1, 128, 0.0, False, 0),
    ([130, 1, 7], [130, 400, 77], 64, 4, 4, 64, 0.0, False, 0),
    ([300, 1], [900, 130], 48, 8, 2, 128, 30.0, False, 0),
    ([77, 20, 0, 129], [600, 20, 5, 129], 32, 6, 2, 128, 0.0, True, 0),
    ([200, 65], [700, 300], 128, 3, 1, 64, 2.0, True, 150),
    ([33, 31], [2000, 31], 256, 10, 2, 128, 0.0, False, 90),
    ([64], [3000], 16, 2, 1, 128, 0.0, False, 0),
    ([20, 1], [25, 600], 16, 24, 1, 64, 0.0, False, 0),
    ([9], [50], 16, 130, 1, 64, 0.0, False, 0),
]


def check(O, L, ref, dtype, few):
    Or, Lr, mag = ref
    n = 4096
    u = 2.0 ** -8
    if dtype == "bf16":
        within(O, Or, u * Or.abs() + ((0 if few else u) + 2.0 ** -12 + n * 2.0 ** -23) * mag + 1e-6, "O")
        within(L, Lr, torch.full_like(Lr, 1e-3), "LSE")
    else:
        within(O, Or, torch.full_like(Or, 1e-4), "O")
        within(L, Lr, torch.full_like(Lr, 1e-4), "LSE")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: f"{c[0][:4]}x{c[2:]}")
def test_attention(lib, case, dtype):
    new, lens, page, Hq, Hkv, d, cap, steep, window = case
    q, _, _, kp, vp, table, off, ln = cache(new, lens, page, Hq, Hkv, d, dtype, 43)
    sl = slopes_of(Hq, steep)
    ref = OR.paged(q, kp, vp, table, off, ln, cap=cap, slopes=sl, window=window)
    # what lies behind a sequence's last token, in its last page and in pages of nobody, is NaN
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for b, x in enumerate(lens):
        for i in range(x):
            used[int(table[b, i // page]), i % page] = True
    for p in (kp, vp):
        p.transpose(1, 2)[~used] = math.nan
    few = max(new) * (Hq // Hkv) <= 16
    dev = [t.cuda() for t in (q, kp, vp, table, off, ln)]
    kw = dict(cap=cap, slopes=None if sl is None else sl.cuda(), window=window)
    O, L = lib.mesh_paged_attention(*dev, max(new), **kw)
    check(O, L, ref, dtype, few)
    # pages with the tokens outside, q a slice of something wider, and a bound of new tokens that picks another kernel
    wide = torch.zeros(q.shape[0], Hq + 2, d, dtype=q.dtype, device="cuda")
    wide[:, 1:1 + Hq] = dev[0]
    outside = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in dev[1:3]]
    O2, L2 = lib.mesh_paged_attention(wide[:, 1:1 + Hq], *outside, *dev[3:], max(new) + 40, **kw)
    check(O2, L2, ref, dtype, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, lens, window", [([1, 1], [900, 131], 100), ([2, 40], [300, 500], 7), ([150], [1000], 260)], ids=str)
def test_pages_before_a_window_need_not_exist(lib, dtype, new, lens, window):
    """A sliding window's old pages have been given away: no entries in the table, other sequences' tokens and NaN in them."""
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 1, 64, dtype, 54)
    ref = OR.paged(q, kp, vp, table, off, ln, window=window)
    for b, x in enumerate(lens):
        gone = max(0, x - new[b] + 1 - window) // 16
        for i in range(gone):
            kp[int(table[b, i])] = math.nan
            vp[int(table[b, i])] = math.nan
            table[b, i] = -1
    for bound in (max(new), max(new) + 60):
        O, L = lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), bound, window=window)
        check(O, L, ref, dtype, False)


def test_offsets_beyond_32_bits(lib):
    """Pages that begin beyond 2^31 elements of the pool, by append and by every attention kernel."""
    n, page, Hkv, d = 1_100_000, 16, 2, 64  # 2.25e9 elements a pool
    for dtype in (torch.bfloat16, torch.float32):
        kp, vp = (torch.empty(n, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
        assert kp.numel() > 1 << 31
        new, lens = [33, 1], [50, 70]
        q, k, v, ks, vs, table, off, ln = cache(new, lens, page, 8, Hkv, d, "bf16" if dtype == torch.bfloat16 else "f32", 55)
        far = torch.arange(n - ks.shape[0], n)
        kp[far.cuda()], vp[far.cuda()] = ks.cuda(), vs.cuda()
        low = table.clone()
        table = torch.where(table < ks.shape[0], table + (n - ks.shape[0]), table)
        dev = [t.cuda() for t in (q, k, v)]
        lib.mesh_paged_append(*dev, kp, vp, table.cuda(), off.cuda(), ln.cuda())
        for i, (b, p) in enumerate(place_of(new, lens)):
            ks[int(low[b, p // page]), :, p % page], vs[int(low[b, p // page]), :, p % page] = k[i], v[i]
        assert torch.equal(kp[far.cuda()].cpu(), ks) and torch.equal(vp[far.cuda()].cpu(), vs)
        name = "bf16" if dtype == torch.bfloat16 else "f32"
        for rows, o, l, t in ((slice(0, 34), off, ln, table), (slice(33, 34), torch.tensor([0, 1], dtype=torch.int32), ln[1:], table[1:])):
            ref = OR.paged(q[rows], ks, vs, low[1:] if rows.start else low, o, l)
            O, L = lib.mesh_paged_attention(dev[0][rows], kp, vp, t.cuda(), o.cuda(), l.cuda(), rows.stop - rows.start)
            check(O, L, ref, name, False)
        del kp, vp


def test_sequences_that_share_pages(lib):
    """A common prefix in pages of several sequences, as its owner wrote it."""
    new, lens = [1, 20, 1], [70, 70, 40]
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 2, 64, "bf16", 56)
    table[1, :2] = table[0, :2]
    table[2, :2] = table[0, :2]
    ref = OR.paged(q, kp, vp, table, off, ln)
    O, L = lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), 20)
    check(O, L, ref, "bf16", False)


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("new, lens, Hq, Hkv", [
    ([70, 1, 33], [5000, 3000, 40], 4, 1),       # few units over a long cache: all but the short one in parts
    ([300], [9000], 2, 1),                       # one sequence, groups of nearly one length
    ([40, 1, 1, 25, 200], [6000, 1, 2500, 25, 1500], 12, 4),  # 3 heads a KV head: 42 tokens a tile
    ([20] * 12, [130 * i + 20 for i in range(12)], 16, 8),    # more units than parts would pay for
], ids=str)
def test_units_of_very_different_lengths(lib, new, lens, Hq, Hkv, window):
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 32, Hq, Hkv, 128, "bf16", 57)
    ref = OR.paged(q, kp, vp, table, off, ln, window=window, cap=30.0)
    args = tuple(t.cuda() for t in (q, kp, vp, table, off, ln))
    O, L = lib.mesh_paged_attention(*args, max(new), window=window, cap=30.0)
    check(O, L, ref, "bf16", False)
    again = lib.mesh_paged_attention(*args, max(new), window=window, cap=30.0)
    assert torch.equal(O, again[0]) and torch.equal(L, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, lens", [([1, 1], [900, 131]), ([70, 1, 33], [5000, 3000, 40])], ids=str)
def test_what_a_workspace_holds_behind_its_head_does_not_matter(lib, dtype, new, lens):
    q, _, _, kp, vp, table, off, ln = (t.cuda() for t in cache(new, lens, 16, 8, 2, 64, dtype, 60))
    want = lib.mesh_paged_attention(q, kp, vp, table, off, ln, max(new))
    ws = lib.new_paged_workspace(q, kp, table, max(new))
    ws[2048:].fill_(255)  # NaN
    got = lib.mesh_paged_attention(q, kp, vp, table, off, ln, max(new), workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_more_sequences_than_are_sorted(lib):
    """900 sequences in one call, one of them with a chunk: more groups of tokens than the plan takes."""
    new, lens = [1] * 450 + [40] + [1] * 449, [1 + 7 * i % 50 for i in range(900)]
    lens[450] = 75
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 1, 64, "bf16", 58)
    ref = OR.paged(q, kp, vp, table, off, ln)
    O, L = lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), 40)
    check(O, L, ref, "bf16", False)


def test_offsets_that_do_not_fit_in_a_sorted_batch(lib):
    """Offsets beyond the batch, not ascending and negative where groups are sorted and cut: recorded, and the next call is right."""
    q, _, _, kp, vp, table, off, ln = (t.cuda() for t in cache([30, 1, 40], [300, 200, 2000], 16, 64, 64, 64, "bf16", 61))
    ws, st = lib.new_paged_workspace(q, kp, table, 40), lib.new_status()
    keep = dict(workspace=ws, status=st, check_status=False)
    want = [t.clone() for t in lib.mesh_paged_attention(q, kp, vp, table, off, ln, 40, **keep)]
    assert lib.mesh_attn_read_status(st) == 0
    for bad in ([0, 30, 90, 90], [71, 1, 0, 2], [-4, 1, 2, 3], [1 << 30, 0, -(1 << 30), 5]):
        lib.mesh_paged_attention(q, kp, vp, table, torch.tensor(bad, dtype=torch.int32, device="cuda"), ln, 40, **keep)
        assert lib.mesh_attn_read_status(st) == 6  # MESH_ATTN_ERR_OUT_OF_RANGE
        got = lib.mesh_paged_attention(q, kp, vp, table, off, ln, 40, **keep)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, lens", [([1, 1], [900, 131]), ([40, 25], [2000, 500])], ids=str)
def test_a_recorded_page_keeps_no_later_call_from_its_work(lib, dtype, new, lens):
    q, _, _, kp, vp, table, off, ln = (t.cuda() for t in cache(new, lens, 16, 8, 2, 64, dtype, 59))
    ws, st = lib.new_paged_workspace(q, kp, table, max(new)), lib.new_status()
    keep = dict(workspace=ws, status=st, check_status=False)
    want = [t.clone() for t in lib.mesh_paged_attention(q, kp, vp, table, off, ln, max(new), **keep)]
    assert lib.mesh_attn_read_status(st) == 0
    bad = table.clone()
    bad[1, 2] = -7
    got = lib.mesh_paged_attention(q, kp, vp, bad, off, ln, max(new), **keep)
    assert lib.mesh_attn_read_status(st) == 6  # MESH_ATTN_ERR_OUT_OF_RANGE
    assert torch.equal(got[0][:new[0]], want[0][:new[0]])  # the other sequence's rows
    got = lib.mesh_paged_attention(q, kp, vp, table, off, ln, max(new), **keep)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_batch_padded_behind(lib):
    """Rows behind the last sequence are left as they are, by both kernels and in both types."""
    for dtype in ("bf16", "f32"):
        for new, lens in (([1, 1], [50, 3]), ([60, 9], [90, 9])):
            q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 2, 64, dtype, 44)
            ref = OR.paged(q, kp, vp, table, off, ln)
            N = q.shape[0]
            qp = torch.cat([q, torch.full((7, 4, 64), math.nan, dtype=q.dtype)]).cuda()
            O, L = torch.full_like(qp, 7.0), torch.full((N + 7, 4), 7.0, device="cuda")
            lib.mesh_paged_attention(qp, *(t.cuda() for t in (kp, vp, table, off, ln)), max(new), O=O, LSE=L)
            check(O[:N], L[:N], ref, dtype, False)
            assert (O[N:] == 7).all() and (L[N:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 40]], ids=str)
def test_what_does_not_fit_is_recorded(lib, dtype, new):
    """Pages, lengths, offsets and bounds that do not fit: recorded, and the sequences that do fit come out right."""
    lens = [90, 33, 100]
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 1, 64, dtype, 45)
    ref = OR.paged(q, kp, vp, table, off, ln)
    dev = [t.cuda() for t in (q, kp, vp)]

    def call(t, o, l, bound):
        st = lib.new_status()
        out = lib.mesh_paged_attention(*dev, t.cuda(), o.cuda(), l.cuda(), bound, status=st, check_status=False)
        return out, lib.mesh_attn_read_status(st)

    for spoil in ("page", "negative", "long", "short", "bound"):
        t, l, bound = table.clone(), ln.clone(), max(new)
        if spoil == "page":
            t[0, 2] = kp.shape[0] + 5
        elif spoil == "negative":
            t[0, 2] = -7
        elif spoil == "long":
            l[0] = 16 * t.shape[1] + 1
        elif spoil == "short":
            l[0] = new[0] - 1
        elif max(new) > 1:
            bound = 35  # the last sequence has more
        (O, L), code = call(t, off, l, bound)
        if spoil == "bound":
            assert code == (6 if max(new) > 1 else 0)
            rows = slice(0, new[0] + new[1])
        else:
            assert code == 6, spoil
            rows = slice(new[0], None)
        check(O[rows], L[rows], tuple(x[rows] for x in ref), dtype, False)
    # offsets beyond the batch, or out of order: recorded, and nothing outside is touched
    for bad in ([0, new[0], q.shape[0] + 9, q.shape[0] + 9], [0, 2, 1, q.shape[0]], [-4, 1, 2, 3], [q.shape[0], 1, 0, 2], [3, 2, 1, 0],
                [1 << 30, 0, -(1 << 30), 5]):
        assert call(table, torch.tensor(bad, dtype=torch.int32), ln, max(new))[1] == 6
    # and the next good call in the same context is right
    (O, L), code = call(table, off, ln, max(new))
    assert code == 0
    check(O, L, ref, dtype, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_serving_loop(lib, dtype):
    """Prompts in chunks, then steps, in one workspace and captured once: the same as attention over the whole sequences, by
    mesh_range_attention's own numbers for them (cap, slopes and positions alike)."""
    Hq, Hkv, d, page, T = 4, 2, 64, 16, 120
    lens = [120, 77, 1]
    g = torch.Generator().manual_seed(46)
    full = [[torch.randn(n, h, d, generator=g).to(DT[dtype]) for h in (Hq, Hkv, Hkv)] for n in lens]
    sl, cap = slopes_of(Hq, True), 25.0
    rope = lib.MeshRope(d, (32,))
    # the dense way: each sequence a document of one row
    q, k, v = (torch.cat([f[i] for f in full]).transpose(0, 1)[None].contiguous() for i in range(3))
    pos = torch.cat([torch.arange(n) for n in lens])
    qr, kr = lib.mesh_rope(q.cuda(), k.cuda(), pos.cuda(), rope)
    lo, hi = lib.mesh_ranges(lens)
    want, wantL = lib.mesh_range_attention(qr, kr, v.cuda(), lo.cuda(), hi.cuda(), cap=cap, slopes=sl.cuda())
    ref = OR.forward(qr.cpu(), kr.cpu(), v, lo, hi, cap=cap, slopes=sl)
    # the paged way: two chunks of each prompt, all but the last 3 tokens, then single steps
    kp = torch.full((24, Hkv, page, d), math.nan, dtype=DT[dtype], device="cuda")
    vp = kp.clone()
    table = torch.arange(24, dtype=torch.int32).view(3, 8).cuda()
    O, L = torch.zeros(sum(lens), Hq, d), torch.zeros(sum(lens), Hq)
    start = [0, lens[0], lens[0] + lens[1]]
    have = [0, 0, 0]
    ws = None

    def run(new):
        nonlocal ws
        tok = [torch.cat([full[b][i][have[b]:have[b] + new[b]] for b in range(3)]).cuda() for i in range(3)]
        for b in range(3):
            have[b] += new[b]
        off = torch.tensor([sum(new[:b]) for b in range(4)], dtype=torch.int32, device="cuda")
        ln = torch.tensor(have, dtype=torch.int32, device="cuda")
        qq = lib.mesh_paged_append(*tok, kp, vp, table, off, ln, rope=rope)
        if ws is None:
            ws = lib.new_paged_workspace(qq, kp, table, max(new))
        o, l = lib.mesh_paged_attention(qq, kp, vp, table, off, ln, max(new), cap=cap, slopes=sl.cuda(), workspace=ws)
        at = 0
        for b in range(3):
            rows = slice(start[b] + have[b] - new[b], start[b] + have[b])
            O[rows], L[rows] = o[at:at + new[b]].cpu().float(), l[at:at + new[b]].cpu()
            at += new[b]

    run([70, 60, 0])
    run([47, 14, 0])
    run([1, 1, 1])
    run([1, 1, 0])
    run([1, 1, 0])
    assert have == lens
    Or, Lr, mag = (x[0].transpose(0, 1) for x in ref)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    # the appended keys and queries are the rotated ones bit for bit, so only the attention differs
    within(O, Or, u * Or.abs() + (u + 2.0 ** -12) * mag + 1e-4, "O")
    within(L, Lr, torch.full_like(Lr, 1e-3 if dtype == "bf16" else 1e-4), "LSE")
    within(want[0].transpose(0, 1), Or, u * Or.abs() + (u + 2.0 ** -12) * mag + 1e-4, "O, dense")


@pytest.mark.parametrize("new, Hq", [([1, 1, 1, 1], 8), ([40, 1, 25, 3], 4)], ids=str)
def test_captured_steps_with_other_lengths(lib, new, Hq):
    """A graph of append and attention replayed with other lengths, tables and pages in the same memory; two at once on two streams."""
    lens = [90, 300, 25, 1000]
    sets = []
    for s in (47, 48):
        q, k, v, kp, vp, table, off, ln = cache(new, lens, 16, Hq, 2, 128, "bf16", s)
        sets.append([t.cuda() for t in (q, k, v, kp, vp, table, off, ln)])
    rope = lib.MeshRope(128, (64,))
    spaces = [lib.new_paged_workspace(s[0], s[3], s[5], max(new)) for s in sets]
    stats = [lib.new_status() for _ in sets]

    def step(s, ws, st):
        q, k, v, kp, vp, table, off, ln = s
        qq = lib.mesh_paged_append(q, k, v, kp, vp, table, off, ln, rope=rope, status=st, check_status=False)
        return lib.mesh_paged_attention(qq, kp, vp, table, off, ln, max(new), workspace=ws, status=st, check_status=False)

    want = [step(s, w, st) for s, w, st in zip(sets, spaces, stats)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                outs[i].append(step(sets[i], spaces[i], stats[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for got in outs[i] for a, b in zip(got, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(sets[0], spaces[0], stats[0])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    sets[0][7].copy_(torch.tensor([95, 64, 200, 3], dtype=torch.int32).clamp(min=torch.tensor(new, dtype=torch.int32)))
    sets[0][5][2] = sets[0][5][3]  # the third sequence's pages are the fourth's now
    sets[0][5][3] = sets[0][5][1].clone()
    again = [t.clone() for t in sets[0]]
    graph.replay()
    torch.cuda.synchronize()
    fresh = step(again, lib.new_paged_workspace(again[0], again[3], again[5], max(new)), stats[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, fresh))
    assert all(lib.mesh_attn_read_status(st) == 0 for st in stats)


def test_a_workspace_serves_sizes_in_turn(lib):
    """One workspace, made for the largest batch: a chunk, a step, a chunk of few units in parts, a step again."""
    big = cache([200, 300], [200, 2000], 16, 8, 2, 128, "bf16", 49)
    small = cache([1, 1, 1], [700, 50, 1500], 16, 8, 2, 128, "bf16", 50)
    mid = cache([20], [4000], 16, 8, 2, 128, "bf16", 51)
    args = lambda c: [c[i].cuda() for i in (0, 3, 4, 5, 6, 7)]  # noqa: E731
    ws = lib.new_paged_workspace(big[0].cuda(), big[3].cuda(), torch.zeros(3, 1, dtype=torch.int32), 300)
    for c, bound in ((big, 300), (small, 1), (mid, 20), (small, 1), (big, 300), (small, 1)):
        O, L = lib.mesh_paged_attention(*args(c), bound, workspace=ws)
        O1, L1 = lib.mesh_paged_attention(*args(c), bound)
        assert torch.equal(O, O1) and torch.equal(L, L1)
    with pytest.raises(lib.MeshAttnError):
        lib.mesh_paged_attention(*args(big), 300, workspace=ws[: 1 << 20])


def test_no_tokens(lib):
    q, k, v, kp, vp, table, off, ln = cache([0, 0], [5, 9], 16, 4, 2, 64, "bf16", 52)
    dev = [t.cuda() for t in (q, k, v, kp, vp, table, off, ln)]
    assert lib.mesh_paged_append(*dev).shape == (0, 4, 64)
    O, L = lib.mesh_paged_attention(dev[0], *dev[3:], 1)
    assert O.shape == (0, 4, 64) and L.shape == (0, 4)


def test_waits_that_run_out(lib):
    q, _, _, kp, vp, table, off, ln = cache([700, 1], [1500, 60], 16, 8, 2, 128, "bf16", 53)
    dev = [t.cuda() for t in (q, kp, vp, table, off, ln)]
    want = lib.mesh_paged_attention(*dev, 700)
    for limit in (0, 1, 2_000, 20_000):
        st = lib.new_status()
        lib.mesh_attn_set_wait_limit_ns(limit)
        try:
            out = lib.mesh_paged_attention(*dev, 700, status=st, check_status=False)
            code = lib.mesh_attn_read_status(st)
        finally:
            lib.mesh_attn_set_wait_limit_ns(2_000_000_000)
        assert code in ((5,) if limit == 0 else (0, 5))  # one look at a barrier waits a microsecond or so by itself
        if code == 0:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(lib.mesh_paged_attention(*dev, 700), want))
