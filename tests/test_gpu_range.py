"""Range-masked attention (forward, backward, autograd) against the fp64 oracle.

Elementwise bounds, derived from the arithmetic (u = finfo.eps / 2, 2^-8 for bf16; mag: the oracle's sums over absolute terms, n the
terms of a sum):
  O, bf16      u |O| (rounded once) + u mag (P rounded to bf16 for its product) + (2^-12 + n 2^-23) mag (exponentials, the scores of exact
               bf16 products in fp32, the cap's polynomial: 6e-7 of a score below cap 50 is 2^-15; fp32 accumulation)
  LSE          1e-3 for bf16 inputs and 1e-4 for fp32: the tolerances of the plain attention calls
  O, fp32      1e-4, as the plain attention calls: inputs are N(0, 1)
  gradients    bf16: u |ref| + (u + 2^-9 + n 2^-23) mag: P or dS rounded once, D from the rounded O, the forward's LSE;
               fp32: 1e-4 (1 + mag)
"""
import math

import pytest
import torch

from oracle import range_attention as OR

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, Hq, Hkv, S, d, dtype, seed, q_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])  # noqa: E731
    return n(B, Hq, S, d) * q_scale, n(B, Hkv, S, d), n(B, Hkv, S, d), n(B, Hq, S, d)


def within(got, ref, bound, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), f"{what}: non-finite pattern differs"
    assert torch.equal(got[~fin], ref[~fin]), f"{what}: infinities differ"
    ratio = ((got - ref).abs() / bound)[fin]
    worst = ratio.max().item() if ratio.numel() else 0.0
    print(f"{what}: {worst:.3f} of the bound")
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def check_out(O, L, ref, dtype, n):
    Or, Lr, mag = ref
    if dtype == "bf16":
        within(O, Or, 2.0 ** -8 * Or.abs() + (2.0 ** -8 + 2.0 ** -12 + n * 2.0 ** -23) * mag + 1e-6, "O")
        within(L, Lr, torch.full_like(Lr, 1e-3), "LSE")
    else:
        within(O, Or, torch.full_like(Or, 1e-4), "O")
        within(L, Lr, torch.full_like(Lr, 1e-4), "LSE")


def check_grads(got, ref, dtype, S, g):
    for name, x in zip(("q", "k", "v"), got):
        r, mag = ref[name]
        n = S * (1 if name == "q" else g)
        b = 1e-4 * (1 + mag) if dtype == "f32" else 2.0 ** -8 * r.abs() + (2.0 ** -8 + 2.0 ** -9 + n * 2.0 ** -23) * mag + 1e-6
        within(x, r, b, "d" + name)


def mask_of(kind, B, S, seed=0):
    """lo, hi [S] or [B, S] on the host."""
    i = torch.arange(S, dtype=torch.int32)
    if kind == "causal":
        return torch.zeros_like(i), i + 1
    if kind == "all":
        return torch.zeros_like(i), torch.full_like(i, S)
    if kind == "docs":
        cut = sorted({0, S, S // 5, S // 5 + 1, S // 2, max(0, S - 3)})
        lo = torch.zeros_like(i)
        for c in cut:
            lo[c:] = c
        return lo, i + 1
    if kind == "prefix":
        half = S // 2
        hi = i + 1
        hi[: S // 3] = S // 3
        lo = torch.where(i >= half, torch.full_like(i, half), torch.zeros_like(i))
        return lo, hi
    if kind == "window":
        return torch.clamp(i - 36, min=0), i + 1
    if kind == "batch":  # another mask for each batch entry, padding behind
        out = []
        for b in range(B):
            lo, hi = mask_of(["docs", "causal", "window"][b % 3], 1, S)
            end = S - (b * S) // 4
            hi = hi.clamp(max=end)
            hi[end:] = 0
            out.append((lo, hi))
        return torch.stack([o[0] for o in out]), torch.stack([o[1] for o in out])
    g = torch.Generator().manual_seed(seed)  # any ranges: bounds outside, empty ones, in no order
    lo = torch.randint(-5, S + 5, (B, S), generator=g, dtype=torch.int32)
    return lo, lo + torch.randint(-20, S, (B, S), generator=g, dtype=torch.int32)


# B, Hq, Hkv, S, d, mask, cap, slopes
CASES = [
    (1, 1, 1, 1, 128, "causal", 0.0, False),
    (1, 2, 1, 2, 64, "all", 5.0, False),
    (2, 2, 2, 63, 128, "docs", 0.0, False),
    (1, 4, 2, 128, 64, "causal", 0.0, True),
    (2, 3, 1, 129, 128, "prefix", 30.0, False),
    (1, 4, 4, 257, 64, "any", 0.0, False),
    (3, 6, 2, 300, 128, "batch", 0.0, True),
    (1, 5, 1, 301, 64, "window", 2.0, True),
    (2, 2, 1, 513, 128, "any", 1.0, True),
    (1, 8, 1, 385, 128, "docs", 50.0, False),
    (1, 7, 7, 200, 128, "all", 0.0, True),
    (1, 16, 1, 190, 64, "causal", 0.3, False),
    (1, 2, 2, 1100, 64, "docs", 20.0, True),
]


def slopes_of(Hq, yes):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)]) if yes else None


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_both_directions(lib, case, dtype):
    B, Hq, Hkv, S, d, kind, cap, steep = case
    q, k, v, g = inputs(B, Hq, Hkv, S, d, dtype, 20)
    lo, hi = mask_of(kind, B, S)
    sl = slopes_of(Hq, steep)
    qd, kd, vd, gd, lod, hid, sd = dev(q, k, v, g, lo, hi, sl)
    O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid, cap=cap, slopes=sd)
    check_out(O, L, OR.forward(q, k, v, lo, hi, cap=cap, slopes=sl), dtype, S)
    grads = lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd, cap=cap, slopes=sd)
    check_grads(grads, OR.backward(q, k, v, g, lo, hi, cap=cap, slopes=sl), dtype, S, Hq // Hkv)
    again = lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd, cap=cap, slopes=sd)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap, q_scale", [(0.0, 6.0), (40.0, 6.0), (8.0, 6.0), (3000.0, 6.0), (1e6, 1.0)], ids=str)
def test_large_scores_and_caps(lib, dtype, cap, q_scale):
    """Scores beyond the cap, near it and far below it: every tier of the cap, and references that grow by more than 2^8."""
    q, k, v, g = inputs(1, 2, 1, 400, 128, dtype, 21, q_scale)
    k = k * torch.linspace(0.1, 2.0, 400)[None, None, :, None].to(k.dtype)
    lo, hi = mask_of("docs", 1, 400)
    qd, kd, vd, gd, lod, hid = dev(q, k, v, g, lo, hi)
    O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid, cap=cap)
    ref = OR.forward(q, k, v, lo, hi, cap=cap)
    if dtype == "bf16":
        check_out(O, L, ref, dtype, 400)
        grads = lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd, cap=cap)
        check_grads(grads, OR.backward(q, k, v, g, lo, hi, cap=cap), dtype, 400, 2)
    else:  # scores of 50 and more: fp32's own rounding of them, 2^-24 * 50 * 2, is in the exponent
        within(O, ref[0], 1e-4 + 1e-4 * ref[2], "O")
        within(L, ref[1], torch.full_like(ref[1], 2e-4), "LSE")


@pytest.mark.parametrize("shape", [(1, 1, 1, 2304, 128), (2, 4, 1, 700, 64), (1, 2, 1, 8200, 64)], ids=str)
def test_few_units_in_parts(lib, shape):
    """Whole tensors of few units, which go in parts of their keys: the same as the oracle on a few rows, whatever the workspace held."""
    B, Hq, Hkv, S, d = shape
    q, k, v, g = inputs(B, Hq, Hkv, S, d, "bf16", 22)
    lo, hi = mask_of("causal", B, S)
    qd, kd, vd, gd, lod, hid = dev(q, k, v, g, lo, hi)
    ws = lib.new_range_workspace(qd, kd, backward=True)
    outs = []
    for fill in (0, 255):
        ws.fill_(fill)
        O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid, workspace=ws)
        ws.fill_(fill)
        outs.append((O, L) + tuple(lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd, workspace=ws)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    O, L = outs[0][:2]
    plan = lib.mesh_attn_plan_create(S, 1, True)
    P, PL = lib.mesh_attention(qd, kd, vd, 1, True, plan=plan)
    PG = lib.mesh_attention_backward(qd, kd, vd, O, L, gd, 1, True, plan=plan)
    # two kernels of the same arithmetic: a rounding of P and of the result each
    assert (O.float() - P.float()).norm() <= 2.0 ** -7 * P.float().norm() and (L - PL).abs().max() <= 1e-4
    for a, b in zip(outs[0][2:], PG):
        assert (a.float() - b.float()).norm() <= 2.0 ** -6 * b.float().norm()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows_and_keys(lib, dtype):
    """Rows that see nothing: 0, -inf and no gradients, for any O and dO there; keys nobody sees: gradients of zero."""
    S = 390
    q, k, v, g = inputs(2, 4, 2, S, 64, dtype, 23)
    lo, hi = torch.full((S,), 140, dtype=torch.int32), torch.full((S,), 250, dtype=torch.int32)
    hi[37] = 140
    lo[200:300] = 250
    qd, kd, vd, gd, lod, hid = dev(q, k, v, g, lo, hi)
    O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid)
    blind = [37] + list(range(200, 300))
    assert (O[:, :, blind] == 0).all() and (L[:, :, blind] == -math.inf).all()
    dq, dk, dv = lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd)
    assert (dq[:, :, blind] == 0).all()
    assert (dk[:, :, :140] == 0).all() and (dv[:, :, :140] == 0).all() and (dk[:, :, 250:] == 0).all() and (dv[:, :, 250:] == 0).all()
    assert (dv[:, :, 140:250] != 0).any()
    none = torch.zeros(S, dtype=torch.int32, device="cuda")
    O, L = lib.mesh_range_attention(qd, kd, vd, none, none, cap=3.0, slopes=torch.ones(4, device="cuda"))
    assert (O == 0).all() and (L == -math.inf).all()
    for x in lib.mesh_range_attention_backward(qd, kd, vd, none, none, O, L, gd, cap=3.0):
        assert (x == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steep_slopes_with_far_keys_only(lib, dtype):
    """Ranges that leave out a row's own key: all weights lie far below those of its neighbourhood."""
    S = 700
    q, k, v, g = inputs(1, 2, 1, S, 64, dtype, 24)
    i = torch.arange(S, dtype=torch.int32)
    lo, hi = torch.where(i < 350, i + 300, torch.zeros_like(i)), torch.where(i < 350, torch.full_like(i, S), i - 290)
    sl = torch.tensor([0.7, 3.0])
    O, L = lib.mesh_range_attention(*dev(q, k, v, lo, hi), slopes=sl.cuda())
    Or, Lr, mag = OR.forward(q, k, v, lo, hi, slopes=sl)
    u = 2.0 ** -8 if dtype == "bf16" else 0.0
    within(O, Or, u * Or.abs() + (u + 2.0 ** -11) * mag + 1e-4, "O")
    within(L, Lr, 1e-3 + 2.0 ** -22 * Lr.abs().nan_to_num(0, 0, 0) * 4, "LSE")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nan_query_stays_in_its_row(lib, dtype):
    q, k, v, g = inputs(1, 4, 2, 300, 128, dtype, 25)
    lo, hi = mask_of("causal", 1, 300)
    qd, kd, vd, lod, hid = dev(q, k, v, lo, hi)
    for cap in (0.0, 20.0):
        O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid, cap=cap)
        bad = qd.clone()
        bad[0, 1, 130, 5] = math.nan
        On, Ln = lib.mesh_range_attention(bad, kd, vd, lod, hid, cap=cap)
        assert On[0, 1, 130].isnan().all() and Ln[0, 1, 130].isnan()
        rest = torch.ones(1, 4, 300, dtype=torch.bool)
        rest[0, 1, 130] = False
        # the others' pass over a block may differ with the NaN row's, by a rounding
        assert (On[rest.cuda()].float() - O[rest.cuda()].float()).abs().max() <= 2.0 ** -7 * 4
        assert torch.isfinite(On[rest.cuda()]).all() and (Ln - L)[rest.cuda()].abs().max() <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd(lib, dtype):
    q, k, v, g = (t.cuda() for t in inputs(2, 4, 2, 150, 64, dtype, 26))
    lo, hi = (t.cuda() for t in mask_of("batch", 2, 150))
    sl = slopes_of(4, True).cuda()
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    O, L = lib.mesh_range_attention_autograd(*leaves, lo, hi, cap=15.0, slopes=sl)
    O.backward(g.transpose(1, 2).contiguous().transpose(1, 2))
    O1, L1 = lib.mesh_range_attention(q, k, v, lo, hi, cap=15.0, slopes=sl)
    grads = lib.mesh_range_attention_backward(q, k, v, lo, hi, O1, L1, g, cap=15.0, slopes=sl)
    assert torch.equal(O, O1) and torch.equal(L, L1) and not L.requires_grad
    for a, b in zip(leaves, grads):
        assert torch.equal(a.grad, b)
    with pytest.raises(ValueError):
        lib.mesh_range_attention_autograd(*leaves, lo, hi, slopes=sl.clone().requires_grad_())
    st = lib.new_status()
    O, _ = lib.mesh_range_attention_autograd(*leaves, lo, hi, check_status=False, status=st)
    (O.float() ** 2).sum().backward()
    assert lib.mesh_attn_read_status(st) == 0


def test_no_rows(lib):
    for shape in ((0, 4, 2, 10, 64), (1, 4, 2, 0, 64), (1, 0, 2, 10, 64)):
        q, k, v, g = (t.cuda() for t in inputs(*shape, "bf16", 27))
        lo = torch.zeros(shape[3], dtype=torch.int32, device="cuda")
        O, L = lib.mesh_range_attention(q, k, v, lo, lo)
        assert O.shape == q.shape and L.shape == q.shape[:3]
        dq, dk, dv = lib.mesh_range_attention_backward(q, k, v, lo, lo, O, L, g)
        assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_streams_graphs_and_two_at_once(lib, dtype):
    sets = [[t.cuda() for t in inputs(1, 4, 2, 520, 64, dtype, s)] for s in (28, 29)]
    lo, hi = (t.cuda() for t in mask_of("docs", 1, 520))
    want, spaces, stats = [], [], [lib.new_status() for _ in sets]
    for q, k, v, g in sets:
        O, L = lib.mesh_range_attention(q, k, v, lo, hi, cap=30.0)
        want.append((O, L) + tuple(lib.mesh_range_attention_backward(q, k, v, lo, hi, O, L, g, cap=30.0)))
        spaces.append(lib.new_range_workspace(q, k, backward=True))
    torch.cuda.synchronize()

    def step(i):
        q, k, v, g = sets[i]
        kw = dict(cap=30.0, workspace=spaces[i], status=stats[i], check_status=False)
        O, L = lib.mesh_range_attention(q, k, v, lo, hi, **kw)
        return (O, L) + tuple(lib.mesh_range_attention_backward(q, k, v, lo, hi, O, L, g, **kw))

    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for got in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(0)
    for t in got:
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    # other inputs and another mask in the same memory
    for a, b in zip(sets[0], sets[1]):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    assert all(lib.mesh_attn_read_status(s) == 0 for s in stats)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_autograd_step(lib, dtype):
    """torch.autograd.grad inside a graph, no other autograd graph of the same tensors being alive."""
    lo, hi = (t.cuda() for t in mask_of("docs", 2, 300))
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda")
    st = lib.new_status()

    def step(q, k, v, g):
        O, L = lib.mesh_range_attention_autograd(q, k, v, lo, hi, cap=20.0, slopes=slopes, check_status=False, status=st)
        return (O.detach(), L, *torch.autograd.grad(O, (q, k, v), g))

    def fresh(seed):
        return [t.cuda().requires_grad_(i < 3) for i, t in enumerate(inputs(2, 4, 2, 300, 64, dtype, seed))]

    bufs, new = fresh(41), fresh(42)
    want = step(*new)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*bufs)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = step(*bufs)
    with torch.no_grad():
        for b, x in zip(bufs, new):
            b.copy_(x)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert lib.mesh_attn_read_status(st) == 0


def test_waits_that_run_out(lib):
    """Every role stops, copies and products are drained, and the next call in the same context gives the same bits.  Without any time
    nothing starts.  One look at a barrier waits a microsecond or so by itself, which the forward's waits may get by with; in the backward
    pass the warps that store dQ wait for a unit of up to 16 blocks of a microsecond each."""
    q, k, v, g = (t.cuda() for t in inputs(2, 8, 2, 2048, 128, "bf16", 30))
    lo, hi = (t.cuda() for t in mask_of("causal", 1, 2048))
    O, L = lib.mesh_range_attention(q, k, v, lo, hi)
    want = (O, L) + tuple(lib.mesh_range_attention_backward(q, k, v, lo, hi, O, L, g))
    ws = lib.new_range_workspace(q, k, backward=True)

    def fwd(st):
        return lib.mesh_range_attention(q, k, v, lo, hi, workspace=ws, status=st, check_status=False)

    def bwd(st):
        return lib.mesh_range_attention_backward(q, k, v, lo, hi, O, L, g, workspace=ws, status=st, check_status=False)

    for call, ref in ((fwd, want[:2]), (bwd, want[2:])):
        for limit in (0, 1, 2_000, 20_000):
            for _ in range(3):
                st = lib.new_status()
                lib.mesh_attn_set_wait_limit_ns(limit)
                try:
                    out = call(st)
                    code = lib.mesh_attn_read_status(st)
                finally:
                    lib.mesh_attn_set_wait_limit_ns(2_000_000_000)
                assert code in ((5,) if limit == 0 or (limit == 1 and call is bwd) else (0, 5)), (limit, st.tolist())
                if code == 0:
                    assert all(torch.equal(a, b) for a, b in zip(out, ref))
        st = lib.new_status()
        assert all(torch.equal(a, b) for a, b in zip(call(st), ref)) and lib.mesh_attn_read_status(st) == 0
    # calls behind one that failed do nothing
    st = torch.tensor([5, 0, 0, 0], dtype=torch.int32, device="cuda")
    o, l = torch.full_like(O, 7.0), torch.full_like(L, 7.0)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    lib.mesh_range_attention(q, k, v, lo, hi, O=o, LSE=l, workspace=ws, status=st, check_status=False)
    lib.mesh_range_attention_backward(q, k, v, lo, hi, O, L, g, dQ=grads[0], dK=grads[1], dV=grads[2], workspace=ws, status=st,
                                      check_status=False)
    assert lib.mesh_attn_read_status(st) == 5 and all((t == 7).all() for t in [o, l] + grads)


def test_many_blocks_of_one_mask(lib):
    """More query blocks than are sorted by length: the order of a causal mask, and all of it right."""
    S = 128 * 515 + 7
    q, k, v, g = (t.cuda() for t in inputs(1, 1, 1, S, 64, "bf16", 31))
    i = torch.arange(S, dtype=torch.int32, device="cuda")
    lo = torch.clamp(i - 200, min=0)
    O, L = lib.mesh_range_attention(q, k, v, lo, i + 1)
    dq, dk, dv = lib.mesh_range_attention_backward(q, k, v, lo, i + 1, O, L, g)
    a, z = S - 700, S  # the last rows, as a batch of their own
    part = [t[:, :, a:z].contiguous() for t in (q, k, v, g)]
    lp, hp = (lo[a:z] - a), (i[a:z] + 1 - a)
    Op, Lp = lib.mesh_range_attention(*part[:3], lp, hp)
    gp = lib.mesh_range_attention_backward(*part[:3], lp, hp, Op, Lp, part[3])
    # rows from the 201st of it on see the same keys, keys from there on the same rows; tiles begin elsewhere: a rounding of P
    tol = lambda x: 2.0 ** -6 * x.float().norm()  # noqa: E731
    for x, y in ((O, Op), (dq, gp[0]), (dk, gp[1]), (dv, gp[2])):
        assert (x[:, :, a + 201:].float() - y[:, :, 201:].float()).norm() <= tol(y[:, :, 201:])
    assert (L[:, :, a + 201:] - Lp[:, :, 201:]).abs().max() <= 1e-4
