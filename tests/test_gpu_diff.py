"""Differential attention (forward, backward, single tokens over a cache) against the fp64 oracle.

Elementwise bounds, derived from the arithmetic (u = finfo.eps / 2, 2^-8 for bf16; mag: the oracle's sums over
absolute terms):
  O, bf16      u |O| (rounded once) + u mag (P rounded to bf16 for its product) + (2^-12 + n 2^-23) mag (exponentials, the
               fp32 scores of exact bf16 products, fp32 accumulation of n terms)
  LSE          1e-3 for bf16 inputs and 1e-4 for fp32: the tolerances of the plain attention calls
  O, fp32      1e-4 mag-free, as the plain attention calls: inputs are N(0, 1)
  gradients    bf16: u |ref| + (u + 2^-9 + n 2^-23) mag: P or dS rounded once, D from the rounded O and O2, the forward's
               LSE; fp32: 1e-4 * (1 + mag)
  dlam         u |ref| + (2^-9 + n 2^-23) sum |P2 dP| / sqrt-free worst case; n = S d terms a row
"""
import math

import pytest
import torch

from oracle import diff_attention as OD

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, Hq, Hkv, S, d, dtype, seed, T=None, lam_n=None, k_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = DT[dtype]
    q, k, v = n(B, Hq, S, d).to(t), (n(B, Hkv, T or S, d) * k_scale).to(t), n(B, Hkv, T or S, d).to(t)
    lam = (0.8 + 0.3 * n(lam_n or Hq)).to(t)
    return q, k, v, lam, n(B, Hq, S, d).to(t)


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
    Or, Lr, _, mag = ref
    if dtype == "bf16":
        within(O, Or, 2.0 ** -8 * Or.abs() + (2.0 ** -8 + 2.0 ** -12 + n * 2.0 ** -23) * mag + 1e-6, "O")
        within(L, Lr, torch.full_like(Lr, 1e-3), "LSE")
    else:
        within(O, Or, torch.full_like(Or, 1e-4), "O")
        within(L, Lr, torch.full_like(Lr, 1e-4), "LSE")


def check_grads(got, ref, dtype, S, g):
    for name, x in zip(("q", "k", "v", "lam"), got):
        r, mag = ref[name]
        n = S * (g if name in ("k", "v") else 1)
        if dtype == "f32":
            b = 1e-4 * (1 + mag) if name != "lam" else 1e-5 * (1 + mag)
        elif name == "lam":  # sums of P2 dP kept in fp32, rounded once at the end
            b = 2.0 ** -8 * r.abs() + (2.0 ** -9 + n * 2.0 ** -23) * mag + 1e-6
        else:
            b = 2.0 ** -8 * r.abs() + (2.0 ** -8 + 2.0 ** -9 + n * 2.0 ** -23) * mag + 1e-6
        within(x, r, b, "d" + name)


# B, Hq, Hkv, S, d, P (0: a ring plan of 3), causal
SHAPES = [
    (1, 1, 1, 1, 128, 1, True),
    (1, 2, 1, 2, 64, 1, False),
    (1, 2, 2, 63, 128, 1, True),
    (2, 2, 1, 64, 64, 1, True),
    (1, 2, 2, 65, 128, 1, False),
    (1, 4, 2, 129, 64, 1, True),
    (2, 3, 1, 300, 128, 1, True),
    (1, 4, 2, 516, 128, 4, True),
    (1, 2, 1, 516, 64, 4, False),
    (1, 2, 2, 1170, 128, 9, True),
    (1, 2, 1, 1170, 64, 9, False),
    (1, 2, 2, 459, 128, 0, True),
    (1, 1, 1, 1024, 128, 1, False),
    (1, 8, 1, 200, 128, 4, True),
]


def plan_of(lib, S, P, causal):
    return lib.mesh_attn_plan_create_ring(S, 3, causal) if P == 0 else lib.mesh_attn_plan_create(S, P, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(lib, shape, dtype):
    B, Hq, Hkv, S, d, P, causal = shape
    q, k, v, lam, _ = inputs(B, Hq, Hkv, S, d, dtype, 20)
    plan = plan_of(lib, S, P, causal)
    O, L = lib.mesh_diff_attention(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), P, causal, plan=plan)
    check_out(O, L, OD.forward(q, k, v, lam, causal), dtype, S)
    O1, O2, L1 = lib.mesh_diff_attention(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), P, causal, plan=plan, return_saved=True)
    assert torch.equal(O, O1) and torch.equal(L, L1)
    z = torch.zeros_like(lam)  # lam = 0 leaves the first map, and O2 is minus the second's share
    Oz, _ = lib.mesh_diff_attention(q.cuda(), k.cuda(), v.cuda(), z.cuda(), P, causal, plan=plan)
    check_out(Oz, L, OD.forward(q, k, v, z, causal), dtype, S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(lib, shape, dtype):
    B, Hq, Hkv, S, d, P, causal = shape
    q, k, v, lam, g = inputs(B, Hq, Hkv, S, d, dtype, 21)
    plan = plan_of(lib, S, P, causal)
    qd, kd, vd, ld = (t.cuda() for t in (q, k, v, lam))
    O, O2, L = lib.mesh_diff_attention(qd, kd, vd, ld, P, causal, plan=plan, return_saved=True)
    grads = lib.mesh_diff_attention_backward(qd, kd, vd, ld, O, O2, L, g.cuda(), P, causal, plan=plan)
    check_grads(grads, OD.backward(q, k, v, lam, g, causal), dtype, S, Hq // Hkv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_lam_for_all_heads_and_signs(lib, dtype):
    q, k, v, _, g = inputs(2, 4, 2, 150, 128, dtype, 22)
    for value in (0.0, -0.75, 2.5):
        lam = torch.tensor([value], dtype=DT[dtype])
        args = [t.cuda() for t in (q, k, v, lam)]
        O, O2, L = lib.mesh_diff_attention(*args, 1, True, return_saved=True)
        check_out(O, L, OD.forward(q, k, v, lam, True), dtype, 150)
        grads = lib.mesh_diff_attention_backward(*args, O, O2, L, g.cuda(), 1, True)
        assert grads[3].shape == (1,)
        check_grads(grads, OD.backward(q, k, v, lam, g, True), dtype, 150, 2)


@pytest.mark.parametrize("shape", [(1, 1, 1, 2304, 128, True), (1, 3, 1, 900, 64, False), (2, 8, 2, 1250, 64, False)], ids=str)
def test_few_tiles_and_a_last_wave_of_few(lib, shape):
    """Tiles cut into parts: all of 18 or 24, short ones among them that have fewer blocks than parts, and 8 of 160."""
    B, Hq, Hkv, S, d, causal = shape
    q, k, v, lam, _ = inputs(B, Hq, Hkv, S, d, "bf16", 41)
    dev = [t.cuda() for t in (q, k, v, lam)]
    plan = lib.mesh_attn_plan_create(S, 1, causal)
    outs = []
    for fill in (0, 255):
        ws = lib.new_diff_workspace(plan, dev[0], dev[1]).fill_(fill)
        outs.append(lib.mesh_diff_attention(*dev, 1, causal, plan=plan, workspace=ws, return_saved=True))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    check_out(outs[0][0], outs[0][2], OD.forward(q, k, v, lam, causal), "bf16", S)


@pytest.mark.parametrize("causal", [False, True])
def test_long_fp32_sums_keep_their_digits(lib, causal):
    """More keys than one accumulation on the tensor cores takes, in each pass.  Norm-wise: sums move on after 13 blocks of 64
    rows, each block 24 truncating additions that lose at most 2^-24 of the sum on average (half an ulp at worst, the
    mean of a truncation): 13 * 24 * 2^-24 = 1.9e-5, and a quarter of it in practice; without moving on, 2,000 rows
    would lose 32 * 24 * 2^-24 = 4.6e-5."""
    q, k, v, lam, g = inputs(1, 2, 1, 2000, 64, "f32", 42)
    dev = [t.cuda() for t in (q, k, v, lam)]
    O, O2, L = lib.mesh_diff_attention(*dev, 1, causal, return_saved=True)
    grads = lib.mesh_diff_attention_backward(*dev, O, O2, L, g.cuda(), 1, causal)
    ref = OD.backward(q, k, v, lam, g, causal)
    for name, x, r in [("O", O, OD.forward(q, k, v, lam, causal)[0])] + [("d" + n, x, ref[n][0]) for n, x in zip("qkv", grads)]:
        e = ((x.double().cpu() - r).norm() / r.norm()).item()
        print(f"{name}: {e:.2e}")
        assert e <= 13 * 24 * 2.0 ** -24, name


def test_large_scores(lib):
    """Scores of some hundred: the running maximum moves, most weights vanish."""
    q, k, v, lam, g = inputs(1, 2, 2, 300, 128, "bf16", 23, k_scale=16.0)
    args = [t.cuda() for t in (q, k, v, lam)]
    O, O2, L = lib.mesh_diff_attention(*args, 4, True, return_saved=True)
    Or, Lr, _, mag = OD.forward(q, k, v, lam, True)
    # a score of up to 2^10 in fp32 is off by 2^-14 + d 2^-24 2^10: its weight by a relative 2^-10, the LSE by 2^-12
    within(O, Or, 2.0 ** -8 * Or.abs() + (2.0 ** -8 + 2.0 ** -9) * mag + 1e-6, "O")
    within(L, Lr, torch.full_like(Lr, 1e-3), "LSE")


@pytest.mark.parametrize("P", [1, 4])
def test_references_that_have_to_rise(lib, P):
    """Scores that outgrow a row's first block by far more than 2^60, in one map, in the other, in one half of a block's
    keys or in both, several times in one sequence: the running reference rises block by block."""
    S, d = 1024, 128
    q, k, v, lam, g = inputs(1, 2, 1, S, d, "bf16", 35)
    q[..., 0] = 8.0   # a column of each map whose product with k lifts a key's score for every row
    q[..., 64] = 8.0
    k[..., 0] = k[..., 64] = 0.0
    scale = 1 / 8.0
    for key, a, b in ((200, 60.0, 0.0), (201, 0.0, 80.0), (330, 120.0, 0.0), (400, 130.0, 140.0), (450, 190.0, 145.0),
                      (700, 250.0, 220.0), (701, 252.0, 222.0), (1000, 310.0, 0.0)):
        k[:, :, key, 0], k[:, :, key, 64] = a, b
    args = [t.cuda() for t in (q, k, v, lam)]
    for causal in (False, True):
        O, O2, L = lib.mesh_diff_attention(*args, P, causal, scale=scale, return_saved=True)
        Or, Lr, _, mag = OD.forward(q, k, v, lam, causal, scale=scale)
        # scores up to 300 in fp32: 2^-15 and d 2^-24 of 300 off, a relative 2^-12 of a weight
        within(O, Or, 2.0 ** -8 * Or.abs() + (2.0 ** -8 + 2.0 ** -11) * mag + 1e-6, "O")
        within(L, Lr, torch.full_like(Lr, 1e-3), "LSE")


def test_equals_two_plain_attentions(lib):
    """O1 and O2 as the framework's plain calls give them, on q and k with the other half zeroed."""
    q, k, v, lam, _ = (t.cuda() for t in inputs(1, 2, 1, 256, 128, "bf16", 24))
    scale = 1 / math.sqrt(64)
    halves = []
    for part in (slice(0, 64), slice(64, 128)):
        qm = torch.zeros_like(q)
        qm[..., part] = q[..., part]
        halves.append(lib.mesh_attention(qm, k, v, 1, True, scale=scale))
    O, O2, L = lib.mesh_diff_attention(q, k, v, lam, 1, True, return_saved=True)
    assert torch.allclose(L[:, :, 0], halves[0][1], atol=2e-6, rtol=0) and torch.allclose(L[:, :, 1], halves[1][1], atol=2e-6, rtol=0)
    o1, o2 = (h[0].double() for h in halves)
    ref = o1 - lam.double().view(1, 2, 1, 1) * o2
    # On either side P is rounded for its product, u relative to sum P |v| of each map (mag carries both, the second times
    # lam), and exponentials and accumulation add 2^-12; o1, o2 and O are rounded once each.
    mag = OD.forward(*(t.cpu() for t in (q, k, v, lam)), True)[3].cuda()
    lo2 = (lam.double().view(1, 2, 1, 1) * o2).abs()
    bound = 2 * (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * (o1.abs() + lo2 + O.double().abs()) + 1e-6
    assert ((O.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd_and_differences(lib, dtype):
    q, k, v, lam, g = inputs(1, 2, 1, 96, 64, dtype, 25)
    leaves = [t.cuda().requires_grad_(True) for t in (q, k, v, lam)]
    O, L = lib.mesh_diff_attention_autograd(*leaves, 1, True)
    assert not L.requires_grad
    O.backward(g.cuda())
    check_grads([t.grad for t in leaves], OD.backward(q, k, v, lam, g, True), dtype, 96, 2)
    # the oracle's gradient against differences of the oracle's output, in fp64
    ref = OD.backward(q, k, v, lam, g, True)
    gen = torch.Generator().manual_seed(1)
    for i, name in enumerate(("q", "k", "v", "lam")):
        args = [t.double() for t in (q, k, v, lam)]
        e = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        f = []
        for h in (1e-6, -1e-6):
            a = list(args)
            a[i] = a[i] + h * e
            f.append((OD.forward(*a, True)[0] * g.double()).sum())
        d = ((f[0] - f[1]) / 2e-6).item()
        r = (ref[name][0] * e).sum().item()
        # central differences: h^2 times a third derivative of order the value, and 2^-53 |f| / h
        assert abs(d - r) <= 1e-5 * (1 + abs(r)), name


def test_shared_leaf_gradients_add_up(lib):
    """A lam expanded from one value, and k used twice: autograd sums what the calls return."""
    q, k, v, _, g = inputs(1, 2, 2, 70, 64, "f32", 26)
    one = torch.tensor([0.6], device="cuda", requires_grad=True)
    kd = k.cuda().requires_grad_(True)
    O, _ = lib.mesh_diff_attention_autograd(q.cuda(), kd, kd, one.expand(2).contiguous(), 1, False)
    O.backward(g.cuda())
    ref = OD.backward(q, k, k, torch.tensor([0.6]), g, False)
    within(one.grad, ref["lam"][0], 1e-5 * (1 + ref["lam"][1]), "dlam")
    within(kd.grad, ref["k"][0] + ref["v"][0], 1e-4 * (2 + ref["k"][1] + ref["v"][1]), "dk + dv")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [1, 4])
def test_same_bits_each_time_and_what_surrounds(lib, dtype, P):
    """Two runs give the same bits; a workspace full of NaN and outputs full of NaN change nothing."""
    q, k, v, lam, g = (t.cuda() for t in inputs(2, 4, 2, 520, 128, dtype, 27))
    plan = lib.mesh_attn_plan_create(520, P, True)
    runs = []
    for fill in (0, 255):
        ws = lib.new_diff_workspace(plan, q, k, backward=True).fill_(fill)
        O, O2, L = lib.mesh_diff_attention(q, k, v, lam, P, True, plan=plan, workspace=ws, return_saved=True)
        grads = [torch.full_like(t, float("nan")) for t in (q, k, v, lam)]
        ws.fill_(fill)
        st = lib.new_status()
        lib.mesh_attn_diff_bwd(plan, q, k, v, lam, O, O2, L, g, None, *grads, ws, st)
        assert lib.mesh_attn_read_status(st) == 0
        runs.append([O, O2, L, *grads])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_many_times(lib, d):
    """More units than SMs in both passes of the backward call, again and again: CTAs that follow one another on an SM, and
    units of one CTA, leave every wait satisfied (the status block stays clear) and every call gives the same bits."""
    q, k, v, lam, g = (t.cuda() for t in inputs(1, 16, 4, 4096, d, "bf16", 36))
    plan = lib.mesh_attn_plan_create(4096, 1, True)
    ws, st = lib.new_diff_workspace(plan, q, k, backward=True), lib.new_status()
    keep = dict(plan=plan, workspace=ws, status=st, check_status=False)
    O, O2, L = lib.mesh_diff_attention(q, k, v, lam, 1, True, return_saved=True, **keep)
    first = lib.mesh_diff_attention_backward(q, k, v, lam, O, O2, L, g, 1, True, **keep)
    for _ in range(50):
        again = lib.mesh_diff_attention_backward(q, k, v, lam, O, O2, L, g, 1, True, **keep)
        o, _ = lib.mesh_diff_attention(q, k, v, lam, 1, True, **keep)
    assert lib.mesh_attn_read_status(st) == 0, st.tolist()
    assert torch.equal(O, o)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_neighbours_nan_stays_out(lib):
    """NaN and infinities in another head, batch or partition's padding never reach a result: L = 100 is no multiple
    of a tile, so tiles reach past a partition's end."""
    for dtype in ("bf16", "f32"):
        q, k, v, lam, g = inputs(2, 2, 2, 400, 128, dtype, 28)
        bad = [t.clone() for t in (q, k, v, g)]
        for t in bad:
            t[1] = float("nan")
            t[0, 1] = float("inf")
        plan = lib.mesh_attn_plan_create(400, 4, True)
        outs = []
        for qq, kk, vv, gg in ((q, k, v, g), bad):
            args = [t.cuda() for t in (qq, kk, vv, lam)]
            O, O2, L = lib.mesh_diff_attention(*args, 4, True, plan=plan, return_saved=True)
            outs.append([O, L, *lib.mesh_diff_attention_backward(*args, O, O2, L, gg.cuda(), 4, True, plan=plan)[:3]])
        for a, b in zip(*outs):
            assert torch.equal(a[0, 0], b[0, 0]), dtype


def test_tables_of_another_plan_are_refused(lib):
    q, k, v, lam, _ = (t.cuda() for t in inputs(1, 1, 1, 64, 64, "bf16", 29))
    for dtype in (torch.bfloat16, torch.float32):
        q, k, v, lam = (t.to(dtype) for t in (q, k, v, lam))
        plan, other = lib.mesh_attn_plan_create(64, 1, True), lib.mesh_attn_plan_create(64, 1, False)
        ws, st = lib.new_diff_workspace(plan, q, k), lib.new_status()
        O, L = torch.full_like(q, 7.0), torch.full((1, 1, 2, 64), 7.0, device="cuda")
        plan._tables[torch.cuda.current_device()] = other.tables("cuda")
        lib.mesh_attn_diff_fwd(plan, q, k, v, lam, None, O, None, L, ws, st)
        assert lib.mesh_attn_read_status(st) == 1
        assert (O == 7).all() and (L == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_training_step(lib, dtype):
    """Forward and backward in one graph, replayed on other inputs; two graphs with workspaces of their own on two streams."""
    shape = (1, 2, 1, 200, 128)
    plan = lib.mesh_attn_plan_create(200, 1, True)
    plan.tables("cuda")
    st = lib.new_status()
    graphs = []
    for i in range(2):
        bufs = [t.cuda() for t in inputs(*shape, dtype, 30 + i)]
        ws = lib.new_diff_workspace(plan, bufs[0], bufs[1], backward=True)
        s, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr, stream=s):
            O, O2, L = lib.mesh_diff_attention(*bufs[:4], 1, True, plan=plan, workspace=ws, status=st, check_status=False,
                                               return_saved=True)
            grads = lib.mesh_diff_attention_backward(*bufs[:4], O, O2, L, bufs[4], 1, True, plan=plan, workspace=ws,
                                                     status=st, check_status=False)
        graphs.append((gr, s, bufs, O, L, grads))
    new = [inputs(*shape, dtype, 40 + i) for i in range(2)]
    for (gr, s, bufs, *_), n in zip(graphs, new):
        for b, x in zip(bufs, n):
            b.copy_(x)
    torch.cuda.synchronize()
    for gr, s, *_ in graphs:
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    assert lib.mesh_attn_read_status(st) == 0
    for (_, _, _, O, L, grads), (q, k, v, lam, g) in zip(graphs, new):
        check_out(O, L, OD.forward(q, k, v, lam, True), dtype, 200)
        check_grads(grads, OD.backward(q, k, v, lam, g, True), dtype, 200, 2)


def test_wait_limit_gives_an_error_and_the_next_call_works(lib):
    q, k, v, lam, g = (t.cuda() for t in inputs(1, 2, 2, 600, 128, "bf16", 33))
    O, O2, L = lib.mesh_diff_attention(q, k, v, lam, 1, True, return_saved=True)
    try:
        lib.mesh_attn_set_wait_limit_ns(0)
        with pytest.raises(lib.MeshAttnError) as e:
            lib.mesh_diff_attention(q, k, v, lam, 1, True)
        assert e.value.code == 5
        with pytest.raises(lib.MeshAttnError) as e:
            lib.mesh_diff_attention_backward(q, k, v, lam, O, O2, L, g, 1, True)
        assert e.value.code == 5
    finally:
        lib.mesh_attn_set_wait_limit_ns(2_000_000_000)
    O1, _ = lib.mesh_diff_attention(q, k, v, lam, 1, True)
    assert torch.equal(O, O1)


def test_backward_refuses_tables_of_another_plan(lib):
    for dtype in ("bf16", "f32"):
        q, k, v, lam, g = (t.cuda() for t in inputs(1, 1, 1, 64, 64, dtype, 37))
        plan, other = lib.mesh_attn_plan_create(64, 1, True), lib.mesh_attn_plan_create(64, 1, False)
        O, O2, L = lib.mesh_diff_attention(q, k, v, lam, 1, True, plan=plan, return_saved=True)
        grads = [torch.full_like(t, 7.0) for t in (q, k, v, lam)]
        plan._tables[torch.cuda.current_device()] = other.tables("cuda")
        ws, st = lib.new_diff_workspace(plan, q, k, backward=True), lib.new_status()
        lib.mesh_attn_diff_bwd(plan, q, k, v, lam, O, O2, L, g, None, *grads, ws, st)
        assert lib.mesh_attn_read_status(st) == 1, dtype
        for t in grads:
            assert (t == 7).all(), dtype


@pytest.mark.parametrize("B, Hq, Hkv, S", [(0, 2, 1, 8), (1, 0, 1, 8), (2, 2, 2, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows_give_zero_gradients(lib, B, Hq, Hkv, S, dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.ones(B, Hq, S, 64, dtype=t, device="cuda")
    k = torch.ones(B, Hkv, S, 64, dtype=t, device="cuda")
    lam = torch.ones(max(Hq, 1), dtype=t, device="cuda")
    O, O2, L = lib.mesh_diff_attention(q, k, k, lam, 1, True, return_saved=True)
    junk = [torch.full((64,), float("nan"), dtype=t, device="cuda") for _ in range(64)]
    del junk  # what the gradients' memory may hold
    for a in lib.mesh_diff_attention_backward(q, k, k, lam, O, O2, L, torch.ones_like(q), 1, True):
        assert (a == 0).all()


def test_dropped_plan_keeps_its_tables_until_another_stream_has_read_them(lib):
    q, k, v, lam, _ = (t.cuda() for t in inputs(1, 2, 1, 200, 64, "bf16", 38))
    plan = lib.mesh_attn_plan_create(200, 4, True)
    O, _ = lib.mesh_diff_attention(q, k, v, lam, 4, True, plan=plan)
    at, n = plan.tables("cuda").data_ptr(), plan.tables("cuda").numel()
    ws, st = lib.new_diff_workspace(plan, q, k), lib.new_status()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        late, _ = lib.mesh_diff_attention(q, k, v, lam, 4, True, plan=plan, workspace=ws, status=st, check_status=False)
    del plan
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert not s.query() and all(t.data_ptr() != at for t in others)
    torch.cuda.synchronize()
    assert lib.mesh_attn_read_status(st) == 0 and torch.equal(O, late)


def test_captured_autograd_step(lib):
    """torch.autograd.grad of both wrappers inside a graph: the plan and its tables exist before, and nothing waits."""
    rope = lib.MeshRope(64, (16,), groups=2)
    pos = torch.arange(130, device="cuda")
    plan = lib.mesh_attn_plan_create(130, 1, True)
    plan.tables("cuda")

    def step(q, k, v, lam, g):
        a, b = lib.mesh_rope_autograd(q, k, pos, rope)
        O, _ = lib.mesh_diff_attention_autograd(a, b, v, lam, 1, True, plan=plan, check_status=False)
        return (O.detach(), *torch.autograd.grad(O, (q, k, v, lam), g))

    def fresh(seed):
        return [t.cuda().requires_grad_(i < 4) for i, t in enumerate(inputs(1, 2, 1, 130, 64, "bf16", seed))]

    bufs, new = fresh(39), fresh(40)
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


# ------------------------------------------------------------------ single tokens over a cache

DECODE = [  # B, Hq, Hkv, d, T, lens
    (1, 1, 1, 128, 1, [1]),
    (1, 2, 2, 64, 16, [0]),
    (2, 4, 1, 128, 130, [130, 1]),
    (3, 3, 3, 64, 257, [0, 257, 128]),
    (2, 6, 2, 128, 1000, [129, 999]),
    (5, 8, 1, 64, 300, [0, 1, 2, 300, 127]),
    (2, 16, 1, 128, 700, [700, 300]),      # a group of 16: two head chunks
    (1, 12, 1, 64, 2000, [1999]),          # 8 + 4 heads
    (300, 1, 1, 64, 40, None),
    (1, 4, 2, 128, 40000, [39999]),        # every CTA a piece
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"B{c[0]}_{c[1]}_{c[2]}_d{c[3]}_T{c[4]}")
def test_decode(lib, case, dtype):
    B, Hq, Hkv, d, T, lens = case
    lens = torch.tensor(lens if lens is not None else [(7 * b) % (T + 1) for b in range(B)], dtype=torch.int32)
    q, k, v, lam, _ = inputs(B, Hq, Hkv, 1, d, dtype, 50, T=T)
    for b in range(B):  # what lies behind a sequence's tokens is never read
        k[b, :, lens[b]:] = float("nan")
        v[b, :, lens[b]:] = float("inf")
    ws = lib.new_diff_decode_workspace(B, Hq, Hkv, d, T)
    args = [t.cuda() for t in (q, k, v, lens, lam)]
    O, L = lib.mesh_diff_decode(*args, workspace=ws)
    check_out(O, L, OD.forward(q, k, v, lam, False, lens=lens), dtype, T)
    # the workspace serves the next call, and the bits do not depend on what was there
    O2, L2 = lib.mesh_diff_decode(*args, workspace=ws)
    assert torch.equal(O, O2) and torch.equal(L, L2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_strided_cache_and_shared_lam(lib, dtype):
    B, Hq, Hkv, d, T = 2, 4, 2, 64, 190
    q, k, v, _, _ = inputs(B, Hq, Hkv, 1, d, dtype, 51, T=T)
    lam = torch.tensor([0.7], dtype=DT[dtype])
    lens = torch.tensor([190, 65], dtype=torch.int32)
    both = torch.stack([k, v], 3).permute(0, 2, 3, 1, 4).contiguous().cuda()  # [B, T, 2, Hkv, d]
    kc, vc = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    O, L = lib.mesh_diff_decode(q.cuda(), kc, vc, lens.cuda(), lam.cuda())
    check_out(O, L, OD.forward(q, k, v, lam, False, lens=lens), dtype, T)


def test_decode_workspace_of_larger_sizes(lib):
    ws = lib.new_diff_decode_workspace(8, 16, 2, 128, 5000)
    for B, Hq, Hkv, d, T, seed in ((8, 16, 2, 128, 500, 52), (1, 2, 1, 64, 3000, 53), (3, 4, 2, 128, 77, 54), (8, 16, 2, 128, 500, 55)):
        q, k, v, lam, _ = inputs(B, Hq, Hkv, 1, d, "bf16", seed, T=T)
        lens = torch.full((B,), T, dtype=torch.int32)
        O, L = lib.mesh_diff_decode(q.cuda(), k.cuda(), v.cuda(), lens.cuda(), lam.cuda(), workspace=ws)
        check_out(O, L, OD.forward(q, k, v, lam, False, lens=lens), "bf16", T)


def test_decode_of_an_empty_cache(lib):
    for dtype in (torch.bfloat16, torch.float32):
        q = torch.ones(2, 4, 1, 64, dtype=dtype, device="cuda")
        cache = torch.empty(2, 2, 0, 64, dtype=dtype, device="cuda")
        O, L = lib.mesh_diff_decode(q, cache, cache, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                    torch.ones(4, dtype=dtype, device="cuda"))
        assert (O == 0).all() and (L == -math.inf).all()


def test_decode_lengths_out_of_range_are_reported(lib):
    q, k, v, lam, _ = inputs(2, 2, 1, 1, 64, "bf16", 56, T=100)
    args = [t.cuda() for t in (q, k, v)]
    st = lib.new_status()
    O, L = lib.mesh_diff_decode(*args, torch.tensor([-3, 1000], dtype=torch.int32).cuda(), lam.cuda(), status=st,
                                check_status=False)
    assert lib.mesh_attn_read_status(st) == 6
    check_out(O, L, OD.forward(q, k, v, lam, False, lens=[0, 100]), "bf16", 100)


def test_decode_captured_with_growing_lengths(lib):
    q, k, v, lam, _ = inputs(2, 4, 2, 1, 128, "bf16", 57, T=3000)
    lens = torch.tensor([1, 2900], dtype=torch.int32)
    args = [t.cuda() for t in (q, k, v, lens, lam)]
    ws, st = lib.new_diff_decode_workspace(2, 4, 2, 128, 3000), lib.new_status()
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        O, L = lib.mesh_diff_decode(*args, workspace=ws, status=st, check_status=False)
    for step in (0, 1, 60):
        now = lens + step
        args[3].copy_(now)
        gr.replay()
        torch.cuda.synchronize()
        check_out(O, L, OD.forward(q, k, v, lam, False, lens=now), "bf16", 3000)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_model_layer_trained_and_served(lib, dtype):
    """Projection -> rotary positions -> differential attention -> loss, with every gradient; then the same tokens one at
    a time over a cache, equal to the rows of the whole pass."""
    B, Hq, Hkv, S, d = 1, 4, 2, 150, 128
    t = DT[dtype]
    xq, xk, v, lam, g = inputs(B, Hq, Hkv, S, d, dtype, 60)
    xq, xk = xq.transpose(1, 2).contiguous(), xk.transpose(1, 2).contiguous()  # [B, S, H, d]
    rope = lib.MeshRope(d, (12, 10, 10), groups=2)
    i = torch.arange(S)
    pos = torch.stack([i // 16, i // 4 % 4, i % 4]).unsqueeze(1) + 70000
    leaves = [x.cuda().requires_grad_(True) for x in (xq, xk, v, lam)]
    q, k = lib.mesh_rope_autograd(leaves[0].transpose(1, 2), leaves[1].transpose(1, 2), pos.cuda(), rope)
    O, L = lib.mesh_diff_attention_autograd(q, k, leaves[2], leaves[3], 1, True)
    O.backward(g.cuda())
    qr, kr = q.detach().cpu(), k.detach().cpu()
    check_out(O.detach(), L, OD.forward(qr, kr, v, lam, True), dtype, S)
    ref = OD.backward(qr, kr, v, lam, g, True)
    for x, name, heads in ((leaves[0], "q", Hq), (leaves[1], "k", Hkv)):
        r, _ = OD.rope(ref[name][0], pos, rope.freq, rope.axis, 2, False, True)
        _, m = OD.rope(ref[name][1], pos, rope.freq, rope.axis, 2, False, True)
        n = S * (Hq // Hkv)
        u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        # the attention's gradient within its bound (rotated: both of a pair enter), then one rounding more
        b = (2 * u + 2.0 ** -8 + 2.0 ** -9 + n * 2.0 ** -23) * m * 2 + 1e-5 if dtype == "bf16" else 4e-4 * (1 + m)
        within(x.grad.transpose(1, 2), r, b, "dx" + name)
    kc, vc = torch.zeros(B, Hkv, S, d, dtype=t, device="cuda"), torch.zeros(B, Hkv, S, d, dtype=t, device="cuda")
    ws = lib.new_diff_decode_workspace(B, Hq, Hkv, d, S)
    full = OD.forward(qr, kr, v, lam, True)
    for s in (0, 1, 17, 127, 128, 149):
        q1, _ = lib.mesh_rope(leaves[0].detach()[:, s:s + 1].transpose(1, 2), None, pos.cuda()[:, :, s:s + 1], rope)
        lib.mesh_attn_rope(rope, leaves[1].detach()[:, :s + 1].transpose(1, 2), None, pos.cuda()[:, :, :s + 1], kc[:, :, :s + 1], None)
        vc[:, :, :s + 1] = v.cuda()[:, :, :s + 1]
        o, l = lib.mesh_diff_decode(q1, kc, vc, torch.tensor([s + 1], dtype=torch.int32, device="cuda"), leaves[3].detach(), workspace=ws)
        check_out(o, l, [x[:, :, s:s + 1] if x.dim() == 4 and x.shape[2] == S else x[..., s:s + 1] for x in full], dtype, S)
