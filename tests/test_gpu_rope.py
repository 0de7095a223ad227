"""Rotary positions with several axes against the fp64 oracle, over types, pair styles, groups, odd pair counts,
strides, alignments and far positions; the backward pass against the transpose; autograd and graphs."""
import pytest
import torch

from oracle import diff_attention as OD

pytestmark = pytest.mark.gpu

# Elementwise bound.  A result is rounded to its type once: u |y|, u = finfo.eps / 2.  Before that, in fp32,
# relative to |a| + |b|: the angle is exact to 2^-25 of a half turn (pi 2^-25 < 2^-23 rad, so each of sine and cosine
# is off by that), sincospi by at most 2 ulp (2^-23 each), and products and sum round three times
# (3 * 2^-24): under 2^-21 together.
REL = 2.0 ** -21


def bound(y, mag, dtype):
    return torch.finfo(dtype).eps / 2 * y.abs() + REL * mag + 1e-30


def make(shape, dtype, seed, layout="bhsd"):
    g = torch.Generator().manual_seed(seed)
    B, H, S, d = shape
    if layout == "bshd":
        return torch.randn(B, S, H, d, generator=g).to(dtype).transpose(1, 2)
    if layout == "gap":  # a slice of a wider tensor: rows further apart than they are long
        return torch.randn(B, H, S, d + 8, generator=g).to(dtype)[..., :d]
    if layout == "odd":  # rows that start at no 16-byte boundary
        return torch.randn(B, H, S, d + 3, generator=g).to(dtype)[..., 1: d + 1]
    return torch.randn(B, H, S, d, generator=g).to(dtype)


def positions(axes, B, S, seed, far=1 << 20, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-far, far, (axes, B, S), generator=g, dtype=dtype)


def check(lib, rope, x, pos, y, inverse=False):
    ref, mag = OD.rope(x, pos, rope.freq, rope.axis, rope.groups, rope.style == "adjacent", inverse)
    err = (y.double().cpu() - ref).abs()
    ratio = (err / bound(ref, mag, x.dtype)).max().item() if err.numel() else 0.0
    assert ratio <= 1.0, ratio


CASES = [  # dtype, d, groups, sections, style, freq, layout
    (torch.bfloat16, 128, 2, (12, 10, 10), "half", "global", "bshd"),
    (torch.bfloat16, 128, 1, (64,), "half", "global", "bhsd"),
    (torch.bfloat16, 64, 1, (14, 14), "adjacent", "axial", "bshd"),
    (torch.bfloat16, 64, 2, (7, 6), "adjacent", "global", "bhsd"),
    (torch.bfloat16, 128, 2, (11, 9, 9), "half", "axial", "gap"),
    (torch.bfloat16, 64, 1, (16, 16), "half", "axial", "odd"),
    (torch.float32, 64, 1, (32,), "adjacent", "global", "bshd"),
    (torch.float32, 128, 2, (12, 10, 10), "half", "axial", "gap"),
    (torch.float32, 64, 2, (1,), "half", "global", "odd"),
    (torch.float32, 6, 1, (1, 1), "half", "axial", "bhsd"),
    (torch.bfloat16, 1024, 2, (100, 100, 56), "adjacent", "global", "bhsd"),
]


@pytest.mark.parametrize("S", [1, 37])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(lib, case, S):
    dtype, d, groups, sections, style, freq, layout = case
    rope = lib.MeshRope(d, sections, groups=groups, style=style, freq=freq)
    q, k = make((2, 3, S, d), dtype, 1, layout), make((2, 2, S, d), dtype, 2, layout)
    pos = positions(len(sections), 2, S, 3)
    q_d, k_d, p_d = q.cuda(), k.cuda(), pos.cuda()
    if layout == "odd":  # .cuda() lays tensors out anew: take the view on the device
        q_d = torch.nn.functional.pad(q_d, (1, 2))[..., 1: d + 1]
        k_d = torch.nn.functional.pad(k_d, (1, 2))[..., 1: d + 1]
        assert q_d.data_ptr() % 16
    elif layout == "gap":
        q_d, k_d = (torch.nn.functional.pad(t, (0, 8))[..., :d] for t in (q_d, k_d))
    elif layout == "bshd":
        q_d, k_d = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q_d, k_d))
    yq, yk = lib.mesh_rope(q_d, k_d, p_d, rope)
    assert yq.is_contiguous() and yk.is_contiguous() and yq.dtype == dtype
    check(lib, rope, q, pos, yq)
    check(lib, rope, k, pos, yk)
    dq, dk = lib.mesh_rope_backward(q_d, k_d, p_d, rope)
    check(lib, rope, q, pos, dq, inverse=True)
    check(lib, rope, k, pos, dk, inverse=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "adjacent"])
@pytest.mark.parametrize("n", [32, 28, 30, 29])  # pairs of 64 columns: 16, 8, 4 and 2 bytes of bf16 an access
@pytest.mark.parametrize("shift", [0, 2, 4])     # elements by which the tensors begin off a 16-byte boundary
def test_every_width_of_access(lib, dtype, style, n, shift):
    rope = lib.MeshRope(64, (n,), style=style)
    x, pos = make((2, 3, 9, 64), dtype, 8), positions(1, 2, 9, 9)
    x_d = torch.nn.functional.pad(x.cuda(), (shift, 8 - shift))[..., shift: shift + 64]  # rows 72 elements apart
    out = torch.full((2, 3, 9, 72), 7.0, dtype=dtype, device="cuda")
    lib.mesh_attn_rope(rope, x_d, None, pos.cuda(), out[..., shift: shift + 64], None)
    check(lib, rope, x, pos, out[..., shift: shift + 64])
    assert (out[..., :shift] == 7).all() and (out[..., shift + 64:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions_of_either_width_shared_and_strided(lib, dtype):
    rope = lib.MeshRope(64, (8, 8), groups=2)
    q = make((3, 2, 40, 64), torch.float32, 5)
    pos = positions(2, 1, 80, 6, dtype=dtype, far=1 << 30)
    y, none = lib.mesh_rope(q.cuda(), None, pos.cuda()[:, 0, ::2], rope)  # [axes, S], every other one
    assert none is None
    check(lib, rope, q, pos[:, :, ::2].expand(2, 3, 40), y)


def test_very_far_positions(lib):
    """2^40 turns no digit into noise: the oracle's own angle is off by 2^40 * 2^-53, ours by 2^40 2^-54 turns."""
    rope = lib.MeshRope(64, (32,), freq=[0.5 ** i for i in range(32)])
    q = make((1, 1, 16, 64), torch.float32, 7)
    # multiples of 2^31 apart: int32 arithmetic anywhere would show
    pos = (torch.arange(16) * (1 << 31) - (1 << 34)).view(1, 1, 16)
    y, _ = lib.mesh_rope(q.cuda(), None, pos.cuda(), rope)
    ref, mag = OD.rope(q, pos, rope.freq, rope.axis)
    # both angles: at most 2^35 positions * (2^-54 turns * 2 pi + 2^-53 rad) < 2^-16 rad, each way
    err = (y.double().cpu() - ref).abs()
    assert (err <= (REL + 2.0 ** -15) * mag).all()


def test_interleaved_axes_and_own_frequencies(lib):
    axis = [i % 3 for i in range(24)]
    freq = [0.1 * (i + 1) for i in range(24)]
    rope = lib.MeshRope(64, (8, 8, 8), freq=freq, axis_of_pair=axis)
    q, pos = make((1, 2, 9, 64), torch.float32, 8), positions(3, 1, 9, 9, far=1000)
    y, _ = lib.mesh_rope(q.cuda(), None, pos.cuda(), rope)
    ref, mag = OD.rope(q, pos, freq, axis)
    assert ((y.double().cpu() - ref).abs() <= bound(ref, mag, torch.float32)).all()


def test_in_place_and_no_tokens(lib):
    rope = lib.MeshRope(128, (32,), groups=2)
    q, k = make((2, 4, 50, 128), torch.bfloat16, 10).cuda(), make((2, 1, 50, 128), torch.bfloat16, 11).cuda()
    pos = positions(1, 2, 50, 12).cuda()
    yq, yk = lib.mesh_rope(q, k, pos, rope)
    lib.mesh_attn_rope(rope, q, k, pos, q, k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    for shape in ((0, 4, 50, 128), (2, 4, 0, 128), (2, 0, 50, 128)):
        x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        y, _ = lib.mesh_rope(x, None, torch.zeros(1, shape[0], shape[2], dtype=torch.int64, device="cuda"), rope)
        assert y.shape == x.shape


def test_autograd_keeps_the_projections_layout(lib):
    rope = lib.MeshRope(64, (6, 5, 5), groups=2)
    B, S = 2, 33
    xq = make((B, S, 4, 64), torch.float32, 13).cuda().requires_grad_(True)
    xk = make((B, S, 2, 64), torch.float32, 14).cuda().requires_grad_(True)
    pos = positions(3, B, S, 15).cuda()
    q, k = lib.mesh_rope_autograd(xq.transpose(1, 2), xk.transpose(1, 2), pos, rope)
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    torch.autograd.backward((q, k), (gq, gk))
    for x, y, gy in ((xq, q, gq), (xk, k, gk)):
        assert x.grad.is_contiguous()
        ref, mag = OD.rope(gy.cpu(), pos.cpu(), rope.freq, rope.axis, 2, False, True)
        assert ((x.grad.transpose(1, 2).double().cpu() - ref).abs() <= bound(ref, mag, torch.float32)).all()
        # against differences: the map is linear, so <y(x + e) - y(x), g> = <e, x.grad>
        e = torch.randn_like(x)
    moved = lib.mesh_rope((xk.detach() + e).transpose(1, 2), None, pos, rope)[0]
    lhs = ((moved - k.detach()).double() * gk.double()).sum().item()
    rhs = (e.double() * xk.grad.double()).sum().item()
    # each of the 3 B S H d fp32 roundings enters the two sums once, |values| below 10: a worst case of 2^-22 * 30 each
    assert abs(lhs - rhs) <= x.numel() * 30 * 2.0 ** -22
    # an expanded gradient, and one of the two outputs unused
    q, k = lib.mesh_rope_autograd(xq.transpose(1, 2), xk.transpose(1, 2), pos, rope)
    (g,) = torch.autograd.grad(q.sum(), xq)
    ref, mag = OD.rope(torch.ones_like(q).cpu(), pos.cpu(), rope.freq, rope.axis, 2, False, True)
    assert ((g.transpose(1, 2).double().cpu() - ref).abs() <= bound(ref, mag, torch.float32)).all()


def test_captured_and_on_another_stream(lib):
    rope = lib.MeshRope(64, (32,))
    q = make((2, 3, 20, 64), torch.bfloat16, 16).cuda()
    pos = positions(1, 2, 20, 17).cuda()
    y = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.mesh_attn_rope(rope, q, None, pos, y, None)
    q.copy_(make((2, 3, 20, 64), torch.bfloat16, 18))
    pos += 7
    g.replay()
    torch.cuda.synchronize()
    check(lib, rope, q.cpu(), pos.cpu(), y)
    z = torch.empty_like(q)
    torch.cuda.synchronize()
    lib.mesh_attn_rope(rope, q, None, pos, z, None, stream=s)
    s.synchronize()
    assert torch.equal(y, z)
