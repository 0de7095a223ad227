"""Range-masked attention at bounds, scores and caps of any size, both directions, against the fp64 oracle.  Bounds as in
test_gpu_range.py."""
import pytest
import torch

from oracle import range_attention as OR
from tests.test_gpu_range import check_grads, check_out, dev, inputs, mask_of, slopes_of, within

pytestmark = pytest.mark.gpu

LOW, HIGH = torch.iinfo(torch.int32).min, torch.iinfo(torch.int32).max


def both(lib, q, k, v, g, lo, hi, dtype, n, **kw):
    """Both directions by the kernels, checked against the oracle."""
    qd, kd, vd, gd, lod, hid = dev(q, k, v, g, lo, hi)
    kd_ = {a: x.cuda() if torch.is_tensor(x) else x for a, x in kw.items()}
    O, L = lib.mesh_range_attention(qd, kd, vd, lod, hid, **kd_)
    check_out(O, L, OR.forward(q, k, v, lo, hi, **kw), dtype, n)
    grads = lib.mesh_range_attention_backward(qd, kd, vd, lod, hid, O, L, gd, **kd_)
    check_grads(grads, OR.backward(q, k, v, g, lo, hi, **kw), dtype, n, q.shape[1] // k.shape[1])


def far_mask(kind, S):
    i = torch.arange(S, dtype=torch.int32)
    if kind == "causal":  # no lower bound
        return torch.full_like(i, LOW), i + 1
    if kind == "all":  # none at all
        return torch.full_like(i, LOW), torch.full_like(i, HIGH)
    if kind == "padding":  # rows behind that see nothing, as far out as it goes
        lo, hi = torch.full_like(i, LOW + 1), i + 1
        lo[S - 70:], hi[S - 70:] = HIGH, LOW
        return lo, hi
    lo, hi = torch.clamp(i - 36, min=0), i + 1  # every bound there is, row beside row
    lo[1::7], lo[2::7], lo[3::7], lo[4::7] = LOW, LOW + 130, -1, HIGH
    hi[1::5], hi[2::5], hi[3::5] = HIGH, HIGH - 130, LOW
    return lo, hi


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["causal", "all", "padding", "mixed"])
@pytest.mark.parametrize("S, d", [(100, 64), (300, 128), (700, 64)], ids=str)
def test_bounds_of_any_size(lib, S, d, kind, dtype):
    """Bounds outside 0 .. S are the nearer bound, down to the type's lowest value and up to its highest."""
    q, k, v, g = inputs(1, 4, 2, S, d, dtype, 70)
    lo, hi = far_mask(kind, S)
    both(lib, q, k, v, g, lo, hi, dtype, S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap, steep", [(0.0, False), (0.0, True), (5.0, False)], ids=str)
def test_masked_scores_beyond_every_number(lib, cap, steep, dtype):
    """Padding whose scores overflow fp32, as queries and as keys, beside rows that see whole blocks: it reaches no gradient."""
    S, n = 384, 300
    q, k, v, g = inputs(1, 2, 1, S, 64, dtype, 71)
    q[:, :, n:] = torch.sign(q[:, :, n:].float()).to(q.dtype) * 2e38
    k[:, :, n:] = torch.sign(k[:, :, n:].float()).to(k.dtype) * 2e38
    lo, hi = torch.zeros(S, dtype=torch.int32), torch.full((S,), n, dtype=torch.int32)
    hi[n:] = 0
    both(lib, q, k, v, g, lo, hi, dtype, S, cap=cap, slopes=slopes_of(2, steep))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale, cap", [(1.0, 2e-7), (0.125, 1e-5), (1e-4, 1e-18), (0.05, 1e15), (2e4, 1e18)], ids=str)
def test_caps_far_from_the_scores(lib, scale, cap, dtype):
    """Caps far below and far above the scores, and queries of zeros, whose scores are 0 whatever the cap."""
    S = 200
    q, k, v, g = inputs(1, 4, 2, S, 64, dtype, 72)
    if scale > 1:
        q = q * (1.0 / 65536)
    q[:, :, ::3] = 0
    q[:, :, 40:160] = 0  # whole warps of them
    lo, hi = mask_of("docs", 1, S)
    both(lib, q, k, v, g, lo, hi, dtype, S, scale=scale, cap=cap)


@pytest.mark.parametrize("shape, kind", [((1, 1, 1, 2304, 128), "causal"), ((2, 4, 1, 700, 64), "causal"), ((1, 2, 1, 8200, 64), "causal"),
                                         ((1, 2, 2, 2304, 64), "prefix"), ((1, 2, 1, 3001, 128), "docs")], ids=str)
def test_every_row_of_units_in_parts(lib, shape, kind):
    """Few long units, which go in parts of their keys: every row and key, those at the borders of parts and tiles among them."""
    B, Hq, Hkv, S, d = shape
    q, k, v, g = inputs(B, Hq, Hkv, S, d, "bf16", 73)
    lo, hi = mask_of(kind, B, S)
    both(lib, q, k, v, g, lo, hi, "bf16", S)
