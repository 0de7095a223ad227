"""A query row with a NaN: its output and its LSEs are NaN, in both types, and no other row's are touched."""
import pytest
import torch

from tests.test_gpu_diff import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 300, 128), (1, 1, 1, 2304, 64), (2, 40, 40, 300, 64)], ids=str)  # whole and in parts
@pytest.mark.parametrize("causal", [False, True])
def test_nan_stays_nan(lib, dtype, shape, causal):
    q, k, v, lam, _ = (t.cuda() for t in inputs(*shape, dtype, 77))
    row = 201
    bad = q.clone()
    bad[0, 0, row, 3] = float("nan")                   # the first map's half
    bad[0, 0, row + 7, shape[4] - 1] = float("nan")    # the second map's
    want = lib.mesh_diff_attention(q, k, v, lam, 1, causal)
    O, L = lib.mesh_diff_attention(bad, k, v, lam, 1, causal)
    assert torch.isnan(O[0, 0, [row, row + 7]]).all()
    assert torch.isnan(L[0, 0, 0, row]) and torch.isnan(L[0, 0, 1, row + 7])
    for r in (row, row + 7):  # everything else as without them
        O[0, 0, r], L[0, 0, :, r] = want[0][0, 0, r], want[1][0, 0, :, r]
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])
