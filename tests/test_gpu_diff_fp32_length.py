"""fp32 differential attention's error does not grow with the length.

Norm-wise, in units of 2^-24.  The tensor cores truncate: an addition loses an ulp at most, half an ulp (one unit of
the partial sum) on average, always towards zero.  A block's products take 24 additions, during which the partial sum grows
from nothing: 12 units of the block's value, and so of the whole sum, since the blocks are added with rounding.  A score
costs 12 in the same way and a dP of 128 columns 24; exponentials, LSE, row terms and the roundings around them 16.
Summed on the tensor cores throughout, 64 blocks would lose 64 * 12 for the sums alone.
"""
import pytest
import torch

from oracle import diff_attention as OD
from tests.test_gpu_diff import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape, causal", [((1, 1, 1, 4096, 64), True), ((1, 1, 1, 3001, 128), False), ((1, 2, 1, 130, 128), True)],
                         ids=str)
def test_error_at_any_length(lib, shape, causal):
    q, k, v, lam, g = inputs(*shape, "f32", 45)
    dev = [t.cuda() for t in (q, k, v, lam)]
    O, O2, L = lib.mesh_diff_attention(*dev, 1, causal, return_saved=True)
    grads = lib.mesh_diff_attention_backward(*dev, O, O2, L, g.cuda(), 1, causal)
    ref = OD.backward(q, k, v, lam, g, causal)
    rows = [("O", O, OD.forward(q, k, v, lam, causal)[0], 12 + 12 + 16), ("dV", grads[2], ref["v"][0], 12 + 12 + 16)]
    rows += [("d" + n, x, ref[n][0], 12 + 12 + 24 + 16) for n, x in zip("qk", grads)]
    for name, x, r, units in rows:
        e = ((x.double().cpu() - r).norm() / r.norm()).item()
        print(f"{name}: {e:.2e} of {units * 2.0 ** -24:.2e}")
        assert e <= units * 2.0 ** -24, (name, e)
