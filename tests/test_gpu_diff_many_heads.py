"""fp32 differential attention of many short sequences and of many heads: nothing but the number of rows bounds a call."""
import pytest
import torch

from oracle import diff_attention as OD
from tests.test_gpu_diff import check_grads, check_out, inputs, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B, Hq, Hkv, S", [(10000, 2, 1, 16), (1, 66000, 33000, 3)], ids=str)
def test_many_short_sequences_and_many_heads(lib, B, Hq, Hkv, S):
    q, k, v, lam, g = inputs(B, Hq, Hkv, S, 64, "f32", 90)
    dev = [t.cuda() for t in (q, k, v, lam)]
    O, O2, L = lib.mesh_diff_attention(*dev, 1, True, return_saved=True)
    dq, dk, dv, dlam = (t.cpu() for t in lib.mesh_diff_attention_backward(*dev, O, O2, L, g.cuda(), 1, True))
    O, O2, L = O.cpu(), O2.cpu(), L.cpu()
    # the oracle on the first, the last and those around the old limits (8,192 sequences, 65,536 heads)
    for b in ((0, 8190, 8191, 8192, B - 1) if B > 1 else (0,)):
        for j in ((0, 32766, 32767, 32768, Hkv - 1) if Hkv > 1 else (0,)):
            hq, hk = slice(2 * j, 2 * j + 2), slice(j, j + 1)
            a = [q[b:b + 1, hq], k[b:b + 1, hk], v[b:b + 1, hk], lam[hq]]
            check_out(O[b:b + 1, hq], L[b:b + 1, hq], OD.forward(*a, True), "f32", S)
            ref = OD.backward(*a, g[b:b + 1, hq], True)
            got = [dq[b:b + 1, hq], dk[b:b + 1, hk], dv[b:b + 1, hk]]
            check_grads(got, ref, "f32", S, 2)
            if B == 1:
                within(dlam[hq], ref["lam"][0], 1e-5 * (1 + ref["lam"][1]), "dlam")
    # lam's gradient over all sequences, from the outputs: each term g . O2 is off by 1e-4 |g| of O2 at most
    want = -(g.double() * O2.double()).sum((0, 2, 3))
    assert torch.isfinite(dlam).all()
    assert ((dlam.double() - want).abs() <= 1e-5 * (1 + (g.double() * O2.double()).abs().sum((0, 2, 3)))).all()
