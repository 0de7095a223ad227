"""The fp64 oracle of range-masked attention against the plain attention oracle, central differences and closed forms, and
mesh_ranges against its words (on the CPU)."""
import math

import pytest
import torch

from oracle import range_attention as OR
from oracle.attention import attention_bhsd


def rand(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def causal(S):
    return torch.zeros(S, dtype=torch.int32), torch.arange(1, S + 1, dtype=torch.int32)


def test_without_extras_it_is_plain_attention():
    q, k, v = rand(2, 4, 33, 16, seed=1), rand(2, 2, 33, 16, seed=2), rand(2, 2, 33, 16, seed=3)
    O, L, _ = OR.forward(q, k, v, *causal(33))
    Or, Lr = attention_bhsd(q, k, v, True)
    assert (O - Or).abs().max() < 1e-12 and (L - Lr).abs().max() < 1e-12


def test_closed_forms():
    S = 9
    lo = torch.tensor([0, 0, 2, 3, 3, 5, 9, 7, -4], dtype=torch.int32)
    hi = torch.tensor([1, 0, 2, 9, 4, 8, 9, 20, 3], dtype=torch.int32)
    k, v = rand(1, 1, S, 8, seed=4), rand(1, 1, S, 8, seed=5)
    O, L, _ = OR.forward(torch.zeros(1, 1, S, 8), k, v, lo, hi)
    for i in range(S):  # equal scores: the mean of the visible values and ln of their number
        a, z = max(int(lo[i]), 0), min(int(hi[i]), S)
        if a >= z:
            assert (O[0, 0, i] == 0).all() and L[0, 0, i] == -math.inf
        else:
            assert torch.allclose(O[0, 0, i], v[0, 0, a:z].mean(0)) and abs(L[0, 0, i] - math.log(z - a)) < 1e-12
    # a steep slope leaves each row its own token; a small cap leaves scores of +-cap
    q = rand(1, 1, S, 8, seed=6)
    O, _, _ = OR.forward(q, k, v, *causal(S), slopes=[1e4])
    assert torch.allclose(O, v)
    q1, k1 = torch.full((1, 1, 2, 8), 50.0), torch.ones(1, 1, 2, 8)
    k1[0, 0, 1] = -1
    _, L, _ = OR.forward(q1, k1, v[:, :, :2], *causal(2), cap=0.5)
    assert abs(L[0, 0, 1] - math.log(math.exp(0.5) + math.exp(-0.5))) < 1e-12


@pytest.mark.parametrize("cap, slopes", [(0.0, None), (0.7, None), (0.0, [0.3, 0.05]), (1.5, [0.2, 0.0])], ids=str)
def test_gradients_against_differences(cap, slopes):
    S = 11
    q, k, v, go = rand(1, 2, S, 6, seed=7), rand(1, 1, S, 6, seed=8), rand(1, 1, S, 6, seed=9), rand(1, 2, S, 6, seed=10)
    lo = torch.tensor([0, 0, 0, 0, 4, 4, 4, 4, 8, 9, 10], dtype=torch.int32)
    hi = torch.tensor([3, 3, 3, 4, 5, 6, 7, 8, 8, 11, 11], dtype=torch.int32)
    got = OR.backward(q, k, v, go, lo, hi, cap=cap, slopes=slopes)

    def loss(q, k, v):
        return (OR.forward(q, k, v, lo, hi, cap=cap, slopes=slopes)[0] * go).sum()

    args = dict(q=q, k=k, v=v)
    for n in args:
        u, e = rand(*args[n].shape, seed=11), 1e-6
        d = (loss(**{**args, n: args[n] + e * u}) - loss(**{**args, n: args[n] - e * u})) / (2 * e)
        assert abs(d - (got[n][0] * u).sum()) < 1e-7, n
        assert (got[n][0].abs() <= got[n][1] + 1e-12).all()


def test_paged_is_the_dense_one():
    S, page, Hq, Hkv, d = 21, 8, 4, 2, 8
    q, k, v = rand(1, Hq, S, d, seed=12), rand(1, Hkv, S, d, seed=13), rand(1, Hkv, S, d, seed=14)
    table = torch.tensor([[4, 1, 3]], dtype=torch.int32)
    kp, vp = rand(5, Hkv, page, d, seed=15), rand(5, Hkv, page, d, seed=16)
    for i in range(S):
        kp[table[0, i // page], :, i % page], vp[table[0, i // page], :, i % page] = k[0, :, i], v[0, :, i]
    n = 6
    for window in (0, 1, 5):
        i = torch.arange(S, dtype=torch.int32)
        lo = torch.clamp(i - (window - 1), min=0) if window else torch.zeros_like(i)
        O, L, _ = OR.forward(q, k, v, lo, i + 1, cap=2.0, slopes=[0.1, 0.2, 0.3, 0.4])
        Op, Lp, _ = OR.paged(q[0].transpose(0, 1)[S - n:], kp, vp, table, [0, n], [S], cap=2.0, slopes=[0.1, 0.2, 0.3, 0.4],
                             window=window)
        assert (Op - O[0, :, S - n:].transpose(0, 1)).abs().max() < 1e-12 and (Lp.T - L[0, :, S - n:]).abs().max() < 1e-12


def test_ranges(lib):
    lo, hi = lib.mesh_ranges([3, 0, 2], length=6)
    assert lo.tolist() == [0, 0, 0, 3, 3, 0] and hi.tolist() == [1, 2, 3, 4, 5, 0]
    lo, hi = lib.mesh_ranges([3, 2], causal=False)
    assert lo.tolist() == [0, 0, 0, 3, 3] and hi.tolist() == [3, 3, 3, 5, 5]
    lo, hi = lib.mesh_ranges([4, 3], prefixes=[2, 9])
    assert lo.tolist() == [0, 0, 0, 0, 4, 4, 4] and hi.tolist() == [2, 2, 3, 4, 7, 7, 7]
    lo, hi = lib.mesh_ranges([5, 2], window=2)
    assert lo.tolist() == [0, 0, 1, 2, 3, 5, 5] and hi.tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert all(t.dtype == torch.int32 for t in (lo, hi))
    assert [t.tolist() for t in lib.mesh_ranges([])] == [[], []]
    for bad in (dict(documents=[-1]), dict(documents=[2], prefixes=[1, 1]), dict(documents=[2], window=-1), dict(documents=[2], length=1)):
        with pytest.raises(ValueError):
            lib.mesh_ranges(**bad)
