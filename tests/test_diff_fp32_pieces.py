"""fp32 differential attention keeps all of fp32's digits in its operands: a lost third bf16 piece of any one of them would show.

Norm-wise bound, in units of 2^-24 (the mean loss of a truncating addition, half an ulp): a row's sums take 24 additions a
block of 64 rows (six piece products of four steps), a score 24 and a dP 48 of the same kind at most, and the
exponentials, row terms and roundings to fp32 around them 16.  At 150 tokens that is 9.5e-6; an operand cut to 16
significant bits (two pieces) is off by 2^-17 a value and more, and moves each gradient it enters by 1.1e-5 or more.
"""
import pytest
import torch

from oracle import diff_attention as OD
from tests.test_gpu_diff import inputs


def bound(S):
    return (24 * min(13, (S + 63) // 64) + 24 + 48 + 16) * 2.0 ** -24


def err(x, ref):
    return ((x.double().cpu() - ref).norm() / ref.norm()).item()


def two_pieces(x):
    return (x.view(torch.int32) & ~0xff).view(torch.float32)


CASES = [((2, 4, 2, 150, d), causal) for d in (64, 128) for causal in (False, True)]
# which results each operand enters
ENTERS = {0: "Oqkv", 1: "Oqkv", 2: "Oqk", 4: "qkv"}


@pytest.mark.parametrize("case", CASES, ids=str)
def test_the_bound_would_show_a_lost_piece(case):
    """The mistake planted in the oracle's operands, one at a time (on the CPU)."""
    shape, causal = case
    args = inputs(*shape, "f32", 44)
    ref, out = OD.backward(*args, causal), OD.forward(*args[:4], causal)[0]
    for i, names in ENTERS.items():
        a = [two_pieces(t) if j == i else t for j, t in enumerate(args)]
        got, o = OD.backward(*a, causal), OD.forward(*a[:4], causal)[0]
        for n in names:
            e = err(o, out) if n == "O" else err(got[n][0], ref[n][0])
            assert e > bound(shape[3]), (i, n, e)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES + [((1, 4, 2, 1001, 128), True), ((1, 2, 1, 1500, 128), False)], ids=str)
def test_digits(lib, case):
    shape, causal = case
    args = inputs(*shape, "f32", 44)
    dev = [t.cuda() for t in args]
    O, O2, L = lib.mesh_diff_attention(*dev[:4], 1, causal, return_saved=True)
    grads = lib.mesh_diff_attention_backward(*dev[:4], O, O2, L, dev[4], 1, causal)
    ref = OD.backward(*args, causal)
    for name, x, r in [("O", O, OD.forward(*args[:4], causal)[0])] + [(n, x, ref[n][0]) for n, x in zip("qkv", grads)]:
        e = err(x, r)
        print(f"{name}: {e:.2e} of {bound(shape[3]):.2e}")
        assert e <= bound(shape[3]), (name, e)
