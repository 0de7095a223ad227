"""Attention over a paged cache at the limits of its lengths, bounds, windows and status block, against the fp64 oracle.  Bounds as in
test_gpu_paged.py."""
import math

import pytest
import torch

from oracle import range_attention as OR
from tests.test_gpu_paged import cache, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new, lens, Hq", [([700, 1], [1500, 60], 8), ([70, 1, 33], [5000, 3000, 40], 4)], ids=str)
def test_a_timeout_behind_a_recorded_page(lib, new, lens, Hq):
    """A status block that holds what an earlier call recorded takes a wait that runs out all the same, parts that were never written are not
    added up, and what comes behind does nothing."""
    args = tuple(t.cuda() for t in (cache(new, lens, 16, Hq, 1, 128, "bf16", 83)[i] for i in (0, 3, 4, 5, 6, 7)))
    want = lib.mesh_paged_attention(*args, max(new))
    ws = lib.new_paged_workspace(args[0], args[1], args[3], max(new))
    for limit in (0, 1, 2_000, 20_000):
        st = torch.tensor([6, 1, 0, 0], dtype=torch.int32, device="cuda")
        O, L = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        lib.mesh_attn_set_wait_limit_ns(limit)
        try:
            lib.mesh_paged_attention(*args, max(new), O=O, LSE=L, workspace=ws, status=st, check_status=False)
            code = lib.mesh_attn_read_status(st)
        finally:
            lib.mesh_attn_set_wait_limit_ns(2_000_000_000)
        assert code in ((5,) if limit == 0 else (5, 6)), limit
        if limit == 0:
            assert (O == 7).all() and (L == 7).all()
        if code == 6:
            assert torch.equal(O, want[0]) and torch.equal(L, want[1])
            continue
        O.fill_(7.0)
        lib.mesh_paged_attention(*args, max(new), O=O, LSE=L, workspace=ws, status=st, check_status=False)
        assert lib.mesh_attn_read_status(st) == 5 and (O == 7).all()
    O, L = lib.mesh_paged_attention(*args, max(new), workspace=ws)
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, lens, page, window", [
    ([1, 1], [900, 131], 64, 100),         # few rows
    ([2, 1], [900, 131], 16, 7),
    ([40, 25], [1000, 500], 128, 301),     # chunks
    ([150, 30], [1000, 333], 48, 130),
    ([200, 1], [9000, 70], 256, 5001),     # in parts
], ids=str)
def test_what_lies_before_every_window_is_never_met(lib, new, lens, page, window, dtype):
    """NaN in the tokens before the first that any new token sees, up to the one beside it in its page."""
    q, _, _, kp, vp, table, off, ln = cache(new, lens, page, 4, 1, 64, dtype, 82)
    ref = OR.paged(q, kp, vp, table, off, ln, window=window)
    for b, (n, m) in enumerate(zip(new, lens)):
        for i in range(max(0, m - n + 1 - window)):
            for p in (kp, vp):
                p[int(table[b, i // page]), :, i % page] = math.nan
    O, L = lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), max(new), window=window)
    check(O, L, ref, dtype, max(new) <= 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, lens, bound, window", [
    ([3, 1, 2], [90, 33, 2], 2, 0),          # few rows
    ([3, 1, 2], [700, 33, 2], 1, 300),
    ([70, 1, 33], [300, 20, 40], 50, 0),     # chunks
    ([170, 1, 33], [5000, 20, 40], 130, 0),  # in parts
    ([170, 1, 33], [900, 20, 40], 40, 100),
], ids=str)
def test_more_new_tokens_than_the_bound(lib, new, lens, bound, window, dtype):
    """Recorded; the sequence's tokens up to the bound come out right, at the places that the append gives them, the others
    are left out."""
    q, _, _, kp, vp, table, off, ln = cache(new, lens, 16, 4, 2, 64, dtype, 80)
    ref = OR.paged(q, kp, vp, table, off, ln, window=window)
    O, L = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    st = lib.new_status()
    lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), bound, window=window, O=O, LSE=L, status=st,
                             check_status=False)
    assert lib.mesh_attn_read_status(st) == 6
    kept = torch.cat([torch.arange(n) < bound for n in new])
    check(O[kept.cuda()], L[kept.cuda()], tuple(x[kept] for x in ref), dtype, False)
    assert (O[~kept.cuda()] == 7).all() and (L[~kept.cuda()] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_new_tokens_than_the_table_holds(lib, dtype):
    """A length that the table just holds, of a sequence with more new tokens than that: recorded, as the append does, and the
    other sequence comes out right."""
    new = [40, 5]
    q, k, v, kp, vp, table, off, ln = cache(new, [32, 20], 16, 4, 2, 64, dtype, 81)
    st = lib.new_status()
    lib.mesh_paged_append(*(t.cuda() for t in (q, k, v, kp, vp, table, off, ln)), status=st, check_status=False)
    assert lib.mesh_attn_read_status(st) == 6
    st = lib.new_status()
    O, L = lib.mesh_paged_attention(*(t.cuda() for t in (q, kp, vp, table, off, ln)), 40, status=st, check_status=False)
    assert lib.mesh_attn_read_status(st) == 6
    one = torch.tensor([0, 5], dtype=torch.int32)
    check(O[40:], L[40:], OR.paged(q[40:], kp, vp, table[1:], one, ln[1:]), dtype, False)
