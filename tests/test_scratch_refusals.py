"""Workspaces and status blocks that are smaller than they say are refused before anything is enqueued (on the CPU)."""
import pytest
import torch


def scratch():
    ws, st = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(4, dtype=torch.int32)
    return [(ws, st[:1], "status"), (ws, torch.zeros(0, dtype=torch.int32), "status"), (ws, st.to(torch.int16), "status"),
            (ws, st.long(), "status"), (ws, st[:1].expand(4), "status"), (ws, torch.zeros(8, dtype=torch.int32)[::2], "status"),
            (ws[:1].expand(1 << 30), st, "workspace"), (ws[::2], st, "workspace")]


@pytest.mark.parametrize("i", range(8))
def test_scratch(lib, i):
    ws, st, what = scratch()[i]
    q, k, lam = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64), torch.zeros(4)
    L, plan = torch.zeros(1, 4, 2, 8), lib.mesh_attn_plan_create(8, 1, True)
    one = torch.zeros(1, 4, 1, 64)
    calls = [lambda: lib.mesh_attn_diff_fwd(plan, q, k, k, lam, None, q, None, L, ws, st),
             lambda: lib.mesh_attn_diff_bwd(plan, q, k, k, lam, q, q, L, q, None, q, k, k, lam, ws, st),
             lambda: lib.mesh_attn_diff_decode(one, k, k, torch.ones(1, dtype=torch.int32), lam, None, one, L[..., :1].contiguous(),
                                               ws, st)]
    for call in calls:
        with pytest.raises(ValueError, match=what):
            call()
