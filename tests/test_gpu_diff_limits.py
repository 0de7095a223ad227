"""Waits of the differential kernels that really run out: a short limit lets an ordinary wait (a load, a product, the other
warps) end without what it waited for.  The kernels then stop every role, drain their copies and products, free
their tensor memory and say so in the status block, and the next call in the same context gives the same bits.

The hardware's own wait inside one look at a barrier takes a microsecond or so, so a call of a few short blocks may get by
with any limit; these sizes have waits of tens of microseconds (a producer waits for a free stage, the last warps
for a whole unit).
"""
import pytest
import torch

from tests.test_gpu_diff import inputs

pytestmark = pytest.mark.gpu

NORMAL = 2_000_000_000
SHAPES = [(1, 2, 1, 2048, 64), (2, 8, 2, 2048, 128)]


def calls(lib, shape, dtype):
    """(forward, backward) of one set of inputs as functions of the status block, and their results without a limit."""
    q, k, v, lam, g = (t.cuda() for t in inputs(*shape, dtype, 70))
    plan = lib.mesh_attn_plan_create(shape[3], 1, True)
    ws = lib.new_diff_workspace(plan, q, k, backward=True)
    keep = dict(plan=plan, workspace=ws, check_status=False)
    saved = lib.mesh_diff_attention(q, k, v, lam, 1, True, plan=plan, return_saved=True)

    def forward(st):
        return lib.mesh_diff_attention(q, k, v, lam, 1, True, return_saved=True, status=st, **keep)

    def backward(st):
        return lib.mesh_diff_attention_backward(q, k, v, lam, *saved, g, 1, True, status=st, **keep)

    return ((forward, saved), (backward, backward(lib.new_status())))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_wait_that_runs_out(lib, shape, dtype):
    for call, want in calls(lib, shape, dtype):
        for limit in (1, 2_000, 8_000, 20_000):
            for _ in range(5):
                st = lib.new_status()
                lib.mesh_attn_set_wait_limit_ns(limit)
                try:
                    out = call(st)
                    code = lib.mesh_attn_read_status(st)
                finally:
                    lib.mesh_attn_set_wait_limit_ns(NORMAL)
                assert code in ((5,) if limit == 1 else (0, 5)), (limit, st.tolist())
                if code == 0:  # every wait got by
                    for a, b in zip(out, want):
                        assert torch.equal(a, b), limit
                else:
                    assert st[1].item() in (1, 2, 3, 5), st.tolist()  # a role of the kernel
        st = lib.new_status()
        out = call(st)
        assert lib.mesh_attn_read_status(st) == 0
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_behind_one_that_ran_out_do_nothing(lib, dtype):
    """Its status block keeps the error until the program clears it: the calls behind write nothing."""
    (forward, _), (_, grads) = calls(lib, SHAPES[0], dtype)
    q, k, v, lam, g = (t.cuda() for t in inputs(*SHAPES[0], dtype, 70))
    plan = lib.mesh_attn_plan_create(SHAPES[0][3], 1, True)
    O, O2, L = lib.mesh_diff_attention(q, k, v, lam, 1, True, plan=plan, return_saved=True)
    st, ws = lib.new_status(), lib.new_diff_workspace(plan, q, k, backward=True)
    lib.mesh_attn_set_wait_limit_ns(1)
    try:
        forward(st)
        assert lib.mesh_attn_read_status(st) == 5
    finally:
        lib.mesh_attn_set_wait_limit_ns(NORMAL)
    outs = [torch.full_like(t, 7.0) for t in (O, O2, L, q, k, v, lam)]
    lib.mesh_attn_diff_fwd(plan, q, k, v, lam, None, *outs[:3], ws, st)
    lib.mesh_attn_diff_bwd(plan, q, k, v, lam, O, O2, L, g, None, *outs[3:], ws, st)
    assert lib.mesh_attn_read_status(st) == 5
    for t in outs:
        assert (t == 7).all()
    st.zero_()
    lib.mesh_attn_diff_bwd(plan, q, k, v, lam, O, O2, L, g, None, *outs[3:], ws, st)
    assert lib.mesh_attn_read_status(st) == 0
    for a, b in zip(outs[3:], grads):
        assert torch.equal(a, b)


def test_a_limit_of_nothing_in_fp32(lib):
    """A limit of 0 is refused before anything starts, in both directions."""
    for call, want in calls(lib, (1, 2, 2, 300, 128), "f32"):
        lib.mesh_attn_set_wait_limit_ns(0)
        st = lib.new_status()
        try:
            call(st)
            code = lib.mesh_attn_read_status(st)
        finally:
            lib.mesh_attn_set_wait_limit_ns(NORMAL)
        if call.__name__ == "backward":  # the forward's kernel is the plain calls', which starts and lets its waits run out
            assert code == 5, st.tolist()
        else:
            assert code in (0, 5), st.tolist()
        st.zero_()
        out = call(st)
        assert lib.mesh_attn_read_status(st) == 0
        for a, b in zip(out, want):
            assert torch.equal(a, b)
