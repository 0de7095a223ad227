"""The autograd call of differential attention records failures of both directions in the caller's status block."""
import pytest
import torch

from tests.test_gpu_diff import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_failures_are_recorded(lib, dtype):
    q, k, v, lam, g = (t.cuda().requires_grad_(i < 4) for i, t in enumerate(inputs(1, 2, 1, 64, 64, dtype, 75)))
    plan, other = lib.mesh_attn_plan_create(64, 1, True), lib.mesh_attn_plan_create(64, 1, False)
    st, dev = lib.new_status(), torch.cuda.current_device()
    keep = dict(plan=plan, check_status=False, status=st)
    O, _ = lib.mesh_diff_attention_autograd(q, k, v, lam, 1, True, **keep)
    assert lib.mesh_attn_read_status(st) == 0
    good = plan.tables("cuda")
    plan._tables[dev] = other.tables("cuda")  # another plan's: the device refuses them
    O.backward(g)
    assert lib.mesh_attn_read_status(st) == 1  # of the backward call
    st.zero_()
    lib.mesh_diff_attention_autograd(q, k, v, lam, 1, True, **keep)
    assert lib.mesh_attn_read_status(st) == 1  # of the forward call
    st.zero_()
    plan._tables[dev] = good
    # with the check on, a failure raises in either direction, and a block that is clear does not
    O, _ = lib.mesh_diff_attention_autograd(q, k, v, lam, 1, True, plan=plan, status=st)
    plan._tables[dev] = other.tables("cuda")
    with pytest.raises(lib.MeshAttnError):
        O.backward(g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_gradients_with_a_status_block(lib, dtype):
    args = [t.cuda() for t in inputs(1, 2, 1, 130, 64, dtype, 76)]
    got = []
    for keep in ({}, dict(status=lib.new_status(), check_status=False)):
        leaves = [t.clone().requires_grad_(True) for t in args[:4]]
        O, _ = lib.mesh_diff_attention_autograd(*leaves, 1, True, **keep)
        O.backward(args[4])
        got.append([t.grad for t in leaves])
    for a, b in zip(*got):
        assert torch.equal(a, b)
