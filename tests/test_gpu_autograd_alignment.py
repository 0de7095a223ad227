"""Gradients that reach the autograd calls as PyTorch hands them on: contiguous, but not on a 16-byte boundary."""
import pytest
import torch

from tests.test_gpu_range import inputs, mask_of

pytestmark = pytest.mark.gpu


def calls(lib, q, lo, hi):
    lam = torch.rand(4, device="cuda").to(q.dtype)
    return {
        "plain": lambda a, b, c: lib.mesh_attention_autograd(a, b, c, 1, True)[0],
        "differential": lambda a, b, c: lib.mesh_diff_attention_autograd(a, b, c, lam, 1, True)[0],
        "range": lambda a, b, c: lib.mesh_range_attention_autograd(a, b, c, lo, hi)[0],
    }


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["plain", "differential", "range"])
def test_a_gradient_behind_an_odd_offset(lib, name, dtype):
    """An output joined behind three numbers of another tensor: its gradient begins 3 elements into the joined one's."""
    q, k, v, _ = (t.cuda() for t in inputs(1, 4, 2, 128, 64, dtype, 90))
    lo, hi = (t.cuda() for t in mask_of("causal", 1, 128))
    call = calls(lib, q, lo, hi)[name]
    got, want = [], []
    for grads, joined in ((got, True), (want, False)):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        O = call(*leaves)
        w = torch.randn(O.numel(), generator=torch.Generator().manual_seed(1)).to(O.dtype).cuda()
        if joined:
            y = torch.cat([torch.zeros(3, dtype=O.dtype, device="cuda"), O.flatten()])
            y.backward(torch.cat([torch.ones(3, dtype=O.dtype, device="cuda"), w]))
        else:
            O.backward(w.view_as(O))
        grads.extend(x.grad for x in leaves)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
