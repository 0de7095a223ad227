"""Plain attention whose partitions are no multiple of a tile: tiles then reach past a partition's end, where the next
partition, head or batch begins.  NaN and infinities there never reach a result."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
L, P = 100, 4


def inputs(dtype, d):
    g = torch.Generator().manual_seed(80)
    return [torch.randn(2, 2, L * P, d, generator=g).to(DT[dtype]) for _ in range(4)]


def run(lib, plan, q, k, v, g, causal):
    q, k, v, g = (t.cuda() for t in (q, k, v, g))
    O, LSE = lib.mesh_attention(q, k, v, P, causal, plan=plan)
    return [O, LSE, *lib.mesh_attention_backward(q, k, v, O, LSE, g, P, causal, plan=plan)]


def plan_of(lib, kind, causal):
    return lib.mesh_attn_plan_create_ring(L * P, P, causal) if kind == "ring" else lib.mesh_attn_plan_create(L * P, P, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["mesh", "ring"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_heads_and_batches(lib, dtype, d, kind, causal):
    clean = inputs(dtype, d)
    bad = [t.clone() for t in clean]
    for t in bad:
        t[1] = float("nan")
        t[0, 1] = float("inf")
    plan = plan_of(lib, kind, causal)
    for name, a, b in zip(("O", "LSE", "dQ", "dK", "dV"), run(lib, plan, *clean, causal), run(lib, plan, *bad, causal)):
        assert torch.isfinite(a).all() and torch.equal(a[0, 0], b[0, 0]), name


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("kind", ["mesh", "ring"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_partitions_behind_the_mask(lib, dtype, kind, value):
    """Keys of later partitions, which the first partition's rows do not see."""
    clean = inputs(dtype, 128)
    bad = [t.clone() for t in clean]
    for t in bad[1:3]:
        t[:, :, L:] = value
    plan = plan_of(lib, kind, True)
    a, b = run(lib, plan, *clean, True), run(lib, plan, *bad, True)
    for i, name in ((0, "O"), (1, "LSE"), (2, "dQ")):
        assert torch.equal(a[i][:, :, :L], b[i][:, :, :L]), name
