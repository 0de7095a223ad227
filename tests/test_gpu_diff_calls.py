"""Calls of differential attention that programs make beside the plain ones: captured with more units than SMs, two at once on
two streams."""
import pytest
import torch

from tests.test_gpu_diff import DT, inputs

pytestmark = pytest.mark.gpu


def setup(lib, shape, dtype, seed):
    bufs = [t.cuda() for t in inputs(*shape, dtype, seed)]
    plan = lib.mesh_attn_plan_create(shape[3], 1, True)
    plan.tables("cuda")
    return bufs, dict(plan=plan, workspace=lib.new_diff_workspace(plan, bufs[0], bufs[1], backward=True), status=lib.new_status(),
                      check_status=False)


def step(lib, bufs, keep):
    q, k, v, lam, g = bufs
    saved = lib.mesh_diff_attention(q, k, v, lam, 1, True, return_saved=True, **keep)
    return (*saved, *lib.mesh_diff_attention_backward(q, k, v, lam, *saved, g, 1, True, **keep))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 16, 4, 4096, 128), (3, 8, 2, 1000, 64)], ids=str)
def test_captured_with_more_units_than_sms(lib, shape, dtype):
    """The work counters are set to zero inside the graph: every replay takes all units again."""
    bufs, keep = setup(lib, shape, dtype, 71)
    new = [t.cuda() for t in inputs(*shape, dtype, 72)]
    want = [t.clone() for t in step(lib, new, keep)]
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = step(lib, bufs, keep)
    for b, x in zip(bufs, new):
        b.copy_(x)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert lib.mesh_attn_read_status(keep["status"]) == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_at_once_on_two_streams(lib, dtype):
    """Calls that overlap on the GPU, each with a workspace and a status block of its own."""
    shape = (1, 8, 2, 1500, 128)
    sets = [setup(lib, shape, dtype, 73 + i) for i in range(2)]
    want = [[t.clone() for t in step(lib, *s)] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(stream):
                got[i].append(step(lib, *s))
    torch.cuda.synchronize()
    for i, (_, keep) in enumerate(sets):
        assert lib.mesh_attn_read_status(keep["status"]) == 0
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)
    assert DT[dtype] == got[0][0][0].dtype
