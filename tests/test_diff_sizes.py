"""Which sizes the fp32 differential calls take: only the number of rows bounds them (checked on the host)."""
import pytest
import torch


@pytest.mark.parametrize("B, Hq, Hkv, S, ok", [
    (10000, 2, 1, 16, True), (1, 66000, 33000, 3, True), (8191, 1, 1, 1, True), (8192, 1, 1, 1, True),
    (1, 1, 1, 357913941, True), (1, 1, 1, 357913942, False), (357913942, 1, 1, 1, False)])  # 6 B Hq S around 2^31
def test_fp32_sizes(lib, B, Hq, Hkv, S, ok):
    plan = lib.mesh_attn_plan_create(S, 1, True)
    if ok:
        assert lib.mesh_attn_diff_workspace_size(plan, torch.float32, B, Hq, Hkv, 64, True) > 0
    else:
        with pytest.raises(lib.MeshAttnError) as e:
            lib.mesh_attn_diff_workspace_size(plan, torch.float32, B, Hq, Hkv, 64, True)
        assert e.value.code == 2
