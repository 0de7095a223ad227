"""The library's older calls need ctypes alone: they load and build where the extension module of the rotary and
differential calls is missing or cannot be built, and only the calls that use it say so."""
import os
import shutil
import subprocess
import sys

import pytest

NAME = "tiled_distributed_attention_gb300"


def test_missing_module_stops_only_the_calls_that_use_it(lib, tmp_path):
    shutil.copytree(os.path.dirname(lib.__file__), tmp_path / NAME, ignore=shutil.ignore_patterns("_binding*", "__pycache__", "csrc"))
    code = f"""
import torch, {NAME} as m
m.load_library()
plan = m.mesh_attn_plan_create(64, 4, True)
assert plan.S == 64 and plan.n_slots > 0
assert m.mesh_attn_workspace_size_for(plan, torch.float32, 1, 2, 1, 64) > 0
assert m.mesh_attn_diff_workspace_size(plan, torch.float32, 1, 2, 1, 64) > 0
q, pos = torch.zeros(1, 1, 4, 64), torch.zeros(1, 4, dtype=torch.int64)
lam, st = torch.zeros(1), torch.zeros(4, dtype=torch.int32)
for call in (lambda: m.mesh_rope(q, None, pos, m.MeshRope(64, (32,))),
             lambda: m.mesh_diff_attention(q, q, q, lam, 1, True),
             lambda: m.mesh_attn_diff_fwd(plan, q, q, q, lam, None, q, None, q, q, st),
             lambda: m.mesh_diff_decode(q[:, :, :1], q, q, torch.ones(1, dtype=torch.int32), lam),
             lambda: m.mesh_attn_diff_decode(q[:, :, :1], q, q, torch.ones(1, dtype=torch.int32), lam, None, q, q, q, st)):
    try:
        call()
    except RuntimeError as e:
        assert "_binding.so is missing" in str(e), e
    else:
        raise AssertionError("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr


def test_library_is_built_where_the_module_cannot_be(monkeypatch, tmp_path):
    from tiled_distributed_attention_gb300 import _build

    def no_module():
        raise RuntimeError("g++ failed on binding.cpp")

    def link(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("library")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "_build_binding", no_module)
    monkeypatch.setattr(_build, "_compile", lambda src, extra: src)
    monkeypatch.setattr(_build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(_build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="binding.cpp"):  # loud all the same
        _build.build()
    assert (tmp_path / "lib.so").read_text() == "library"
