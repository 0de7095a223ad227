"""What the paged-cache and range-masked calls refuse, on the CPU: every check runs before anything is enqueued."""
import ctypes
import math
import os
import re

import pytest
import torch

import tiled_distributed_attention_gb300 as m

P = 0x10000  # a pointer's value: never read by a host check


def ptr(x):
    return ctypes.c_void_p(x)


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def append(lib, **kw):
    a = dict(dtype=1, N=5, B=2, Hq=4, Hkv=2, d=64, q=P, qs=i64(512, 64), qo=P, qos=i64(256, 64), k=P, ks=i64(512, 64), v=P, vs=i64(512, 64),
             n_pages=7, page=8, kp=P, kps=i64(1024, 512, 64), vp=P, vps=i64(1024, 512, 64), table=P, max_pages=3, ts=3, off=P, lens=P,
             groups=1, n=32, axes=1, freq=[1.0] * 32, axis=[0] * 32, adj=0, pos=None, bits=64, ps=i64(0, 1), st=P)
    a.update(kw)
    f = None if a["freq"] is None else (ctypes.c_double * 300)(*a["freq"])
    x = None if a["axis"] is None else (ctypes.c_int32 * 300)(*a["axis"])
    return lib._lib.mesh_attn_paged_append(
        a["dtype"], a["N"], a["B"], a["Hq"], a["Hkv"], a["d"], ptr(a["q"]), a["qs"], ptr(a["qo"]), a["qos"], ptr(a["k"]), a["ks"],
        ptr(a["v"]), a["vs"], a["n_pages"], a["page"], ptr(a["kp"]), a["kps"], ptr(a["vp"]), a["vps"], ptr(a["table"]), a["max_pages"],
        a["ts"], ptr(a["off"]), ptr(a["lens"]), a["groups"], a["n"], a["axes"], f, x, a["adj"], ptr(a["pos"]), a["bits"], a["ps"],
        ptr(a["st"]), None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), 1), (dict(N=-1), 1), (dict(B=-1), 1), (dict(Hq=-1), 1), (dict(Hkv=0), 1), (dict(n_pages=-1), 1), (dict(page=0), 1),
    (dict(max_pages=-1), 1), (dict(N=1 << 31), 2), (dict(d=0), 1), (dict(d=1026), 1), (dict(groups=0), 1), (dict(groups=3), 1),
    (dict(n=33), 1), (dict(n=-1), 1), (dict(axes=0), 1), (dict(axes=9), 1), (dict(adj=2), 1), (dict(freq=None), 1), (dict(axis=None), 1),
    (dict(freq=[math.nan] * 32), 1), (dict(axis=[1] * 32), 1), (dict(axes=2), 1), (dict(pos=P, bits=16), 1), (dict(pos=P, ps=None), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(qs=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(kps=None), 1), (dict(table=None), 1), (dict(off=None), 1), (dict(lens=None), 1), (dict(st=None), 1),
    (dict(kps=i64(0, 512, 64)), 1), (dict(vps=i64(1024, 0, 64)), 1), (dict(qos=i64(0, 64)), 1), (dict(q=P + 1), 3), (dict(vp=P + 1), 3),
    (dict(table=P + 2), 3), (dict(off=P + 1), 3), (dict(st=P + 2), 3), (dict(pos=P + 4), 3), (dict(N=0, k=None), 0), (dict(B=0, k=None), 0),
], ids=str)
def test_append(lib, kw, code):
    assert append(lib, **kw) == code
    assert bool(lib._lib.mesh_attn_last_error()) == (code != 0)


def attend(lib, **kw):
    a = dict(dtype=1, N=5, B=2, Hq=4, Hkv=2, d=64, q=P, qs=i64(256, 64), n_pages=7, page=16, kp=P, ks=i64(2048, 1024, 64), vp=P,
             vs=i64(2048, 1024, 64), table=P, max_pages=3, ts=3, off=P, lens=P, max_new=4, scale=0.1, cap=0.0, slopes=None, window=0, O=P,
             L=P, ws=P, n=1 << 40, st=P)
    a.update(kw)
    return lib._lib.mesh_attn_paged_attn(
        a["dtype"], a["N"], a["B"], a["Hq"], a["Hkv"], a["d"], ptr(a["q"]), a["qs"], a["n_pages"], a["page"], ptr(a["kp"]), a["ks"],
        ptr(a["vp"]), a["vs"], ptr(a["table"]), a["max_pages"], a["ts"], ptr(a["off"]), ptr(a["lens"]), a["max_new"], a["scale"], a["cap"],
        ptr(a["slopes"]), a["window"], ptr(a["O"]), ptr(a["L"]), ptr(a["ws"]), a["n"], ptr(a["st"]), None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=4), 1), (dict(N=-1), 1), (dict(B=-1), 1), (dict(Hq=-4), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(d=96), 2),
    (dict(page=0), 2), (dict(page=24), 2), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1), (dict(B=4097), 2), (dict(max_pages=1 << 27), 2),
    (dict(N=(1 << 24) + 1), 2), (dict(N=1 << 24, Hq=128), 2), (dict(Hq=65536, Hkv=1), 2), (dict(scale=0.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(cap=-1.0), 1), (dict(cap=math.nan), 1), (dict(cap=math.inf), 1), (dict(cap=1e-30), 2),
    (dict(window=-1), 1), (dict(max_new=0), 1), (dict(max_new=-3), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(q=None), 1),
    (dict(kp=None), 1), (dict(vs=None), 1), (dict(table=None), 1), (dict(off=None), 1), (dict(lens=None), 1), (dict(O=None), 1),
    (dict(L=None), 1), (dict(ws=None), 1), (dict(st=None), 1), (dict(q=P + 8), 3), (dict(kp=P + 2), 3), (dict(O=P + 8), 3),
    (dict(ws=P + 4), 3), (dict(slopes=P + 2), 3), (dict(off=P + 1), 3), (dict(qs=i64(260, 64)), 3), (dict(qs=i64(256, 0)), 3),
    (dict(ks=i64(2048, 1024, 68)), 3), (dict(vs=i64(-2048, 1024, 64)), 3), (dict(n=1000), 9), (dict(N=0, q=None), 0), (dict(B=0, q=None), 0),
    (dict(Hq=0, q=None), 0)], ids=str)
def test_attention_over_pages(lib, kw, code):
    assert attend(lib, **kw) == code


RANGE = [
    (dict(dtype=3), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(Hq=-2), 1), (dict(Hkv=0), 1), (dict(Hq=3), 1), (dict(d=32), 2),
    (dict(S=(1 << 24) + 1), 2), (dict(B=65536), 2), (dict(B=64, S=1 << 24), 2), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(cap=-2.0), 1), (dict(cap=math.inf), 1), (dict(q=None), 1), (dict(v=None), 1), (dict(lo=None), 1), (dict(hi=None), 1),
    (dict(O=None), 1), (dict(L=None), 1), (dict(ws=None), 1), (dict(st=None), 1), (dict(ms=3), 1), (dict(q=P + 8), 3), (dict(O=P + 2), 3),
    (dict(lo=P + 1), 3), (dict(slopes=P + 2), 3), (dict(ws=P + 8), 3), (dict(n=8), 9), (dict(B=0, q=None), 0), (dict(S=0, q=None), 0),
    (dict(Hq=0, q=None), 0)]


def range_call(lib, back, **kw):
    a = dict(dtype=1, B=2, Hq=4, Hkv=2, S=40, d=64, q=P, k=P, v=P, lo=P, hi=P, ms=40, slopes=None, O=P, L=P, g=P, scale=0.1, cap=0.0, dq=P,
             dk=P, dv=P, ws=P, n=1 << 40, st=P)
    a.update(kw)
    head = (a["dtype"], a["B"], a["Hq"], a["Hkv"], a["S"], a["d"], ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["lo"]), ptr(a["hi"]),
            a["ms"], ptr(a["slopes"]))
    tail = (ptr(a["ws"]), a["n"], ptr(a["st"]), None)
    if back:
        return lib._lib.mesh_attn_range_bwd(*head, ptr(a["O"]), ptr(a["L"]), ptr(a["g"]), a["scale"], a["cap"], ptr(a["dq"]), ptr(a["dk"]),
                                            ptr(a["dv"]), *tail)
    return lib._lib.mesh_attn_range_fwd(*head, a["scale"], a["cap"], ptr(a["O"]), ptr(a["L"]), *tail)


@pytest.mark.parametrize("kw, code", RANGE, ids=str)
def test_range_forward(lib, kw, code):
    assert range_call(lib, False, **kw) == code


@pytest.mark.parametrize("kw, code", RANGE + [(dict(g=None), 1), (dict(dq=None), 1), (dict(dv=None), 1), (dict(g=P + 8), 3),
                                              (dict(dk=P + 4), 3)], ids=str)
def test_range_backward(lib, kw, code):
    assert range_call(lib, True, **kw) == code


def test_sizes(lib):
    n = ctypes.c_size_t()
    f = lib._lib.mesh_attn_paged_workspace_size
    assert f(1, 64, 64, 32, 8, 128, 1, ctypes.byref(n)) == 0
    step = n.value
    assert f(1, 4096, 64, 32, 8, 128, 512, ctypes.byref(n)) == 0 and n.value >= step
    big = n.value  # enough for any smaller batch too, whatever its parts
    for N, B in ((1, 1), (7, 3), (100, 64), (2048, 8), (4096, 64)):
        assert f(1, N, B, 32, 8, 128, min(N, 512), ctypes.byref(n)) == 0 and n.value <= big
    assert f(1, 1, 1, 4, 2, 128, 1, None) == 1 and f(1, 1, 1, 4, 3, 128, 1, ctypes.byref(n)) == 1 and f(0, 1, 1, 4, 2, 80, 1, ctypes.byref(n)) == 2
    g = lib._lib.mesh_attn_range_workspace_size
    for dt in (0, 1):
        assert g(dt, 1, 4, 2, 300, 128, 0, ctypes.byref(n)) == 0
        fwd = n.value
        assert g(dt, 1, 4, 2, 300, 128, 1, ctypes.byref(n)) == 0 and n.value >= fwd > 0
    assert g(1, 1, 4, 2, 300, 128, 2, ctypes.byref(n)) == 1 and g(1, 1, 4, 2, 300, 128, 0, None) == 1
    assert g(1, 0, 4, 2, 0, 128, 1, ctypes.byref(n)) == 0


def pages(n=4, Hkv=2, page=16, d=64, dtype=torch.float32):
    return torch.zeros(n, Hkv, page, d, dtype=dtype)


def test_tensors_of_the_cache(lib):
    k, v = torch.zeros(5, 2, 64), torch.zeros(5, 2, 64)
    q, kp, vp = torch.zeros(5, 4, 64), pages(), pages()
    table, off, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    st, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    good = [q, k, v, kp, vp, table, off, lens]
    rope = lib.MeshRope(64, (32,))
    for i, bad in ((0, q[:4]), (0, q.bfloat16()), (0, q[:, :, :32]), (1, k[:, :1]), (1, k[0]), (1, k.transpose(1, 2)), (2, v[:3]),
                   (2, v.double()), (3, kp[0]), (3, kp.double()), (4, vp[:2]), (4, vp.bfloat16()), (5, table.long()), (5, table[0]),
                   (5, table.T), (6, off[:2]), (6, off.long()), (7, lens[:1]), (7, lens.float())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            lib.mesh_paged_append(*args, rope=rope, status=st)
    for kw in (dict(rope=lib.MeshRope(128, (32,))), dict(positions=torch.zeros(5, dtype=torch.int32)),
               dict(rope=rope, positions=torch.zeros(4, dtype=torch.int32)), dict(rope=rope, positions=torch.zeros(5)),
               dict(rope=rope, positions=torch.zeros(2, 5, dtype=torch.int32)), dict(rope=rope, q_out=q[:2]), dict(rope=rope, status=st[:1]),
               dict(rope=rope)):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            lib.mesh_paged_append(*good, **{"status": st, **kw})
    with pytest.raises(ValueError):
        lib.mesh_paged_append(None, *good[1:], q_out=q, status=st)
    good = [q, kp, vp, table, off, lens]
    for i, bad in ((0, q[:, :3]), (0, q[0]), (0, q.bfloat16()), (0, q.double()), (1, pages(Hkv=3)), (2, vp[:1]), (3, table.long()), (4, off[:2]),
                   (5, lens.long())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            lib.mesh_paged_attention(*args, 1, workspace=ws, status=st)
    for kw in (dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4).double()), dict(O=q[:2]), dict(O=q.bfloat16()), dict(LSE=torch.zeros(5)),
               dict(status=st[:2]), dict(workspace=ws[::2]), dict()):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            lib.mesh_paged_attention(*good, 1, **{"workspace": ws, "status": st, **kw})


def test_tensors_of_ranges(lib):
    q, k = torch.zeros(2, 4, 9, 64), torch.zeros(2, 2, 9, 64)
    lo, hi = torch.zeros(2, 9, dtype=torch.int32), torch.zeros(2, 9, dtype=torch.int32)
    L, st, ws = torch.zeros(2, 4, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    good = [q, k, k, lo, hi]
    for i, bad in ((0, q[0]), (0, q[:, :3]), (0, q[:, :, :8]), (0, q.transpose(1, 2)), (0, q.bfloat16()), (1, k[:, :1]), (2, k[:1]), (3, lo[:, :8]),
                   (3, lo.long()), (3, lo[0]), (4, hi.T), (4, hi.float())):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            lib.mesh_range_attention(*args, workspace=ws, status=st)
        with pytest.raises(ValueError):
            lib.mesh_range_attention(*args)
        with pytest.raises(ValueError):
            lib.mesh_range_attention_backward(*args, q, L, q, workspace=ws, status=st)
    for kw in (dict(slopes=torch.zeros(3)), dict(O=q[:1]), dict(LSE=L[:1]), dict(status=st[:1]), dict(workspace=ws[::2]), dict()):
        with pytest.raises(ValueError):
            lib.mesh_range_attention(*good, **{"workspace": ws, "status": st, **kw})
    for o, l, g in ((q[:1], L, q), (q, L[:1], q), (q, L, q.bfloat16()), (q, L.double(), q)):
        with pytest.raises(ValueError):
            lib.mesh_range_attention_backward(*good, o, l, g, workspace=ws, status=st)
    with pytest.raises(ValueError):
        lib.mesh_range_attention_backward(*good, q, L, q, dK=q, workspace=ws, status=st)


# ------------------------------------------------------------------ what the sources promise, also those that are headers

CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")
HEADERS = ["score_fwd.cuh", "score_bwd.cuh"]


def code_of(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", HEADERS + ["paged_append.cu", "paged_rows.cu", "score_simt.cu"])
def test_results_of_an_overlapped_predecessor_are_read_by_plain_loads(name):
    code = code_of(name)
    assert "wait_for_kernel_before()" in code
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code)
    for kernel in re.findall(r"__global__[^{;]*\{.*?\n\}", code, flags=re.S):
        if "run_pass" not in kernel:  # whose passes wait themselves
            assert "wait_for_kernel_before()" in kernel


@pytest.mark.parametrize("name", HEADERS)
def test_register_splits_are_checked(name):
    src = open(os.path.join(CSRC, name)).read()
    used = set(re.findall(r"regs_(?:inc|dec)<(\w+)>", src))
    check = re.search(r"fa\.numRegs \* NUM_THREADS < ([^)]*)\)", src)
    assert used and check and all(n in check.group(1) for n in used)
    value = {n: int(v) for n, v in re.findall(r"(\w+_REGS) = (\d+)", src)}
    threads = int(re.search(r"NUM_THREADS = (\d+);", src).group(1))
    assert eval(check.group(1), {}, value) <= threads * {384: 168, 512: 128}[threads]
