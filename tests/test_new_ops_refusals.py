"""What the rotary, differential and decode calls refuse, on the CPU: every check runs before anything
is enqueued, so the C entry points answer with their status codes without a GPU."""
import ctypes
import math

import pytest
import torch

P = 0x10000  # a pointer's value: never read by a host check


def ptr(x):
    return ctypes.c_void_p(x)


def s3(*x):
    return (ctypes.c_int64 * 3)(*x)


def rope_call(lib, **kw):
    a = dict(dtype=1, B=1, S=4, d=64, Hq=2, q=P, qs=s3(512, 256, 64), qo=P, qos=s3(512, 256, 64), Hk=0, k=None, ks=None,
             ko=None, kos=None, groups=1, n=32, axes=1, freq=[1.0] * 32, axis=[0] * 32, adj=0, inv=0, pos=P, bits=64,
             ps=s3(0, 0, 1))
    a.update(kw)
    f = None if a["freq"] is None else (ctypes.c_double * 300)(*a["freq"])
    x = None if a["axis"] is None else (ctypes.c_int32 * 300)(*a["axis"])
    return lib._lib.mesh_attn_rope(a["dtype"], a["B"], a["S"], a["d"], a["Hq"], ptr(a["q"]), a["qs"], ptr(a["qo"]), a["qos"],
                                   a["Hk"], ptr(a["k"]), a["ks"], ptr(a["ko"]), a["kos"], a["groups"], a["n"], a["axes"], f,
                                   x, a["adj"], a["inv"], ptr(a["pos"]), a["bits"], a["ps"], None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(Hq=-1), 1), (dict(Hk=-2), 1), (dict(groups=0), 1), (dict(d=0), 1),
    (dict(d=1026), 1), (dict(groups=3), 1), (dict(n=0), 1), (dict(n=33), 1), (dict(groups=2, n=17), 1), (dict(axes=0), 1),
    (dict(axes=9), 1), (dict(bits=16), 1), (dict(adj=2), 1), (dict(inv=-1), 1), (dict(freq=None), 1), (dict(axis=None), 1),
    (dict(freq=[math.nan] * 32), 1), (dict(freq=[math.inf] * 32), 1), (dict(axis=[1] * 32), 1), (dict(axis=[-1] * 32), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(qs=None), 1), (dict(qos=None), 1), (dict(pos=None), 1), (dict(ps=None), 1),
    (dict(Hk=1), 1), (dict(qos=s3(512, 0, 64)), 1), (dict(q=P + 1), 3), (dict(qo=P + 1), 3), (dict(pos=P + 4), 3),
    (dict(B=0, q=None, pos=None), 0), (dict(S=0, q=None, pos=None), 0), (dict(Hq=0, q=None, pos=None), 0),
], ids=str)
def test_rope(lib, kw, code):
    assert rope_call(lib, **kw) == code
    assert bool(lib._lib.mesh_attn_last_error()) == (code != 0)


def test_rope_handle_and_tensors(lib):
    for bad in (dict(sections=()), dict(sections=(0,)), dict(sections=(-1, 2)), dict(sections=(33,)), dict(sections=(17,), groups=2),
                dict(sections=(4,), groups=0), dict(sections=(4,), groups=3), dict(sections=(4,), style="x"),
                dict(sections=(4,), freq="x"), dict(sections=(4,), freq=[1.0]), dict(sections=(4,), base=0.0),
                dict(sections=(2, 2), axis_of_pair=[0, 1, 2, 0]), dict(sections=(2, 2), axis_of_pair=[0])):
        with pytest.raises(ValueError):
            lib.MeshRope(64, **bad)
    r = lib.MeshRope(64, (16, 16))
    q, pos = torch.zeros(1, 2, 4, 64), torch.zeros(2, 1, 4, dtype=torch.int64)
    for args in ((torch.zeros(2, 4, 64), None, pos), (torch.zeros(1, 2, 4, 32), None, pos), (q, torch.zeros(1, 2, 5, 64), pos),
                 (q, q.double(), pos), (q, None, pos[:1]), (q, None, pos.float()), (q, None, torch.zeros(2, 3, 4, dtype=torch.int64)),
                 (q, None, pos)):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            lib.mesh_rope(*args, r)
    # the ladders
    assert r.freq[0] == 1.0 and r.freq[16] == pytest.approx(10000.0 ** -0.5)
    ax = lib.MeshRope(64, (16, 8), freq="axial")
    assert ax.freq[16] == 1.0 and ax.freq[17] == pytest.approx(10000.0 ** (-1 / 8)) and ax.axis[15:17] == (0, 1)


def diff_fwd(lib, plan, **kw):
    a = dict(tables=P, dtype=1, B=1, Hq=2, Hkv=1, d=64, q=P, k=P, v=P, lam=P, lam_n=2, scale=0.1, O=P, O2=None, L=P, ws=P,
             n=1 << 40, st=P)
    a.update(kw)
    return lib._lib.mesh_attn_diff_fwd(plan, ptr(a["tables"]), a["dtype"], a["B"], a["Hq"], a["Hkv"], a["d"], ptr(a["q"]),
                                       ptr(a["k"]), ptr(a["v"]), ptr(a["lam"]), a["lam_n"], a["scale"], ptr(a["O"]), ptr(a["O2"]),
                                       ptr(a["L"]), ptr(a["ws"]), a["n"], ptr(a["st"]), None)


DIFF_BAD = [
    (dict(dtype=3), 1), (dict(B=-1), 1), (dict(Hq=-2), 1), (dict(Hkv=0), 1), (dict(Hq=3, Hkv=2), 1), (dict(d=96), 2),
    (dict(B=1 << 20, Hq=16, Hkv=1), 2), (dict(lam_n=0), 1), (dict(lam_n=3), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(tables=None), 1), (dict(q=None), 1), (dict(lam=None), 1), (dict(O=None), 1), (dict(L=None), 1),
    (dict(ws=None), 1), (dict(st=None), 1), (dict(q=P + 8), 3), (dict(tables=P + 4), 3), (dict(O=P + 2), 3), (dict(ws=P + 8), 3),
    (dict(lam=P + 1), 3), (dict(L=P + 2), 3), (dict(n=100), 9), (dict(B=0, q=None), 0), (dict(Hq=0, q=None), 0),
]


@pytest.mark.parametrize("kw, code", DIFF_BAD, ids=str)
def test_diff_forward(lib, kw, code):
    plan = lib.mesh_attn_plan_create(256, 4, True)
    assert diff_fwd(lib, plan.handle, **kw) == code
    assert diff_fwd(lib, None) == 1
    assert diff_fwd(lib, lib.mesh_attn_plan_create(0, 1, True).handle, q=None) == 0


def diff_bwd(lib, plan, **kw):
    a = dict(tables=P, dtype=1, B=1, Hq=2, Hkv=1, d=64, q=P, k=P, v=P, lam=P, lam_n=2, scale=0.1, O=P, O2=P, L=P, g=P, dq=P, dk=P,
             dv=P, dl=P, ws=P, n=1 << 40, st=P)
    a.update(kw)
    return lib._lib.mesh_attn_diff_bwd(plan, ptr(a["tables"]), a["dtype"], a["B"], a["Hq"], a["Hkv"], a["d"], ptr(a["q"]),
                                       ptr(a["k"]), ptr(a["v"]), ptr(a["lam"]), a["lam_n"], ptr(a["O"]), ptr(a["O2"]), ptr(a["L"]),
                                       ptr(a["g"]), a["scale"], ptr(a["dq"]), ptr(a["dk"]), ptr(a["dv"]), ptr(a["dl"]), ptr(a["ws"]),
                                       a["n"], ptr(a["st"]), None)


@pytest.mark.parametrize("kw, code", DIFF_BAD + [
    (dict(O2=None), 1), (dict(g=None), 1), (dict(dq=None), 1), (dict(dl=None), 1), (dict(g=P + 8), 3), (dict(dv=P + 8), 3),
    (dict(dl=P + 1), 3)], ids=str)
def test_diff_backward(lib, kw, code):
    plan = lib.mesh_attn_plan_create(256, 4, True)
    assert diff_bwd(lib, plan.handle, **kw) == code


def decode(lib, **kw):
    a = dict(dtype=1, B=2, Hq=4, Hkv=2, d=128, T=100, q=P, k=P, ks=s3(25600, 12800, 128), v=P, vs=s3(25600, 12800, 128), lens=P,
             lam=P, lam_n=4, scale=0.1, O=P, L=P, ws=P, n=1 << 40, st=P)
    a.update(kw)
    return lib._lib.mesh_attn_diff_decode(a["dtype"], a["B"], a["Hq"], a["Hkv"], a["d"], a["T"], ptr(a["q"]), ptr(a["k"]), a["ks"],
                                          ptr(a["v"]), a["vs"], ptr(a["lens"]), ptr(a["lam"]), a["lam_n"], a["scale"], ptr(a["O"]),
                                          ptr(a["L"]), ptr(a["ws"]), a["n"], ptr(a["st"]), None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=5), 1), (dict(B=-1), 1), (dict(Hq=-4), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(d=96), 2),
    (dict(B=4097), 2), (dict(T=(1 << 30) + 1), 2), (dict(lam_n=2), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(lens=None), 1), (dict(lam=None), 1),
    (dict(O=None), 1), (dict(L=None), 1), (dict(ws=None), 1), (dict(st=None), 1), (dict(q=P + 8), 3), (dict(k=P + 2), 3),
    (dict(ks=s3(25600, 12800, 132)), 3), (dict(vs=s3(25601, 12800, 128)), 3), (dict(lens=P + 2), 3), (dict(lam=P + 1), 3),
    (dict(B=0, q=None), 0), (dict(Hq=0, lam_n=1, q=None), 0)], ids=str)
def test_decode(lib, kw, code):
    assert decode(lib, **kw) == code


def test_sizes(lib):
    n = ctypes.c_size_t()
    f = lib._lib.mesh_attn_diff_decode_workspace_size
    assert f(2, 4, 2, 128, 100, ctypes.byref(n)) == 0 and n.value > 0
    small = n.value
    assert f(64, 32, 2, 128, 10**6, ctypes.byref(n)) == 0 and n.value > small
    assert f(2, 4, 2, 128, 100, None) == 1 and f(2, 4, 3, 128, 100, ctypes.byref(n)) == 1 and f(2, 4, 2, 80, 100, ctypes.byref(n)) == 2
    plan = lib.mesh_attn_plan_create(300, 4, True)
    fwd = lib.mesh_attn_diff_workspace_size(plan, torch.bfloat16, 1, 4, 2, 128)
    both = lib.mesh_attn_diff_workspace_size(plan, torch.bfloat16, 1, 4, 2, 128, True)
    assert 0 < fwd <= both
    g = lib._lib.mesh_attn_diff_workspace_size
    assert g(plan.handle, 1, 1, 4, 2, 128, 2, ctypes.byref(n)) == 1 and g(None, 1, 1, 4, 2, 128, 0, ctypes.byref(n)) == 1
    t = lib._lib.mesh_attn_plan_tables_size
    assert t(plan.handle, ctypes.byref(n)) == 0 and t(None, ctypes.byref(n)) == 1
    buf = (ctypes.c_uint8 * n.value)()
    w = lib._lib.mesh_attn_plan_tables_write
    assert w(plan.handle, buf, n.value) == 0 and w(plan.handle, buf, n.value - 1) == 9 and w(plan.handle, None, n.value) == 1


def test_diff_tensors(lib):
    q, k, lam = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64), torch.zeros(4)
    for a in ((q[0], k, k, lam), (q, k, k[:, :1], lam), (q, torch.zeros(1, 3, 8, 64), torch.zeros(1, 3, 8, 64), lam),
              (q, k, k, torch.zeros(2)), (q, k, k, torch.zeros(1, 4)), (q, k, k, lam.double()), (q, k.bfloat16(), k.bfloat16(), lam),
              (q, k, k, lam)):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            lib.mesh_diff_attention(*a, 1, True)
        with pytest.raises(ValueError):
            lib.mesh_diff_decode(a[0][..., :1, :], a[1], a[2], torch.ones(1, dtype=torch.int32), a[3])
