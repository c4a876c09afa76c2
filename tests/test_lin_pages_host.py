"""Host-side refusals of kda_lin_* and kda_pages_* (no GPU needed): every bad argument is answered before
anything is launched, with pointers that are never dereferenced."""
import ctypes

import pytest
import torch

import kda_linear_attention_02_b200 as kda
from kda_linear_attention_02_b200 import build as kbuild

vp = ctypes.c_void_p
ARG, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda._load()


def chunk(lib, **over):
    a = dict(q=0x1000, k=0x2000, v=0x3000, la=0x4000, per=1, s0=None, cu=0x6000, n=2, T=100, Hqk=2, H=4, dk=128, dv=128,
             dt=0, stride=0, o=0x7000, fs=None, ck=None, ckcu=None, ws=0x10000, wsb=1 << 30)
    a.update(over)
    return lib.kda_lin_chunk_fwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["la"]), a["per"], vp(a["s0"]), vp(a["cu"]), a["n"],
                                 a["T"], a["Hqk"], a["H"], a["dk"], a["dv"], a["dt"], a["stride"], vp(a["o"]), vp(a["fs"]),
                                 vp(a["ck"]), vp(a["ckcu"]), vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), ARG), (dict(T=-1), ARG), (dict(T=1 << 31), ARG), (dict(H=0), ARG), (dict(Hqk=0), ARG), (dict(Hqk=3), ARG),
    (dict(per=2), ARG), (dict(stride=-64), ARG), (dict(stride=100, ck=0x1000, ckcu=0x1000), ARG), (dict(stride=64), ARG),
    (dict(dt=2), ARG), (dict(dt=7), ARG), (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(la=None), ARG),
    (dict(o=None), ARG), (dict(cu=None), ARG), (dict(ws=None), ARG), (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED),
    (dict(q=0x1008), ALIGN), (dict(o=0x7002), ALIGN), (dict(s0=0x8004), ALIGN), (dict(fs=0x8004), ALIGN), (dict(la=0x4002), ALIGN),
    (dict(cu=0x6001), ALIGN), (dict(ws=0x10080), ALIGN), (dict(wsb=64), WORKSPACE), (dict(n=0), ARG),
    (dict(s0=0x100000, fs=0x100000), ARG), (dict(s0=0x100000, fs=0x100000 + 2 * 4 * 128 * 128 * 4 - 16), ARG)])
def test_chunk_refusals(lib, over, want):
    assert chunk(lib, **over) == want


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("name,size", [("q", 100 * 2 * 128), ("k", 100 * 2 * 128), ("v", 100 * 4 * 128)])
def test_outputs_over_inputs_are_refused(lib, dt, name, size):
    # o [100, 4, 128] begins at the input, or 16 bytes ahead of the input's end, or ends 16 bytes behind its start
    es, at = (2, 4)[dt], 1 << 30
    apart = dict(q=1 << 32, k=2 << 32, v=3 << 32, dt=dt)
    for o in (at, at + size * es - 16, at - 100 * 4 * 128 * es + 16):
        assert chunk(lib, **{**apart, name: at, "o": o}) == ARG
        assert step(lib, **{**apart, name: at, "o": o, "n": 100, "ns": 100}) == ARG


def test_chunk_of_nothing_is_fine(lib):
    assert chunk(lib, n=0, T=0) == 0


def test_workspace_query(lib):
    f = kda.kda_lin_chunk_fwd_workspace_bytes
    assert f(0, 0, 1, 64, 64) > 0 and f(1 << 20, 8, 32, 128, 128) > f(100, 8, 32, 128, 128) > 0
    assert f(100, 1, 2, 96, 64) == 0 and f(-1, 1, 2, 64, 64) == 0 and f(100, 1, 2, 64, 64, kda.KDA_MXFP8) == 0
    assert f(100, 1, 0, 64, 64) == 0 and f(1 << 31, 1, 1, 64, 64) == 0


def step(lib, **over):
    a = dict(state=0x1000, ns=8, slots=0x2000, stride=1, q=0x3000, k=0x4000, v=0x5000, la=0x6000, per=1, n=4, Hqk=2, H=4,
             dk=128, dv=128, dt=0, o=0x7000)
    a.update(over)
    return lib.kda_lin_recurrent_step(vp(a["state"]), a["ns"], vp(a["slots"]), a["stride"], vp(a["q"]), vp(a["k"]), vp(a["v"]),
                                      vp(a["la"]), a["per"], a["n"], a["Hqk"], a["H"], a["dk"], a["dv"], a["dt"], vp(a["o"]), None)


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), ARG), (dict(ns=-1), ARG), (dict(slots=None, ns=3), ARG), (dict(stride=0), ARG), (dict(H=0), ARG),
    (dict(Hqk=3), ARG), (dict(per=-1), ARG), (dict(dt=2), ARG), (dict(dk=32), UNSUPPORTED), (dict(state=None), ARG),
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(la=None), ARG), (dict(o=None), ARG),
    (dict(state=0x1008), ALIGN), (dict(q=0x3001), ALIGN), (dict(v=0x5002, dt=1), ALIGN), (dict(slots=0x2002), ALIGN),
    (dict(n=1 << 30, H=32), ARG)])
def test_step_refusals(lib, over, want):
    assert step(lib, **over) == want


def test_step_of_nothing_is_fine(lib):
    assert step(lib, n=0) == 0


def copy(lib, **over):
    a = dict(dst=0x100000, nd=8, src=0x200000, ns=8, dp=0x1000, sp=0x2000, n=4, pb=1024)
    a.update(over)
    return lib.kda_pages_copy(vp(a["dst"]), a["nd"], vp(a["src"]), a["ns"], vp(a["dp"]), vp(a["sp"]), a["n"], a["pb"], None)


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), ARG), (dict(nd=-1), ARG), (dict(ns=1 << 31), ARG), (dict(pb=0), ARG), (dict(pb=1000), ARG),
    (dict(pb=(1 << 30) + 16), ARG), (dict(dp=None, nd=3), ARG), (dict(sp=None, ns=3), ARG), (dict(dst=None), ARG),
    (dict(src=None), ARG), (dict(dst=0x100008), ALIGN), (dict(src=0x200004), ALIGN), (dict(dp=0x1002), ALIGN),
    (dict(src=0x100400), ARG), (dict(src=0x100010), ARG), (dict(src=0xff000), ARG)])
def test_copy_refusals(lib, over, want):
    assert copy(lib, **over) == want


def test_copy_of_nothing_is_fine(lib):
    assert copy(lib, n=0) == 0


def fork(lib, **over):
    a = dict(pool=0x100000, planes=1, np=8, pb=64, refs=0x1000, table=0x2000, counts=0x3000, rows=4, most=3, p=0x4000, c=0x5000,
             sh=0x6000, fr=None, n=2, zero=0, ws=0x10000, wsb=1 << 20)
    a.update(over)
    return lib.kda_pages_fork(vp(a["pool"]), a["planes"], a["np"], a["pb"], vp(a["refs"]), vp(a["table"]), vp(a["counts"]),
                              a["rows"], a["most"], vp(a["p"]), vp(a["c"]), vp(a["sh"]), vp(a["fr"]), a["n"], a["zero"],
                              vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), ARG), (dict(planes=0), ARG), (dict(np=-1), ARG), (dict(pb=8), ARG), (dict(rows=-1), ARG),
    (dict(rows=(1 << 20) + 1), ARG), (dict(most=0), ARG), (dict(zero=2), ARG), (dict(n=1 << 20, most=1 << 12), ARG),
    (dict(pool=None), ARG), (dict(refs=None), ARG), (dict(table=None), ARG), (dict(counts=None), ARG), (dict(p=None), ARG),
    (dict(c=None), ARG), (dict(sh=0x6002), ALIGN), (dict(ws=None), ARG), (dict(pool=0x100008), ALIGN), (dict(table=0x2001), ALIGN),
    (dict(fr=0x7002), ALIGN), (dict(ws=0x10010), ALIGN), (dict(wsb=64), WORKSPACE)])
def test_fork_refusals(lib, over, want):
    assert fork(lib, **over) == want


def test_fork_workspace(lib):
    need = lib.kda_pages_fork_workspace_bytes(2, 3)
    assert need > 0 and fork(lib, wsb=need - 1) == WORKSPACE and fork(lib, n=0) == 0
    assert lib.kda_pages_fork_workspace_bytes(-1, 3) == 0 and lib.kda_pages_fork_workspace_bytes(1 << 20, 1 << 12) == 0


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), ARG), (dict(np=-1), ARG), (dict(rows=-1), ARG), (dict(most=0), ARG), (dict(refs=None), ARG), (dict(r=None), ARG),
    (dict(table=None), ARG), (dict(counts=None), ARG), (dict(refs=0x1002), ALIGN), (dict(r=0x4001), ALIGN), (dict(n=0), 0)])
def test_free_refusals(lib, over, want):
    a = dict(refs=0x1000, np=8, table=0x2000, counts=0x3000, rows=4, most=3, r=0x4000, n=2)
    a.update(over)
    assert lib.kda_pages_free(vp(a["refs"]), a["np"], vp(a["table"]), vp(a["counts"]), a["rows"], a["most"], vp(a["r"]), a["n"],
                              None) == want


@pytest.mark.parametrize("over,want", [
    (dict(planes=0), ARG), (dict(np=-1), ARG), (dict(pb=24), ARG), (dict(rows=-1), ARG), (dict(most=0), ARG), (dict(pool=None), ARG),
    (dict(refs=None), ARG), (dict(remap=None), ARG), (dict(table=None), ARG), (dict(ws=None), ARG), (dict(pool=0x100004), ALIGN),
    (dict(remap=0x4002), ALIGN), (dict(nl=0x5001), ALIGN), (dict(ws=0x10001), ALIGN), (dict(wsb=16), WORKSPACE)])
def test_compact_refusals(lib, over, want):
    a = dict(pool=0x100000, planes=1, np=8, pb=64, refs=0x1000, table=0x2000, counts=0x3000, rows=4, most=3, remap=0x4000, nl=None,
             ws=0x10000, wsb=1 << 20)
    a.update(over)
    assert lib.kda_pages_compact(vp(a["pool"]), a["planes"], a["np"], a["pb"], vp(a["refs"]), vp(a["table"]), vp(a["counts"]),
                                 a["rows"], a["most"], vp(a["remap"]), vp(a["nl"]), vp(a["ws"]), a["wsb"], None) == want


def test_bindings_refuse_wrong_tensors(lib):
    z = torch.zeros
    i32 = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    q, v, la, cu, o = z(4, 1, 64), z(4, 2, 64), z(4, 2), i32(2), z(4, 2, 64)
    for bad in (dict(q=z(4, 64)), dict(k=z(4, 2, 64)), dict(v=z(5, 2, 64)), dict(la=z(4, 3)), dict(la=z(3)), dict(cu=z(2)),
                dict(o=z(4, 2, 64, dtype=torch.float16)), dict(q=q.half()), dict(s0=z(1, 2, 64, 32)), dict(q=q.transpose(0, 2)),
                dict()):                                       # the last: everything right, but not on a GPU
        a = dict(q=q, k=q, v=v, la=la, s0=None, cu=cu, o=o)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_lin_chunk_fwd(*a.values())
    st = z(3, 2, 64, 64)
    for bad in (dict(slots=z(4)), dict(slots=i32(5)), dict(state=st.double()), dict(q=z(5, 1, 64)), dict(slots=None), dict(slots=i32(1).expand(4))):
        a = dict(state=st, q=q, slots=i32(4))
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_lin_recurrent_step(a["state"], a["q"], q, v, la, o, slots=a["slots"])
    for bad in ((z(4, 3), z(4, 3)), (z(4, 8), z(4, 4)), (z(4, 8), z(4, 8).int()), (z(4, 8), None), (z(0, 8), z(4, 8))):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_pages_copy(*bad)
    pool, refs, table, counts = z(1, 5, 8), i32(5), i32(3, 2), i32(3)
    for f in (lambda p, r, t, c: kda.kda_pages_fork(p, r, t, c, i32(1), i32(1)), kda.kda_pages_compact):
        for bad in ((pool[0], refs, table, counts), (pool, i32(4), table, counts), (pool, refs, table[0], counts),
                    (pool, refs, table, i32(2)), (pool, refs.long(), table, counts)):
            with pytest.raises((ValueError, TypeError)):
                f(*bad)
    with pytest.raises((ValueError, TypeError)):
        kda.kda_pages_fork(pool, refs, table, counts, i32(2), i32(1))
    with pytest.raises((ValueError, TypeError)):
        kda.kda_pages_free(refs, table, counts, z(2))
