"""Refusals of kda_lin_* and kda_pages_* that guard memory and results (no GPU needed): sizes that the kernels' indices
could not hold, and outputs over other arguments.  Pointers are made up; nothing is launched."""
import ctypes

import pytest
import torch

import kda_linear_attention_02_b200 as kda
from kda_linear_attention_02_b200 import build as kbuild

vp = ctypes.c_void_p
ARG = -1
TOO_MANY = [(1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1]


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda._load()


@pytest.mark.parametrize("n", TOO_MANY)
def test_lists_and_pools_that_wrap_an_index_are_refused(lib, n):
    a, b, c, d, e, f, ws = (vp(i << 40) for i in range(1, 8))
    most = (1 << 31) - 1
    assert lib.kda_pages_copy(a, most, b, most, c, d, n, 16, None) == ARG
    assert lib.kda_pages_copy(a, most, b, most, None, d, n, 16, None) == ARG
    assert lib.kda_pages_fork(a, 1, n, 16, b, c, d, 4, 3, e, f, None, None, 2, 0, ws, 1 << 40, None) == ARG
    assert lib.kda_pages_compact(a, 1, n, 16, b, c, d, 4, 3, e, None, ws, 1 << 40, None) == ARG
    assert lib.kda_pages_compact_workspace_bytes(n) == 0 < lib.kda_pages_compact_workspace_bytes(1 << 30)
    assert lib.kda_pages_free(a, n, b, c, 4, 3, d, 2, None) == ARG
    assert lib.kda_pages_free(a, 8, b, c, 4, 3, d, n, None) == ARG
    assert lib.kda_lin_recurrent_step(a, 8, b, 1, c, c, d, e, 1, n, 1, 1, 64, 64, 0, f, None) == ARG


def spans(**sizes):
    """A place of its own for each name, 2^36 bytes apart (no more is used of any)."""
    return {name: (i + 1) << 36 for i, name in enumerate(sizes)}


def over(at, out, n_out, name, n):
    """Places of `out` that touch `name`: at its start, at its last 16 bytes, and ending 16 bytes behind its start."""
    return [at[name], at[name] + (n - 1) // 16 * 16, at[name] - n_out // 16 * 16 + 16]


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("per", [0, 1])
@pytest.mark.parametrize("out", ["o", "fs", "ws"])
@pytest.mark.parametrize("name", ["q", "k", "v", "la", "s0", "cu", "ckcu", "o", "fs", "ws"])
def test_chunk_outputs_over_anything_are_refused(lib, dt, per, out, name):
    n, T, Hqk, H, dk, dv = 3, 100, 2, 4, 128, 64
    es = (2, 4)[dt]
    ws = lib.kda_lin_chunk_fwd_workspace_bytes(T, n, H, dk, dv, dt)
    size = dict(q=T * Hqk * dk * es, k=T * Hqk * dk * es, v=T * H * dv * es, la=(T if per else 1) * H * 4, s0=n * H * dk * dv * 4,
                cu=(n + 1) * 4, ckcu=(n + 1) * 4, o=T * H * dv * es, fs=n * H * dk * dv * 4, ws=ws, ck=0)

    def call(at):
        return lib.kda_lin_chunk_fwd(vp(at["q"]), vp(at["k"]), vp(at["v"]), vp(at["la"]), per, vp(at["s0"]), vp(at["cu"]), n, T,
                                     Hqk, H, dk, dv, dt, 64, vp(at["o"]), vp(at["fs"]), vp(at["ck"]), vp(at["ckcu"]), vp(at["ws"]),
                                     ws, None)
    at = spans(**size)
    if out != name:
        for x in over(at, out, size[out], name, size[name]):
            if out != "ws" or x % 256 == 0:      # (a workspace elsewhere is refused for its alignment)
                assert call({**at, out: x}) == ARG


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("out", ["o", "state"])
@pytest.mark.parametrize("name", ["q", "k", "v", "la", "slots", "state", "o"])
def test_step_outputs_over_anything_are_refused(lib, dt, out, name):
    n, ns, Hqk, H, dk, dv, stride = 5, 7, 2, 4, 64, 128, 3
    es = (2, 4)[dt]
    size = dict(q=n * Hqk * dk * es, k=n * Hqk * dk * es, v=n * H * dv * es, la=n * H * 4, slots=((n - 1) * stride + 1) * 4,
                state=ns * H * dk * dv * 4, o=n * H * dv * es)

    def call(at):
        return lib.kda_lin_recurrent_step(vp(at["state"]), ns, vp(at["slots"]), stride, vp(at["q"]), vp(at["k"]), vp(at["v"]),
                                          vp(at["la"]), 1, n, Hqk, H, dk, dv, dt, vp(at["o"]), None)
    at = spans(**size)
    if out != name:
        for x in over(at, out, size[out], name, size[name]):
            assert call({**at, out: x}) == ARG


@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "initial_state", "o", "final_state", "workspace", "cu_seqlens", "ckpt_cu"])
def test_checkpoints_over_anything_are_refused(lib, name):
    T, H, d = 128, 2, 64
    f = torch.zeros
    a = dict(q=f(T, H, d), k=f(T, H, d), v=f(T, H, d), log_alpha=f(T, H), initial_state=f(1, H, d, d), cu_seqlens=f(2).int(), o=f(T, H, d),
             final_state=f(1, H, d, d))
    kw = dict(ckpt_stride=64, checkpoints=f(2, H, d, d), ckpt_cu=f(2).int(), workspace=f(1 << 16, dtype=torch.uint8))
    buf = f(1 << 18)
    kw["checkpoints"] = buf[100_000:100_000 + 2 * H * d * d].view(2, H, d, d)
    old = {**a, **kw}[name]
    n = old.nbytes // 4
    new = buf[100_000 + 2 * H * d * d - 4:][:n].view(old.dtype).view(old.shape)      # the checkpoints' last 16 bytes
    (a if name in a else kw)[name] = new
    with pytest.raises(ValueError, match=f"and {name} must not overlap"):
        kda.kda_lin_chunk_fwd(*a.values(), **kw)
