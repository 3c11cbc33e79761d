"""Argument checks of the linear-attention entry points (no GPU needed)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
P = ctypes.c_void_p
MB = 1 << 24  # fake, aligned addresses, never dereferenced
BASE = dict(q=MB, ldq=256, k=2 * MB, ldk=256, v=3 * MB, ldv=256, decay=4 * MB, beta=5 * MB,
            rows=100, hk=2, hv=4, dk=128, dv=64, state=6 * MB, n_slots=3, slots=7 * MB, o=8 * MB,
            ldo=256)


@pytest.fixture(scope="module")
def L():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4.lib()


def prompts(L, n_seq=3, cu=9 * MB, resume=10 * MB, ws=11 * MB, short=0, **kw):
    a = {**BASE, **kw}
    need = L.nvfp4_linear_attention_workspace_bytes(a["rows"], n_seq, a["hk"], a["hv"], a["dk"])
    return L.nvfp4_linear_attention(
        P(a["q"]), a["ldq"], P(a["k"]), a["ldk"], P(a["v"]), a["ldv"], P(a["decay"]), P(a["beta"]), 1.0,
        a["rows"], a["hk"], a["hv"], a["dk"], a["dv"], n_seq, P(cu), P(a["state"]), a["n_slots"],
        P(a["slots"]), P(resume), P(a["o"]), a["ldo"], P(ws), need - short, None)


def step(L, **kw):
    a = {**BASE, **kw}
    return L.nvfp4_linear_attention_step(
        P(a["q"]), a["ldq"], P(a["k"]), a["ldk"], P(a["v"]), a["ldv"], P(a["decay"]), P(a["beta"]), 1.0,
        a["rows"], a["hk"], a["hv"], a["dk"], a["dv"], P(a["state"]), a["n_slots"], P(a["slots"]),
        P(a["o"]), a["ldo"], None)


@pytest.mark.parametrize("call", [prompts, step])
def test_shared_checks(L, call):
    for name in ("q", "k", "v", "decay", "o"):
        assert call(L, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "o", "state"):
        assert call(L, **{name: BASE[name] + 8}) == MISALIGNED, name
    for name in ("decay", "beta", "slots"):
        assert call(L, **{name: BASE[name] + 2}) == MISALIGNED, name
    for name in ("ldq", "ldk", "ldv", "ldo"):
        assert call(L, **{name: 248}) == INVALID, name      # shorter than the heads
        assert call(L, **{name: 260}) == MISALIGNED, name   # not a multiple of 8
    assert call(L, hv=3, hk=2) == INVALID                   # no whole group
    assert call(L, hk=0) == INVALID
    assert call(L, rows=-1) == INVALID
    assert call(L, n_slots=-1) == INVALID
    assert call(L, dk=96) == UNSUPPORTED
    assert call(L, dv=48) == UNSUPPORTED
    assert call(L, rows=1 << 31) == UNSUPPORTED
    # o over an input
    assert call(L, o=BASE["q"]) == INVALID
    assert call(L, o=BASE["v"] + 512) == INVALID
    assert call(L, o=BASE["q"] + 256, ldo=1024, ldq=1024) == INVALID   # columns that meet
    assert call(L, o=BASE["decay"]) == INVALID
    assert call(L, o=BASE["state"] + 4096) == INVALID


def test_prompt_checks(L):
    assert prompts(L, n_seq=0) == INVALID
    assert prompts(L, cu=None) == INVALID                   # several sequences need offsets
    assert prompts(L, ws=None) == INVALID
    assert prompts(L, ws=11 * MB + 128) == MISALIGNED
    assert prompts(L, short=1) == INVALID
    assert prompts(L, state=None) == INVALID                # slots without a pool
    assert prompts(L, state=None, slots=None) == INVALID    # resume without a pool
    assert prompts(L, slots=None, n_slots=2) == INVALID     # sequence i has slot i
    assert prompts(L, resume=10 * MB + 2) == MISALIGNED


def test_step_checks(L):
    assert step(L, state=None) == INVALID
    assert step(L, slots=None, n_slots=99) == INVALID       # row i has slot i
    assert step(L, hv=65534, hk=2, ldq=256, ldk=256, ldv=65534 * 64, ldo=65534 * 64, rows=1 << 20,
                o=1 << 50) == UNSUPPORTED


def test_workspace_bytes(L):
    f = L.nvfp4_linear_attention_workspace_bytes
    assert f(0, 1, 1, 1, 128) > 0
    assert f(64, 1, 1, 1, 128) == 2 * f(0, 1, 1, 1, 128)
    assert f(100, 3, 2, 4, 96) == 0
    assert f(-1, 1, 1, 1, 128) == 0
    assert f(5, 0, 1, 1, 128) == 0


def test_good_calls_pass_the_checks(L):
    """Without a GPU a call that passes every check fails in CUDA."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for kw in (dict(), dict(beta=None), dict(dk=64, ldq=128, ldk=128), dict(rows=1),
               dict(o=BASE["q"] + 512, ldo=1024, ldq=1024)):
        assert prompts(L, **kw) == CUDA, kw
        assert step(L, **kw) == CUDA, kw
    assert prompts(L, state=None, slots=None, resume=None) == CUDA
    assert prompts(L, n_seq=1, cu=None) == CUDA
    assert prompts(L, rows=0, q=None, k=None, v=None, decay=None, o=None) == CUDA
    assert step(L, rows=0, q=None, k=None, v=None, decay=None, o=None) == OK
