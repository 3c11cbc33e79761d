"""Argument checks of linear attention's self-test (no GPU needed)."""
import pytest

from test_abi_linear_attention import BASE, CUDA, INVALID, MB, MISALIGNED, L, P  # noqa: F401


def stall(L, kernel=0, cta=0, limit=1_000_000, **kw):  # noqa: F811
    a = {**BASE, **kw}
    need = L.nvfp4_linear_attention_workspace_bytes(a["rows"], 3, a["hk"], a["hv"], a["dk"])
    return L.nvfp4_selftest_linear_attention_stall(
        P(a["q"]), a["ldq"], P(a["k"]), a["ldk"], P(a["v"]), a["ldv"], P(a["decay"]), P(a["beta"]), 1.0,
        a["rows"], a["hk"], a["hv"], a["dk"], a["dv"], 3, P(9 * MB), P(a["state"]), a["n_slots"],
        P(a["slots"]), P(10 * MB), P(a["o"]), a["ldo"], P(11 * MB), need, kernel, cta, limit, None)


def test_checks(L):  # noqa: F811
    assert stall(L, kernel=2) == INVALID
    assert stall(L, kernel=-1) == INVALID
    assert stall(L, cta=-1) == INVALID
    assert stall(L, limit=999) == INVALID
    assert stall(L, limit=20_000_000_000) == INVALID
    assert stall(L, q=None) == INVALID
    assert stall(L, q=BASE["q"] + 8) == MISALIGNED


def test_a_good_call_passes_the_checks(L):  # noqa: F811
    """Without a GPU it then fails in CUDA."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert stall(L) == CUDA and stall(L, kernel=1, cta=5) == CUDA
