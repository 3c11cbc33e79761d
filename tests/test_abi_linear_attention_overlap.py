"""What linear attention writes (o, the pool of states, its workspace) may not lie
over what it reads, or over one another (no GPU needed)."""
import pytest

from test_abi_linear_attention import BASE, CUDA, INVALID, MB, L, prompts, step  # noqa: F401

STATE = 3 * 4 * 128 * 64 * 4   # bytes of BASE's pool


@pytest.mark.parametrize("call", [prompts, step])
def test_the_pool_over_an_input(L, call):  # noqa: F811
    more = dict(n_seq=3) if call is prompts else {}
    for name in ("q", "k", "v", "decay", "beta", "slots", "o"):
        assert call(L, state=BASE[name], **more) == INVALID, name
        assert call(L, state=BASE[name] + 256 - STATE, **more) == INVALID, name   # its end
    assert call(L, state=BASE["v"] + 99 * 512 + 496) == INVALID    # over v's last columns
    # a pool whose bytes no 64-bit number holds
    assert call(L, hv=1 << 15, hk=1, dv=1 << 15, ldv=1 << 30, ldo=1 << 30, n_slots=1 << 30, rows=3,
                state=MB // 2) == INVALID


def test_the_workspace_over_anything(L):  # noqa: F811
    need = L.nvfp4_linear_attention_workspace_bytes(100, 3, 2, 4, 128)
    where = dict(BASE, cu=9 * MB, resume=10 * MB)
    for name in ("q", "k", "v", "decay", "beta", "state", "slots", "o", "cu", "resume"):
        assert prompts(L, ws=where[name]) == INVALID, name
        assert prompts(L, ws=where[name] - need // 256 * 256 + 256) == INVALID, name


def test_offsets_are_not_written(L):  # noqa: F811
    for name in ("o", "state"):
        assert prompts(L, cu=BASE[name]) == INVALID
        assert prompts(L, resume=BASE[name] + 64) == INVALID
    assert prompts(L, slots=BASE["o"]) == INVALID
    assert step(L, slots=BASE["o"]) == INVALID


def test_neighbours_are_fine(L):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    need = L.nvfp4_linear_attention_workspace_bytes(100, 3, 2, 4, 128)
    end = lambda name, n: BASE[name] + -(-n // 256) * 256  # noqa: E731
    assert prompts(L, state=end("v", 99 * 512 + 512)) == CUDA
    assert step(L, state=BASE["q"] - STATE) == CUDA
    assert prompts(L, ws=end("state", STATE)) == CUDA
    assert prompts(L, ws=BASE["q"] - -(-need // 256) * 256) == CUDA
    assert prompts(L, cu=BASE["slots"]) == CUDA               # inputs may share bytes
    assert prompts(L, resume=9 * MB) == CUDA
