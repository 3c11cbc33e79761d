"""Argument checks of the GEMM epilogue's entry points (no GPU needed)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
P = ctypes.c_void_p
FAKE = 1 << 24  # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4.lib()


def lin(L, m=8, k=64, n=64, bias=None, act=0, res=None, ldr=64, y=FAKE, yd=0, ldy=64):
    need = L.nvfp4_linear_workspace_bytes(m, n, k)
    return L.nvfp4_linear_epilogue(P(FAKE * 8), m, k, k, None, P(FAKE * 2), P(FAKE * 3), P(FAKE * 4),
                                   n, P(bias), act, P(res), ldr, P(y), yd, ldy, P(FAKE * 5), need, None)


def gemm(L, m=8, k=64, n=64, bias=None, act=0, res=None, ldr=64, y=FAKE, yd=0, ldy=64):
    return L.nvfp4_gemm_epilogue(P(FAKE * 8), P(FAKE * 9), P(FAKE * 2), P(FAKE * 3), P(FAKE * 4),
                                 P(FAKE * 5), P(bias), act, P(res), ldr, P(y), yd, ldy, m, n, k,
                                 None, 0, None)


@pytest.mark.parametrize("call", [lin, gemm])
def test_epilogue_argument_checks(L, call):
    other = FAKE * 6
    assert call(L, act=5) == INVALID
    assert call(L, act=-1) == INVALID
    assert call(L, bias=other + 2) == MISALIGNED
    assert call(L, res=other + 2) == MISALIGNED
    assert call(L, res=other, ldr=68) == MISALIGNED       # ldr % 8
    assert call(L, res=other, ldr=56) == INVALID          # ldr < n
    assert call(L, bias=FAKE + 64) == INVALID             # the bias inside Y
    # the residual over Y: only the same rows in place, or disjoint columns
    assert call(L, res=FAKE + 256, ldr=64) == INVALID     # two rows down
    assert call(L, res=FAKE, ldr=72) == INVALID           # another pitch
    assert call(L, res=FAKE, yd=1) == INVALID             # FP32 Y over a bf16 residual
    assert call(L, res=FAKE + 32, ldr=200, ldy=200) == INVALID  # columns 16.. of Y's own 64
    assert call(L, res=FAKE + 288, ldr=200, ldy=200) == INVALID  # columns 144.. reach into the next row
    # what the product's own checks refuse stays refused
    assert call(L, k=48) == UNSUPPORTED
    assert call(L, m=0) == INVALID
    assert call(L, ldy=32) == INVALID
    assert call(L, n=60, ldy=60) == MISALIGNED


def test_the_input_is_not_the_output(L):
    """X + layer(X) into X would be read while it is written."""
    x = FAKE * 8
    assert lin(L, y=x, res=x) == INVALID
    assert lin(L, m=300, y=x, res=x) == INVALID
    assert lin(L, y=x + 64 * 2) == INVALID                # a row down
    import torch
    if not torch.cuda.is_available():
        assert lin(L, y=FAKE, res=x) == CUDA              # X as the residual only


@pytest.mark.parametrize("call", [lin, gemm])
def test_epilogue_accepts(L, call):
    """Good arguments pass every check: without a GPU the call then fails in
    CUDA, with one it would launch on addresses that do not exist, so this
    runs only where there is none."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    other = FAKE * 6
    for kw in (dict(), dict(bias=other), dict(res=other), dict(res=FAKE), dict(act=4),
               dict(res=FAKE + 128, ldr=200, ldy=200), dict(yd=1, res=other),
               dict(m=1, res=FAKE, ldr=128)):
        assert call(L, **kw) == CUDA, kw
