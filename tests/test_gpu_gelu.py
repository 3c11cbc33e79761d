"""GPU test of the epilogue's erf-gelu over its whole range, element by element:
the tokens are zero, so the pre-activations are the bias, exactly.

Tolerance. gelu(z) = z Phi(z); the exponential e^(-z^2/2) is off by 2 + 1.173 t
steps of 2^-23 at an exponent of t = z^2/2 (CUDA's published bound for the fast
one), the fit by 1.7e-7, 1.4 of those steps, its polynomial, reciprocal and
products by 4 more (half a step each): (8 + 1.173 t) 2^-23 of |gelu(z)|, also in
the far tail. Below the smallest normal number results are zero. The output's
rounding is half a step of its own: 2^-8 (bf16) or 2^-24 (FP32)."""
import math

import numpy as np
import pytest
import torch

from parity import bits, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


@pytest.mark.parametrize("m", [4, 40, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gelu_keeps_its_digits(nv, orc, m, dtype):
    n, k = 4096, 512
    z = torch.cat([torch.linspace(-14, 0, n // 2), torch.linspace(0, 14, n // 4),
                   -torch.logspace(-30, 1, n // 8), torch.logspace(-30, 1, n // 8)]).to(torch.bfloat16)
    w = (torch.randn((n, k), generator=torch.Generator().manual_seed(1)) * 0.05).to(torch.bfloat16)
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    y = nv.linear(x, upload(orc.quantize(bits(w))), out_dtype=dtype, bias=z.cuda(), activation="gelu")
    z = z.double().numpy()
    want = 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2.0))
    tol = (8 + 1.173 * z * z / 2) * 2.0 ** -23 * np.abs(want) + 2.0 ** -120
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = tol * (1 + half) + half * np.abs(want)
    worst = (np.abs(y.double().cpu().numpy() - want) / tol).max()
    assert worst <= 1.0, f"{worst:.2f} of the tolerance"


@pytest.mark.parametrize("m", [4, 40, 200])
def test_gelu_at_the_ends(nv, orc, m):
    """Infinities, NaN, zeros and numbers whose square overflows."""
    n, k = 64, 512
    w = (torch.randn((n, k), generator=torch.Generator().manual_seed(1)) * 0.05).to(torch.bfloat16)
    bias = torch.zeros(n, dtype=torch.bfloat16)
    for i, b in enumerate((math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-38, -1e-38)):
        bias[i] = b
    y = nv.linear(torch.zeros(m, k, dtype=torch.bfloat16, device="cuda"), upload(orc.quantize(bits(w))),
                  out_dtype=torch.float32, bias=bias.cuda(), activation="gelu").cpu()
    assert bool((y[:, 0] == math.inf).all()) and bool((y[:, 1] == 0).all())
    assert bool(torch.isnan(y[:, 2]).all())
    assert bool((y[:, 3] == float(bias[3])).all()) and bool((y[:, 4:7].abs() <= 1e-38).all())
    assert not y[:, 7:].any()
