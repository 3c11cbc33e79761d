"""GPU tests of the GEMM epilogue (nvfp4_gemm_epilogue, nvfp4_linear_epilogue):
y = act(P + bias) + residual against the same formula in FP64 on the oracle's
product P (the product itself: news article "Qwen3.8-27B最激进4bit量化开源…" §02).

Tolerance, per element. P is a sum of k terms in FP32: within
k 2^-24 ||x_hat_m|| ||w_hat_n|| of the exact sum (each addition is off by half
a step of a partial sum that Cauchy-Schwarz bounds), and alpha = 1/(g g) and
the product with it add 3 half steps of |P|. The activations have slopes of at
most 1.13. Their fast exponential is off by 2 + 1.173 |t| steps (CUDA's
published bound), the addition, division and products by 6 more. gelu is
z/2 + z/2 erf(z / sqrt 2): erff is off by 2 steps of a value of at most 1, and
its argument, rounded twice, moves it by at most 2 sqrt(2/pi e) 2^-24 more
(x erf'(x) <= sqrt(2/(pi e)) < 0.49); times |z|/2, with the last sum's half
step of |z|/2, that is within 2 |z| 2^-23 (an absolute bound: where the two
halves cancel, the far negative tail, the relative digits are lost). The sums
with bias and residual are each half a step, and the output type's rounding
half a step of its own: 2^-8 of |y| in bf16.
"""
import math

import numpy as np
import pytest
import torch

from parity import bits, norms, upload

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def gaussian(rows, k, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, k), generator=g) * sigma).to(torch.bfloat16)


def act64(z, name):
    """(act(z), |t| of the activation's exponential)."""
    if name == "relu":
        return np.maximum(z, 0.0), 0.0
    if name == "silu":
        return z / (1.0 + np.exp(np.minimum(-z, 700.0))), np.abs(z)
    if name == "gelu":
        erfc = np.vectorize(math.erfc)
        return 0.5 * z * erfc(-z / math.sqrt(2.0)), 0.0
    if name == "gelu_tanh":
        t = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        return z / (1.0 + np.exp(np.minimum(-t, 700.0))), np.abs(t)
    return z, 0.0


def check(y, p_ref, row_norm, col_norm, k, bias, act, res, what):
    z = p_ref + (0.0 if bias is None else bias.double().numpy())
    a, t = act64(z, act)
    ref = a + (0.0 if res is None else res.double().numpy())
    tol = 1.13 * (k * 2.0 ** -24 * np.outer(row_norm, col_norm)
                  + 3 * 2.0 ** -24 * np.abs(p_ref) + 2.0 ** -24 * np.abs(z))
    tol += (8 + 1.173 * np.minimum(t, 100.0)) * 2.0 ** -23 * np.abs(a) + 1e-35
    if act == "gelu":
        tol += 2.0 * 2.0 ** -23 * np.abs(z)
    tol += 2.0 ** -24 * np.abs(ref)
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(y.double().cpu().numpy() - ref)
    worst = (err / tol).max()
    assert worst <= 1.0, f"{what}: {worst:.2f} of the tolerance"


# few-token kernels (in-kernel quantization up to 8), their 16/32/64-token
# tiles, and the paired kernel; n ragged against 8, 32, 128 and 256 columns
@pytest.mark.parametrize("m,n,k", [(1, 640, 512), (8, 1000, 2048), (9, 136, 512), (17, 1000, 2048),
                                   (33, 296, 512), (64, 1000, 1056), (65, 296, 512),
                                   (300, 1000, 2048), (100, 328, 8192), (1, 19000, 256),
                                   (40, 19000, 256)])
@pytest.mark.parametrize("act", ACTS)
def test_linear_epilogue(nv, orc, m, n, k, act):
    x, w = gaussian(m, k, m + n), gaussian(n, k, 7, 1.5 / math.sqrt(k))
    qx, qw = orc.quantize(bits(x)), orc.quantize(bits(w))
    ref = orc.gemm(qx, qw)
    W = upload(qw)
    bias, res = gaussian(1, n, 8)[0], gaussian(m, n, 9, 2.0)
    ws = nv.linear_workspace(m, n, k)
    gws = torch.empty(max(16, nv.gemm_workspace_bytes(m, n, k)), dtype=torch.uint8, device="cuda")
    A = nv.quantize(x.cuda())
    for b, r in ((bias, res), (bias, None), (None, res)):
        bd, rd = (None if t is None else t.cuda() for t in (b, r))
        for dt in (torch.bfloat16, torch.float32):
            y = nv.linear(x.cuda(), W, out_dtype=dt, bias=bd, activation=act, residual=rd, workspace=ws)
            what = f"{m}x{n}x{k} {act} bias={b is not None} res={r is not None} {dt}"
            check(y, ref, norms(orc, qx), norms(orc, qw), k, b, act, r, what)
            y2 = nv.gemm(A, W, out_dtype=dt, bias=bd, activation=act, residual=rd, workspace=gws)
            assert torch.equal(y, y2), what
            # without a workspace the few-token GEMM does not split: another order of sums
            y3 = nv.gemm(A, W, out_dtype=dt, bias=bd, activation=act, residual=rd)
            check(y3, ref, norms(orc, qx), norms(orc, qw), k, b, act, r, what + " unsplit")
    assert nv.read_fault() == 0


@pytest.mark.parametrize("m,n,k", [(3, 640, 512), (20, 640, 2048), (300, 520, 512), (100, 328, 8192)])
def test_residual_in_place_and_as_columns(nv, orc, m, n, k):
    """The residual may be Y itself, or other columns of Y's matrix; rows and
    columns outside Y stay as they were."""
    x, w = gaussian(m, k, 1), gaussian(n, k, 2, 0.05)
    W = upload(orc.quantize(bits(w)))
    res, bias = gaussian(m, n, 3), gaussian(1, n, 4)[0].cuda()
    ref = nv.linear(x.cuda(), W, bias=bias, activation="silu", residual=res.cuda())
    y = res.cuda().clone()
    nv.linear(x.cuda(), W, out=y, bias=bias, activation="silu", residual=y)
    assert torch.equal(y, ref)
    wide = torch.full((m + 1, 2 * n + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:m, n + 8:] = res.cuda()
    nv.linear(x.cuda(), W, out=wide[:m, :n], bias=bias, activation="silu", residual=wide[:m, n + 8:])
    assert torch.equal(wide[:m, :n], ref)
    assert torch.equal(wide[:m, n + 8:], res.cuda())
    assert bool((wide[:m, n:n + 8] == 5).all()) and bool((wide[m] == 5).all())


@pytest.mark.parametrize("m", [4, 40, 200])
def test_no_epilogue_is_linear_and_extremes(nv, orc, m):
    n, k = 520, 512
    x, w = gaussian(m, k, 1), gaussian(n, k, 2, 0.05)
    W = upload(orc.quantize(bits(w)))
    plain = nv.linear(x.cuda(), W)
    zero = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(plain, nv.linear(x.cuda(), W, bias=zero))
    # pre-activations far outside the exponentials' range, both ways
    for act in ACTS:
        for big in (1e3, -1e3, 3e38, -3e38):
            bias = torch.full((n,), big, dtype=torch.bfloat16, device="cuda")
            y = nv.linear(x.cuda(), W, out_dtype=torch.float32, bias=bias, activation=act)
            want = big if (big > 0 or act == "none") else 0.0
            assert bool(((y - want).abs() <= 1e-2 * max(abs(want), 1e-30) + 0.0).all()), (act, big)


@pytest.mark.parametrize("m", [2, 40, 200])
def test_epilogue_in_a_graph(nv, orc, m):
    """Captured and replayed with new inputs in the same buffers."""
    n, k = 640, 1024
    W = upload(orc.quantize(bits(gaussian(n, k, 2, 0.05))))
    x, res = gaussian(m, k, 1).cuda(), gaussian(m, n, 3).cuda()
    bias = gaussian(1, n, 4)[0].cuda()
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ws = nv.linear_workspace(m, n, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nv.linear(x, W, out=y, bias=bias, activation="gelu", residual=res, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.linear(x, W, out=y, bias=bias, activation="gelu", residual=res, workspace=ws)
    for seed in (10, 11):
        x.copy_(gaussian(m, k, seed))
        res.copy_(gaussian(m, n, seed + 5))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, nv.linear(x, W, bias=bias, activation="gelu", residual=res))


@pytest.mark.parametrize("m", [4, 40, 200])
@pytest.mark.parametrize("act", ACTS)
def test_not_a_number_stays(nv, orc, m, act):
    """A NaN in one column's bias or one element of the residual reaches that
    column or element, whatever the activation, and nothing else."""
    n, k = 520, 512
    x, W = gaussian(m, k, 1).cuda(), upload(orc.quantize(bits(gaussian(n, k, 2, 0.05))))
    bias, res = gaussian(1, n, 4)[0].cuda(), gaussian(m, n, 3).cuda()
    ref = nv.linear(x, W, bias=bias, activation=act, residual=res)
    bias[77] = res[m - 1, 300] = float("nan")
    y = nv.linear(x, W, bias=bias, activation=act, residual=res)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[:, 77] = bad[m - 1, 300] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], ref[~bad])


def test_binding_refuses(nv, orc):
    x, W = gaussian(4, 64, 1).cuda(), upload(orc.quantize(bits(gaussian(64, 64, 2))))
    a = nv.quantize(x)
    bias, res = torch.zeros(64, dtype=torch.bfloat16).cuda(), torch.zeros(4, 64, dtype=torch.bfloat16).cuda()
    for call in (lambda **kw: nv.linear(x, W, **kw), lambda **kw: nv.gemm(a, W, **kw)):
        for kw in (dict(activation="tanh"), dict(bias=bias.float()), dict(bias=bias[:32]), dict(bias=bias.cpu()),
                   dict(bias=bias[None]), dict(residual=res[:3]), dict(residual=res.float()),
                   dict(residual=res.cpu()), dict(residual=res.t().contiguous().t()),
                   dict(bias=bias, out=torch.empty(3, 64, dtype=torch.bfloat16, device="cuda")),
                   dict(bias=bias, out=torch.empty(4, 64, dtype=torch.bfloat16))):
            with pytest.raises(ValueError):
                call(**kw)
        for kw in (dict(residual=res[:1].expand(4, 64)), dict(bias=bias, out=bias.expand(4, 64))):
            with pytest.raises((ValueError, nv.NVFP4Error)):
                call(**kw)
    with pytest.raises(nv.NVFP4Error):
        nv.linear(x, W, residual=x, out=x)
