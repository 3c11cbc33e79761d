"""The operators of a Gated DeltaNet layer run together, as a server runs them:
the fused input projection (nvfp4_linear on the repaired group), the gated delta
rule over a prompt and then token by token, and the output projection with the
residual stream in its epilogue. (News article "Qwen3.8-27B最激进4bit量化开源…" §01
lists the layer's projections and the gated delta rule, §03 the fused group.)

Every stage is checked against FP64 on the inputs it was given on the GPU: the
recurrence as in test_gpu_linear_attention.py, the output projection as in
test_gpu_epilogue.py.
"""
import numpy as np
import pytest
import torch

from parity import bits, norms, upload
from test_gpu_epilogue import check as check_linear
from test_gpu_linear_attention import check as check_recurrence, recurrence

pytestmark = pytest.mark.gpu

D, HK, HV, DK, DV = 512, 2, 4, 128, 128
QKV, Z = 2 * HK * DK + HV * DV, HV * DV


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def gaussian(rows, k, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, k), generator=g) * sigma).to(torch.bfloat16)


class Layer:
    """Weights of one layer and a pass over packed rows."""

    def __init__(self, nv, orc):
        self.nv = nv
        sizes = ((QKV, 0.05, 1), (Z, 0.05, 2), (HV, 0.05, 3), (HV, 0.05, 4))
        self.w_in = nv.fuse_group([nv.quantize(gaussian(n, D, s, sig).cuda()) for n, sig, s in sizes])
        self.q_out = orc.quantize(bits(gaussian(D, HV * DV, 5, 0.05)))
        self.w_out = upload(self.q_out)
        g = torch.Generator().manual_seed(6)
        self.a = 1.0 + 15.0 * torch.rand(HV, generator=g).cuda()
        self.dt_bias = torch.log(torch.expm1(torch.exp(torch.rand(HV, generator=g) * 4.6 - 6.9))).cuda()

    def project(self, x):
        y = self.nv.linear(x, self.w_in)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(torch.bfloat16)
        q = unit(y[:, :HK * DK].unflatten(1, (HK, DK)))
        k = unit(y[:, HK * DK:2 * HK * DK].unflatten(1, (HK, DK)))
        v = y[:, 2 * HK * DK:QKV].unflatten(1, (HV, DV))  # a view of the projection
        a, b = y[:, QKV + Z:QKV + Z + HV].float(), y[:, QKV + Z + HV:].float()
        decay = -self.a * torch.nn.functional.softplus(a + self.dt_bias)
        return q, k, v, decay, torch.sigmoid(b)

    def out(self, o, x):
        return self.nv.linear(o.flatten(1), self.w_out, residual=x)

    def check_out(self, orc, y, o, x, what):
        o = o.flatten(1).cpu()
        qx = orc.quantize(bits(o))
        check_linear(y, orc.gemm(qx, self.q_out), norms(orc, qx), norms(orc, self.q_out), HV * DV,
                     None, "none", x.cpu(), what)


def test_prompts_then_single_tokens(nv, orc):
    layer = Layer(nv, orc)
    lens = [70, 3, 130]
    total, n, steps = sum(lens), len(lens), 3
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    slots = torch.tensor([2, 0, 3], dtype=torch.int32).cuda()
    pool = torch.full((4, HV, DK, DV), 7.0, device="cuda")
    scale = DK ** -0.5

    x = gaussian(total, D, 10).cuda()
    ins = layer.project(x)
    o = nv.linear_attention(*ins, cu_seqlens=cu, state=pool, slots=slots)
    y = layer.out(o, x)
    layer.check_out(orc, y, o, x, "prompts")
    S = []
    for i in range(n):
        r = slice(int(cu[i]), int(cu[i + 1]))
        ref = recurrence(*(t[r] for t in ins), torch.zeros(HV, DK, DV, device="cuda"), scale)
        check_recurrence(o[r], pool[slots[i]], ref, ins[0][r], scale,
                         8 * (-(-lens[i] // 64) + 1) * 2.0 ** -17, f"prompt {i}")
        S.append(pool[slots[i]].clone())
    assert bool((pool[1] == 7).all())

    # decode: one captured graph of the layer for a padded batch, replayed
    batch = 8
    row = torch.full((batch,), -1, dtype=torch.int32).cuda()
    row[[1, 4, 6]] = slots
    x1 = torch.zeros(batch, D, dtype=torch.bfloat16, device="cuda")
    before = pool.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def decode():
        ins = layer.project(x1)
        o = torch.zeros(batch, HV, DV, dtype=torch.bfloat16, device="cuda")
        nv.linear_attention_step(*ins, state=pool, slots=row, out=o)
        return ins, o, layer.out(o, x1)

    with torch.cuda.stream(s):
        decode()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ins1, o1, y1 = decode()
    pool.copy_(before)
    for t in range(steps):
        x1.copy_(gaussian(batch, D, 20 + t))
        g.replay()
        torch.cuda.synchronize()
        layer.check_out(orc, y1, o1, x1, f"step {t}")
        for i, b in enumerate((1, 4, 6)):
            r = slice(b, b + 1)
            ref = recurrence(*(u[r] for u in ins1), S[i], scale)
            check_recurrence(o1[r], pool[slots[i]], ref, ins1[0][r], scale, (DK + 8) * 2.0 ** -24,
                             f"step {t} of sequence {i}")
            S[i] = pool[slots[i]].clone()
        assert not o1[[0, 2, 3, 5, 7]].any() and bool((pool[1] == 7).all())
    assert nv.read_fault() == 0


def test_gate_sensitivity_reaches_the_layer_output(nv):
    """The command's errors of the layer's outputs and states against the same
    measurement with the recurrence in FP64. The recurrence's own error (below
    8 (chunks + 1) 2^-17 of a state, outputs rounded to bf16: 2^-8) is what may
    differ; it adds to both sides of a difference of two runs."""
    from nvfp4_w4a4_quantized_elem_b200 import gate_sensitivity, workloads
    rows = 192
    got = gate_sensitivity.measure(rows=rows, sigmas_a=(0.1, 0.005))
    cfg = workloads.gates()
    q, k, v = (t.cuda() for t in cfg.qkv(rows))
    x, w_b = cfg.x(rows).cuda(), cfg.w_b().cuda()
    X, Wb = nv.quantize(x), nv.quantize(w_b)
    for r in got:
        w_a = cfg.w_a(r["sigma_a"]).cuda()
        y = nv.gemm(X, nv.fuse_group([nv.quantize(w_a), Wb]), out_dtype=torch.float32).double()
        a, b = x.double() @ w_a.double().T, x.double() @ w_b.double().T
        zero = torch.zeros(cfg.heads, 128, 128, device="cuda")
        res = []
        for ya, yb in ((a, b), (y[:, :cfg.heads], y[:, cfg.heads:])):
            g, _, be = gate_sensitivity._gates(ya, yb, cfg.a_log().cuda(), cfg.dt_bias().cuda())
            res.append(recurrence(q, k, v, g, be, zero, 128 ** -0.5))
        for key, i in (("out", 0), ("state", 1)):
            ref = float((res[1][i] - res[0][i]).norm() / res[0][i].norm())
            assert abs(r[key] - ref) <= 2 * 2.0 ** -8 * (i == 0) + 2 * 8 * 4 * 2.0 ** -17, (key, r[key], ref)
        assert 0 < r["state"] < 1
