"""GPU tests of ``stream=``: a call that makes its own output and workspace,
while the current stream still works on blocks of the same sizes that were
freed there (an allocator that handed those out, or a zero fill queued behind
that work, would spoil the results)."""
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


def busy(sizes):
    """Work on the current stream, then blocks of these sizes filled behind it and freed."""
    a = torch.ones(4096, 4096, device="cuda")
    for _ in range(20):
        a = (a @ a) * 2.0 ** -12
    for n in sizes:
        t = torch.empty(n, dtype=torch.uint8, device="cuda")
        t.fill_(255)
        del t


def again(call, sizes):
    """call(stream) on a side stream over a busy current one: what it gives, three times."""
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        busy(sizes)
        got = call(s)
        s.synchronize()
        # read on the caller's stream once it is ordered behind `s`
        torch.cuda.current_stream().wait_stream(s)
        yield got


@pytest.mark.parametrize("m,n,k", [(1, 640, 4096), (37, 640, 4096), (200, 512, 8192)])
@pytest.mark.parametrize("epilogue", [True, False])
def test_linear(nv, orc, m, n, k, epilogue):
    g = torch.Generator().manual_seed(m)
    x = torch.randn((m, k), generator=g).to(torch.bfloat16).cuda()
    w = upload(orc.quantize(bits((torch.randn((n, k), generator=g) / math.sqrt(k)).to(torch.bfloat16))))
    bias = torch.randn(n, generator=g).to(torch.bfloat16).cuda()
    kw = dict(bias=bias, activation="silu") if epilogue else {}
    want = nv.linear(x, w, workspace=nv.linear_workspace(m, n, k), **kw)
    sizes = (nv.linear_workspace_bytes(m, n, k), 2 * m * n)
    for got in again(lambda s: nv.linear(x, w, stream=s, **kw), sizes):
        assert torch.equal(got, want)
    A = nv.quantize(x)
    want = nv.gemm(A, w, **kw)
    for got in again(lambda s: nv.gemm(A, w, stream=s, **kw), sizes):
        assert torch.equal(got, want)
    for got in again(lambda s: nv.quantize(x, stream=s), (m * k // 2, nv.sf_bytes(m, k), 16384)):
        assert torch.equal(got.codes, A.codes) and torch.equal(got.global_scale, A.global_scale)
    assert nv.read_fault() == 0


@pytest.mark.parametrize("delta", [True, False])
def test_linear_attention(nv, delta):
    lens, hk, hv, dk, dv = [130, 70, 64], 2, 4, 128, 64
    total, g = sum(lens), torch.Generator().manual_seed(3)
    q, k = (torch.nn.functional.normalize(torch.randn(total, hk, dk, generator=g), dim=-1).bfloat16().cuda()
            for _ in range(2))
    v = torch.randn(total, hv, dv, generator=g).bfloat16().cuda()
    decay = -torch.rand(total, hv, generator=g).cuda()
    beta = torch.rand(total, hv, generator=g).cuda() if delta else None
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    want = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu)
    sizes = (nv.linear_attention_workspace_bytes(total, 3, hk, hv, dk), 2 * total * hv * dv)
    for got in again(lambda s: nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, stream=s), sizes):
        assert torch.equal(got, want)
    pool = torch.randn(total, hv, dk, dv, generator=g).cuda()
    want = nv.linear_attention_step(q, k, v, decay, beta, state=pool.clone())
    for got in again(lambda s: nv.linear_attention_step(q, k, v, decay, beta, state=copy(pool, s), stream=s),
                     (2 * total * hv * dv,)):
        assert torch.equal(got, want)
    assert nv.read_fault() == 0


def copy(t, stream):
    """A copy of `t` that belongs to `stream`."""
    with torch.cuda.stream(stream):
        return t.clone()


def test_captured_on_a_forked_stream(nv, orc):
    """Calls given a stream that a capture forked to, with buffers of their own:
    the graph's replays give what the calls give."""
    g = torch.Generator().manual_seed(9)
    n, k = 640, 1024
    x = torch.randn((37, k), generator=g).to(torch.bfloat16).cuda()
    w = upload(orc.quantize(bits((torch.randn((n, k), generator=g) * 0.05).to(torch.bfloat16))))
    bias = torch.randn(n, generator=g).to(torch.bfloat16).cuda()
    q, kk, v = (torch.randn(90, 2, 64, generator=g).to(torch.bfloat16).cuda() * 0.1 for _ in range(3))
    decay, beta = -torch.rand(90, 2, generator=g).cuda(), torch.rand(90, 2, generator=g).cuda()
    s = torch.cuda.Stream()

    def both(stream):
        return (nv.linear(x, w, bias=bias, activation="gelu", stream=stream),
                nv.linear_attention(q, kk, v, decay, beta, stream=stream))

    both(None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = both(s)
        torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2):
        x.copy_(torch.randn((37, k), generator=g).to(torch.bfloat16))
        v.copy_(torch.randn(90, 2, 64, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both(None)))
    assert nv.read_fault() == 0
