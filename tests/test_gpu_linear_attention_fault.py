"""Linear attention's kernels giving up, without a fault: the self-test leaves one
CTA's first product or load unissued and limits every wait to 20 ms. The kernel
records its bit and returns; the state of the head and sequence it worked on
stays as it was, everything else gets its result, and the next call is right."""
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DV = 64


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def inputs(lens, hk, hv, dk):
    g = torch.Generator().manual_seed(sum(lens) + hv + dk)
    total = sum(lens)
    q, k = (torch.nn.functional.normalize(torch.randn(total, hk, dk, generator=g), dim=-1).bfloat16().cuda()
            for _ in range(2))
    v = torch.randn(total, hv, DV, generator=g).bfloat16().cuda()
    decay = -torch.rand(total, hv, generator=g).cuda()
    beta = torch.rand(total, hv, generator=g).cuda()
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    pool = torch.randn(len(lens), hv, dk, DV, generator=g).cuda()
    return q, k, v, decay, beta, cu, pool


# few heads: 16 columns of d_v per CTA; many: 32, and more CTAs than SMs
@pytest.mark.parametrize("hk,hv", [(1, 2), (8, 48)])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("kernel", [0, 1])
def test_a_stalled_cta(nv, kernel, delta, dk, hk, hv):
    lens = [130, 70]
    q, k, v, decay, beta, cu, pool = inputs(lens, hk, hv, dk)
    beta = beta if delta else None
    resume = torch.ones(2, dtype=torch.int32).cuda()
    ws = torch.empty(nv.linear_attention_workspace_bytes(sum(lens), 2, hk, hv, dk), dtype=torch.uint8, device="cuda")
    want_state = pool.clone()
    want = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=want_state, resume=resume, workspace=ws)
    ws.fill_(255)            # what an earlier call left is not taken for this one's
    state = pool.clone()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = DV // (16 if 2 * 2 * hv * (DV // 32) <= sms else 32)
    # the second chunk of the first sequence, head 1; the second sequence's head 1
    seq, head = (0, 1) if kernel == 0 else (1, 1)
    cta = hv + head if kernel == 0 else (seq * hv + head) * blocks
    torch.cuda.synchronize()
    assert nv.read_fault() == 0
    t0 = time.perf_counter()
    got = nv.selftest_linear_attention_stall(q, k, v, decay, beta, kernel=kernel, cta=cta, limit_ns=20_000_000,
                                             cu_seqlens=cu, state=state, resume=resume, workspace=ws)
    fault = nv.read_fault()
    assert time.perf_counter() - t0 < 5.0
    assert fault == 512 if kernel == 0 else fault and fault & (1024 | 2048) == fault, fault
    assert nv.read_fault() == 0
    cols = slice(None) if kernel == 0 else slice(0, DV // blocks)
    assert torch.equal(state[seq, head, :, cols], pool[seq, head, :, cols]), "a state moved on"
    others = torch.ones_like(state, dtype=torch.bool)
    others[seq, head, :, cols] = False
    assert torch.equal(state[others], want_state[others])
    rows = torch.ones_like(got, dtype=torch.bool)
    first, last = (0, 130) if kernel == 0 else (130, 200)
    rows[first:last, head, cols] = False   # the sequence's rows of that head are undefined
    assert torch.equal(got[rows], want[rows])
    # the context works on
    state = pool.clone()
    again = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=state, resume=resume, workspace=ws)
    assert torch.equal(again, want) and torch.equal(state, want_state)
    assert nv.read_fault() == 0


def test_a_cta_that_is_not_there_stalls_nothing(nv):
    q, k, v, decay, beta, cu, pool = inputs([70], 1, 2, 64)
    want = nv.linear_attention(q, k, v, decay, beta)
    for kernel in (0, 1):
        assert torch.equal(nv.selftest_linear_attention_stall(q, k, v, decay, beta, kernel=kernel, cta=999), want)
    assert nv.read_fault() == 0
