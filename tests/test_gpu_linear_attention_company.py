"""A sequence's results are the same bits alone and in any company, also where the
company's size chooses other kernels: alone a sequence's CTAs are few and take 16
columns of d_v each, in a batch 32, with one buffer of the factors where there
are more CTAs than SMs."""
import numpy as np
import pytest
import torch

from test_gpu_linear_attention import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


@pytest.mark.parametrize("n_seq", [12, 30])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
def test_alone_and_in_a_batch(nv, delta, dk, n_seq):
    hk, hv, dv = 2, 4, 64
    lens = ([70, 200, 1, 64, 33, 129, 128, 0, 400, 65] * 3)[:n_seq]
    q, k, v, decay, beta = inputs(sum(lens), hk, hv, dk, dv, dk + n_seq)
    beta = beta if delta else None
    cu = np.concatenate(([0], np.cumsum(lens)))
    g = torch.Generator().manual_seed(1)
    pool = torch.randn(n_seq, hv, dk, dv, generator=g).cuda()
    state, ones = pool.clone(), torch.ones(n_seq, dtype=torch.int32, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 2 * hv * dv // 32 <= sms < 2 * n_seq * hv * dv // 32     # other kernels
    assert (n_seq * hv * dv // 32 > sms) == (n_seq == 30)
    o = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                            state=state, resume=ones)
    for i in range(n_seq):
        r = slice(int(cu[i]), int(cu[i + 1]))
        S = pool[i:i + 1].clone()
        alone = nv.linear_attention(q[r], k[r], v[r], decay[r], None if beta is None else beta[r],
                                    state=S, resume=ones[:1])
        assert torch.equal(alone, o[r]) and torch.equal(S[0], state[i]), i
