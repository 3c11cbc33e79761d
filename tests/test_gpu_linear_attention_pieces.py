"""GPU tests of how exact the chunked linear-attention kernels are: every chunk
within la_bound's element-by-element bound (which no run that loses a piece of an
operand keeps: test_linear_attention_pieces.py), and a prompt of many chunks the
same, bit for bit, as its chunks one call after the other from the state each
leaves, so that the bound of one chunk holds for all of them."""
import pytest
import torch

import la_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def stacked(make, heads, n, dk, dv, seed):
    """`heads` different cases of `make` as the heads of one call."""
    cases = [make(n, dk, dv, seed + h) for h in range(heads)]
    q, k, v = (torch.stack([c[i] for c in cases], 1).cuda() for i in range(3))
    g, beta = (torch.stack([c[i] for c in cases], 1).float().cuda() for i in (3, 4))
    return cases, q, k, v, g, beta, torch.stack([c[5] for c in cases])[None].float().cuda()


# heads of 64 columns: 2 take the kernels of 16 columns per CTA, 48 and 80 those
# of 32, 80 more CTAs than the GPU has SMs
@pytest.mark.parametrize("heads,n", [(2, 1), (2, 2), (2, 37), (2, 64), (48, 64), (80, 63)])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("make", [la_bound.usual, la_bound.one_hot, la_bound.cancelling])
def test_a_chunk(nv, make, delta, dk, heads, n):
    dv, scale = 64, dk ** -0.5
    cases, q, k, v, g, beta, state = stacked(make, heads, n, dk, dv, 100 * n)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    o = nv.linear_attention(q, k, v, g, beta if delta else None, state=state, resume=one, scale=scale)
    torch.cuda.synchronize()
    assert nv.read_fault() == 0
    o, state = o.cpu(), state.cpu()
    for h, (qh, kh, vh, gh, bh, S) in enumerate(cases):
        ref = la_bound.chunk(qh, kh, vh, gh, bh if delta else None, S, scale)
        out, st = la_bound.worst(o[:, h], state[0, h], ref)
        assert out <= 1.0 and st <= 1.0, f"head {h}: outputs {out:.2f}, state {st:.2f} of the bound"


@pytest.mark.parametrize("heads", [2, 48, 80])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
def test_a_prompt_is_its_chunks(nv, delta, dk, heads):
    n, dv = 64 * 9 + 21, 64
    _, q, k, v, g, beta, state = stacked(la_bound.usual, heads, n, dk, dv, 7)
    beta = beta if delta else None
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    by_chunk = state.clone()
    o = nv.linear_attention(q, k, v, g, beta, state=state, resume=one)
    for t in range(0, n, 64):
        r = slice(t, min(t + 64, n))
        part = nv.linear_attention(q[r], k[r], v[r], g[r], None if beta is None else beta[r],
                                   state=by_chunk, resume=one)
        assert torch.equal(part, o[r]), f"tokens from {t}"
    assert torch.equal(by_chunk, state)
