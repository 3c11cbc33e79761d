"""A NaN or an infinity in one token's inputs, prompt against the same tokens one
by one (the step kernel, in FP32): the chunks before the token's, other heads and
other sequences keep their bits; the tokens before it in its chunk and the other
columns of a value are still the recurrence's (within test_gpu_linear_attention's
tolerance: from that chunk on the head goes token by token); what the recurrence
makes of it afterwards is not finite in the prompt either."""
import math

import numpy as np
import pytest
import torch

from test_gpu_linear_attention import check, inputs, recurrence

pytestmark = pytest.mark.gpu

HK, HV, LENS = 2, 4, [100, 150, 70]
SEQ = 1   # the sequence with the bad token


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def prompt(nv, args, cu, state):
    return nv.linear_attention(*args, cu_seqlens=cu, state=state,
                               resume=torch.ones(len(LENS), dtype=torch.int32, device="cuda"))


def steps(nv, args, first, n, state):
    """The sequence's tokens one by one: (o, state)."""
    S, out = state[SEQ:SEQ + 1].clone(), []
    for t in range(first, first + n):
        out.append(nv.linear_attention_step(*(None if a is None else a[t:t + 1] for a in args), state=S))
    return torch.cat(out), S[0]


# 4 sequences' worth of few CTAs (16 columns each), and many (32, one buffer)
@pytest.mark.parametrize("heads", [HV, 96])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("what", ["q", "k", "v", "decay", "beta"])
@pytest.mark.parametrize("at,value", [(0, math.nan), (1, math.nan), (63, math.inf), (77, -math.inf), (78, math.nan),
                                      (149, math.nan)])
def test_one_bad_token(nv, at, value, what, delta, dk, heads):
    if what == "beta" and not delta:
        pytest.skip("no beta")
    if what == "decay" and value < 0:
        pytest.skip("-inf forgets")
    hk, dv = heads // 2, 64
    q, k, v, decay, beta = inputs(sum(LENS), hk, heads, dk, dv, 70 + at)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(LENS))), dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    pool = torch.randn(len(LENS), heads, dk, dv, generator=g).cuda()
    args = [q, k, v, decay, beta if delta else None]
    first, n = int(cu[SEQ]), LENS[SEQ]
    whole = slice(first, first + n)
    ro, rS, top = recurrence(q[whole], k[whole], v[whole], decay[whole], beta[whole] if delta else None,
                             pool[SEQ], dk ** -0.5)
    good_state = pool.clone()
    good = prompt(nv, args, cu, good_state)
    t = first + at
    if what in ("q", "k"):
        {"q": q, "k": k}[what][t, 1, 7] = value      # value heads 2 and 3
        bad_heads = [2, 3]
    elif what == "v":
        v[t, 2, 19] = value
        bad_heads = [2]
    else:
        {"decay": decay, "beta": beta}[what][t, 2] = value
        bad_heads = [2]
    state = pool.clone()
    got = prompt(nv, args, cu, state)
    torch.cuda.synchronize()
    assert nv.read_fault() == 0
    # chunks before the token's, other heads and sequences: the same bits
    touched = torch.zeros_like(got, dtype=torch.bool)
    touched[first + at // 64 * 64:first + n, bad_heads] = True
    assert torch.equal(got[~touched], good[~touched])
    changed = torch.zeros_like(state, dtype=torch.bool)
    changed[SEQ, bad_heads] = True
    assert torch.equal(state[~changed], good_state[~changed])
    # tokens before it, and other columns of a value: the recurrence
    rel, qs = 8 * 4 * 2.0 ** -17, q[whole].clone()
    qs[at, 1, 7] = 1.0
    check(got[whole][:at], None, (ro[:at], rS, top), qs[:at], dk ** -0.5, rel, "before the token")
    if what == "v":
        others = [c for c in range(dv) if c != 19]
        check(got[whole][..., others], state[SEQ][..., others], (ro[..., others], rS[..., others], top[..., others]),
              qs, dk ** -0.5, rel, "other columns")
    elif what == "q":
        rest = [i for i in range(n) if i != at]
        check(got[whole][rest], state[SEQ], (ro[rest], rS, top), qs[rest], dk ** -0.5, rel, "other tokens")
    # from the token on: not finite where the recurrence is not
    o, S = steps(nv, args, first, n, pool)
    here = got[first:first + n]
    assert not bool(torch.isfinite(here[~torch.isfinite(o)]).any())
    assert not bool(torch.isfinite(state[SEQ][~torch.isfinite(S)]).any())


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("what", ["k", "q"])
def test_products_that_overflow(nv, what, delta):
    """Finite keys and queries whose products are not: nothing finite comes out
    from there on, and nothing before is touched."""
    q, k, v, decay, beta = inputs(130, 1, 2, 128, 64, 80)
    beta = beta if delta else None
    good = nv.linear_attention(q, k, v, decay, beta)
    if what == "k":
        k[70:72] = 1e25
        q[71] = 1e25
    else:
        k[70], q[71] = 1e20, 3e20
        k[70, 0, ::2] *= -1
        q[71, 0, ::2] *= -1
    got = nv.linear_attention(q, k, v, decay, beta)
    assert torch.equal(got[:64], good[:64])
    ref = recurrence(q[:70], k[:70], v[:70], decay[:70], None if beta is None else beta[:70],
                     torch.zeros(2, 128, 64, device="cuda"), 128 ** -0.5)
    check(got[:70], None, ref, q[:70], 128 ** -0.5, 8 * 3 * 2.0 ** -17, "before the token")
    assert not bool(torch.isfinite(got[71]).any())
