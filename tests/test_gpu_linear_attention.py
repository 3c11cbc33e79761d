"""GPU tests of linear attention with a decay for each head (news article
"Qwen3.8-27B最激进4bit量化开源…" §01: the gated delta rule of the recurrent
layers), prompts and single tokens, against the token-by-token recurrence in
FP64.

Tolerances. The step kernel works in FP32: the products with the state are
sums of d_k terms, the update adds a few half steps, so a column of the state
is within (d_k + 8) 2^-24 of its scale, which is the largest norm it went
through plus |v|. The chunked kernels split FP32 operands into two bf16
pieces: the rest is at most 2^-18 of the value and the dropped product of two
rests as much again, so each product is within 2^-17 of the product of the
operands' norms; four products per chunk (scores, factors, U, update) stand
one behind the other, and an update with beta |k|^2 <= 2 does not stretch what
is already there, so errors add up over the chunks: 8 (chunks + 1) 2^-17 of
the same scale leaves a factor of two for the FP32 sums. An output is a column
of the state times scale |q|, rounded to bf16: 2^-8 of itself in addition.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_w4a4_quantized_elem_b200 import build, nvfp4
    build.build()
    return nvfp4


def inputs(rows, hk, hv, dk, dv, seed, strong=False):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.nn.functional.normalize(torch.randn(rows, hk, dk, generator=g), dim=-1)
            for _ in range(2))
    qkv = torch.cat([q.flatten(1), k.flatten(1), torch.randn(rows, hv * dv, generator=g)], 1)
    qkv = qkv.to(torch.bfloat16).cuda()  # columns of one matrix, as a fused projection leaves them
    decay = -torch.exp(torch.randn(rows, hv, generator=g) * (3.0 if strong else 1.0) - 2.0)
    beta = torch.sigmoid(torch.randn(rows, hv, generator=g))
    return (qkv[:, :hk * dk].unflatten(1, (hk, dk)),
            qkv[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk)),
            qkv[:, 2 * hk * dk:].unflatten(1, (hv, dv)), decay.cuda(), beta.cuda())


def recurrence(q, k, v, decay, beta, S, scale):
    """FP64, token by token: (o, S, scale of each state column)."""
    rep = v.shape[1] // q.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = S.double().clone()
    o = torch.zeros_like(v)
    top = S.norm(dim=1)
    for t in range(v.shape[0]):
        S = S * torch.exp(decay[t].double())[:, None, None]
        u = v[t]
        if beta is not None:
            u = beta[t].double()[:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][:, :, None] * u[:, None, :]
        o[t] = scale * torch.einsum("hk,hkv->hv", q[t], S)
        top = torch.maximum(top, S.norm(dim=1) + v[t].abs())
    return o, S, top


def check(o, S, ref, q, scale, rel, what):
    ro, rS, top = ref
    qn = q.double().norm(dim=-1).repeat_interleave(ro.shape[1] // q.shape[1], 1)
    tol = rel * scale * qn[..., None] * top
    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ro.abs() + 1e-30
    worst = float(((o.double() - ro).abs() / tol).max()) if o.numel() else 0.0
    assert worst <= 1.0, f"{what}: output {worst:.2f} of the tolerance"
    if S is not None:
        worst = float(((S.double() - rS).norm(dim=1) / (rel * top + 1e-30)).max())
        assert worst <= 1.0, f"{what}: state {worst:.2f} of the tolerance"


def run_prompts(nv, lens, hk, hv, dk, dv, delta, resume, seed, strong=False, behind=3):
    total = sum(lens) + behind
    q, k, v, decay, beta = inputs(total, hk, hv, dk, dv, seed, strong)
    for x in (q, k, v, decay, beta):
        x[sum(lens):] = float("nan")  # behind the last sequence: never read
    beta = beta if delta else None
    n = len(lens)
    g = torch.Generator().manual_seed(seed + 1)
    pool = torch.randn(n + 2, hv, dk, dv, generator=g).cuda() * 0.3
    before = pool.clone()
    slots = torch.randperm(n + 2, generator=g)[:n].int().cuda()
    flags = torch.tensor([(i % 2 == 0) * 7 for i in range(n)], dtype=torch.int32).cuda() if resume else None
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    out = torch.full((total, hv, dv), 9.0, dtype=torch.bfloat16, device="cuda")
    scale = dk ** -0.5
    nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=pool, slots=slots, resume=flags, out=out)
    torch.cuda.synchronize()
    assert nv.read_fault() == 0
    at = 0
    for i, length in enumerate(lens):
        s = int(slots[i])
        S0 = before[s] if resume and i % 2 == 0 else torch.zeros_like(before[s])
        r = slice(at, at + length)
        ref = recurrence(q[r], k[r], v[r], decay[r], None if beta is None else beta[r], S0, scale)
        rel = 8 * (-(-length // 64) + 1) * 2.0 ** -17
        check(out[r], pool[s], ref, q[r], scale, rel, f"sequence {i} of {lens}")
        at += length
    assert bool((out[at:] == 9).all()), "rows behind the last sequence changed"
    free = sorted(set(range(n + 2)) - set(slots.tolist()))
    assert torch.equal(pool[free], before[free]), "another slot changed"


@pytest.mark.parametrize("lens", [[1], [2], [63], [64], [65], [300], [5, 0, 64, 1, 129, 63]])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32)])
def test_prompts(nv, lens, delta, dk, dv):
    run_prompts(nv, lens, 2, 4, dk, dv, delta, True, 5 + sum(lens))


@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 128, 32), (2, 6, 64, 96), (3, 3, 128, 64), (1, 5, 128, 160)])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("resume", [True, False])
def test_head_layouts(nv, hk, hv, dk, dv, delta, resume):
    run_prompts(nv, [130, 7], hk, hv, dk, dv, delta, resume, hk + hv + dv)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 256)])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("strong", [True, False])
def test_many_sequences(nv, dk, dv, delta, strong):
    """More CTAs of the chain than the GPU holds at a time, lengths around whole
    chunks."""
    lens = [1, 64, 65, 200, 63, 0, 128, 129, 2, 70] * 4
    run_prompts(nv, lens, 2, 4, dk, dv, delta, True, 31 + dv, strong=strong)


@pytest.mark.parametrize("delta", [True, False])
def test_strong_and_vanishing_decays(nv, delta):
    """Decays from e^-1000 to 1 next to one another in a chunk."""
    run_prompts(nv, [200, 64], 2, 2, 128, 64, delta, True, 3, strong=True)


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("where", [0, 1, 63, 64, 100])
def test_decay_of_zero_forgets(nv, delta, where):
    """g = -inf at a token: what stands before it has no part in what follows."""
    q, k, v, decay, beta = inputs(150, 1, 2, 128, 32, 4)
    beta = beta if delta else None
    decay[where] = float("-inf")
    state = torch.randn(1, 2, 128, 32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    S0 = state[0].clone()
    o = nv.linear_attention(q, k, v, decay, beta, state=state, resume=one)
    ref = recurrence(q, k, v, decay, beta, S0, 128 ** -0.5)
    check(o, state[0], ref, q, 128 ** -0.5, 8 * 4 * 2.0 ** -17, "forgetting")
    tail = slice(where, 150)
    alone = nv.linear_attention(q[tail], k[tail], v[tail], decay[tail],
                                None if beta is None else beta[tail])
    ref2 = recurrence(q[tail], k[tail], v[tail], decay[tail], None if beta is None else beta[tail],
                      torch.zeros_like(S0), 128 ** -0.5)
    check(alone, state[0], ref2, q[tail], 128 ** -0.5, 8 * 4 * 2.0 ** -17, "the tail alone")


def test_repeated_keys_and_full_write_strength(nv):
    """beta = 1, the same unit key throughout, no decay: every write replaces
    the one before, the worst case for the chunk's triangular inverse."""
    q, k, v, decay, beta = inputs(200, 1, 1, 128, 32, 6)
    k[:] = 0.0
    k[:, :, 3] = 1.0
    q[:] = k
    decay[:] = 0.0
    beta[:] = 1.0
    state = torch.empty(1, 1, 128, 32, device="cuda")
    o = nv.linear_attention(q, k, v, decay, beta, state=state, scale=1.0)
    ref = recurrence(q, k, v, decay, beta, torch.zeros(1, 128, 32, device="cuda"), 1.0)
    check(o, state[0], ref, q, 1.0, 8 * 5 * 2.0 ** -17, "repeated keys")
    assert torch.equal(o[:, 0], v[:, 0]), "each write is read back exactly"


def test_sequences_do_not_touch_one_another(nv):
    """Bits of a sequence are the same alone, in any company and order; NaN in
    a neighbour stays there."""
    lens = [70, 200, 1, 64, 33]
    total = sum(lens)
    q, k, v, decay, beta = inputs(total, 2, 4, 128, 64, 8)
    cu = np.concatenate(([0], np.cumsum(lens)))
    bad = slice(int(cu[1]), int(cu[2]))
    for x in (q, k, v, decay, beta):
        x[bad] = float("nan")
    state = torch.full((5, 4, 128, 64), float("nan"), device="cuda")
    o = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                            state=state)
    for i in (0, 2, 3, 4):
        r = slice(int(cu[i]), int(cu[i + 1]))
        S = torch.empty(1, 4, 128, 64, device="cuda")
        alone = nv.linear_attention(q[r], k[r], v[r], decay[r], beta[r], state=S)
        assert torch.equal(alone, o[r]) and torch.equal(S[0], state[i]), i
        assert bool(torch.isfinite(alone).all()) and bool(torch.isfinite(S).all())


def test_slots_outside_the_pool_or_named_twice(nv):
    lens = [66, 10, 70, 5]
    q, k, v, decay, beta = inputs(sum(lens), 1, 2, 64, 32, 9)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    pool = torch.randn(3, 2, 64, 32, device="cuda")
    before = pool.clone()
    slots = torch.tensor([1, -1, 1, 3], dtype=torch.int32).cuda()
    ones = torch.ones(4, dtype=torch.int32).cuda()
    o = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=pool, slots=slots, resume=ones)
    S = before[1:2].clone()
    first = nv.linear_attention(q[:66], k[:66], v[:66], decay[:66], beta[:66], state=S, resume=ones[:1])
    rest = [nv.linear_attention(q[a:b], k[a:b], v[a:b], decay[a:b], beta[a:b])
            for a, b in ((66, 76), (76, 146), (146, 151))]
    assert torch.equal(o, torch.cat([first, *rest]))
    assert torch.equal(pool[1], S[0])
    assert torch.equal(pool[[0, 2]], before[[0, 2]])


def test_offsets_that_leave_the_buffer_are_cut(nv):
    """Bad offsets are cut to the packed rows: nothing outside is read or written."""
    q, k, v, decay, beta = inputs(100, 1, 1, 64, 32, 10)
    guard = torch.full((300, 1, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    out = guard[100:200]
    cu = torch.tensor([-50, 40, 100000], dtype=torch.int32).cuda()
    nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, out=out)
    good = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=torch.tensor([0, 40, 100], dtype=torch.int32).cuda())
    assert torch.equal(out, good)
    assert bool((guard[:100] == 5).all()) and bool((guard[200:] == 5).all())


@pytest.mark.parametrize("delta", [True, False])
def test_prompt_in_pieces_and_single_tokens(nv, delta):
    """A prompt whole, in two pieces, and as a prompt and single tokens."""
    n, cut, hk, hv, dk, dv = 150, 90, 2, 4, 128, 64
    q, k, v, decay, beta = inputs(n, hk, hv, dk, dv, 12)
    b = (lambda r: beta[r]) if delta else (lambda r: None)
    ref = recurrence(q, k, v, decay, b(slice(None)), torch.zeros(hv, dk, dv, device="cuda"), dk ** -0.5)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    S = torch.zeros(2, hv, dk, dv, device="cuda")
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    head, tail = slice(0, cut), slice(cut, n)
    o1 = nv.linear_attention(q[head], k[head], v[head], decay[head], b(head), state=S, slots=slot)
    S2 = S.clone()
    o2 = nv.linear_attention(q[tail], k[tail], v[tail], decay[tail], b(tail), state=S, slots=slot, resume=one)
    rel = 8 * 4 * 2.0 ** -17
    check(torch.cat([o1, o2]), S[1], ref, q, dk ** -0.5, rel, "two pieces")
    steps = [nv.linear_attention_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], decay[t:t + 1],
                                      b(slice(t, t + 1)), state=S2, slots=slot) for t in range(cut, n)]
    check(torch.cat([o1, *steps]), S2[1], ref, q, dk ** -0.5, rel + 60 * 2.0 ** -17, "prompt and steps")
    assert not S[0].any() and not S2[0].any()


@pytest.mark.parametrize("batch", [1, 5, 130])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 64, 32), (2, 4, 128, 128), (2, 6, 128, 96)])
@pytest.mark.parametrize("delta", [True, False])
def test_step(nv, batch, hk, hv, dk, dv, delta):
    q, k, v, decay, beta = inputs(batch, hk, hv, dk, dv, batch + dv, strong=True)
    beta = beta if delta else None
    if batch > 4:
        decay[2] = float("-inf")
    g = torch.Generator().manual_seed(batch)
    pool = torch.randn(batch + 3, hv, dk, dv, generator=g).cuda()
    before = pool.clone()
    slots = torch.randperm(batch + 3, generator=g)[:batch].int()
    if batch > 4:
        slots[1], slots[4] = -1, batch + 3  # padding: outside the pool on either side
        for x in (q, k, v, decay):
            x[1] = float("nan")
    out = torch.full((batch, hv, dv), 9.0, dtype=torch.bfloat16, device="cuda")
    nv.linear_attention_step(q, k, v, decay, beta, state=pool, slots=slots.cuda(), out=out)
    live = [i for i in range(batch) if 0 <= slots[i] < batch + 3]
    for i in live[:12]:
        r = slice(i, i + 1)
        ref = recurrence(q[r], k[r], v[r], decay[r], None if beta is None else beta[r],
                         before[slots[i]], dk ** -0.5)
        check(out[r], pool[slots[i]], ref, q[r], dk ** -0.5, (dk + 8) * 2.0 ** -24, f"row {i}")
    dead = [i for i in range(batch) if i not in live]
    assert bool((out[dead] == 9).all()), "a padding row changed"
    free = sorted(set(range(batch + 3)) - {int(slots[i]) for i in live})
    assert torch.equal(pool[free], before[free])


def test_step_rows_of_one_slot_are_taken_in_order(nv):
    hk, hv, dk, dv = 1, 2, 128, 64
    q, k, v, decay, beta = inputs(6, hk, hv, dk, dv, 20)
    pool = torch.randn(2, hv, dk, dv, device="cuda")
    one = pool.clone()
    slots = torch.tensor([1, 0, 1, -1, 1, 0], dtype=torch.int32).cuda()
    out = torch.zeros(6, hv, dv, dtype=torch.bfloat16, device="cuda")
    nv.linear_attention_step(q, k, v, decay, beta, state=pool, slots=slots, out=out)
    for i in (0, 1, 2, 4, 5):
        r = slice(i, i + 1)
        o = nv.linear_attention_step(q[r], k[r], v[r], decay[r], beta[r], state=one, slots=slots[r].contiguous())
        assert torch.equal(o, out[r]), i
    assert torch.equal(pool, one)
    assert not out[3].any()


def test_another_stream_and_graph_replay(nv):
    """On a stream of its own, and captured: one graph that prefills, steps and
    is replayed on new inputs and offsets."""
    hk, hv, dk, dv = 1, 2, 128, 64
    q, k, v, decay, beta = inputs(200, hk, hv, dk, dv, 21)
    cu = torch.tensor([0, 120, 200], dtype=torch.int32).cuda()
    state = torch.zeros(2, hv, dk, dv, device="cuda")
    ws = torch.empty(nv.linear_attention_workspace_bytes(200, 2, hk, hv, dk), dtype=torch.uint8, device="cuda")
    out, out1 = torch.empty(200, hv, dv, dtype=torch.bfloat16, device="cuda"), torch.empty(2, hv, dv, dtype=torch.bfloat16, device="cuda")

    def both(**kw):
        nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=state, out=out, **kw)
        nv.linear_attention_step(q[:2], k[:2], v[:2], decay[:2].contiguous(), beta[:2].contiguous(),
                                 state=state, out=out1, stream=kw.get("stream"))

    both()
    want = out.clone(), out1.clone(), state.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x in (out, out1, state):
        x.zero_()
    torch.cuda.synchronize()
    both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, out1, state)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(workspace=ws)
    v2 = inputs(200, hk, hv, dk, dv, 22)[2]
    v.copy_(v2)
    cu.copy_(torch.tensor([0, 30, 190], dtype=torch.int32))
    both()
    want = out.clone(), out1.clone(), state.clone()
    out.zero_()
    out[190:] = want[0][190:]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, out1, state)))
    assert nv.read_fault() == 0


@pytest.mark.parametrize("delta", [True, False])
def test_no_tokens(nv, delta):
    """A call without tokens: fresh sequences leave a zero state, resumed ones
    theirs."""
    hk, hv, dk, dv = 1, 2, 64, 32
    q, k, v, decay, beta = inputs(0, hk, hv, dk, dv, 1)
    state = torch.randn(3, hv, dk, dv, device="cuda")
    before = state.clone()
    cu = torch.zeros(3, dtype=torch.int32).cuda()
    out = nv.linear_attention(q, k, v, decay, beta if delta else None, cu_seqlens=cu, state=state,
                              resume=torch.tensor([0, 1], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert out.shape == (0, hv, dv) and nv.read_fault() == 0
    assert not state[0].any() and torch.equal(state[1:], before[1:])
    assert nv.linear_attention_step(q, k, v, decay, beta, state=state).shape == (0, hv, dv)


def test_two_calls_at_once(nv):
    """Calls on two streams, each with its own workspace and states, again and
    again: the results are those of calls one after the other."""
    shapes = [([900, 65, 400], 2, 4, 128, 64), ([64, 1500], 3, 6, 64, 96)]
    work = []
    for i, (lens, hk, hv, dk, dv) in enumerate(shapes):
        args = inputs(sum(lens), hk, hv, dk, dv, 40 + i)
        cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
        pool = torch.zeros(len(lens), hv, dk, dv, device="cuda")
        ws = torch.empty(nv.linear_attention_workspace_bytes(sum(lens), len(lens), hk, hv, dk),
                         dtype=torch.uint8, device="cuda")
        out = torch.empty(sum(lens), hv, dv, dtype=torch.bfloat16, device="cuda")
        kw = dict(cu_seqlens=cu, state=pool, out=out, workspace=ws)
        nv.linear_attention(*args, **kw)
        torch.cuda.synchronize()
        work.append((args, kw, out.clone(), pool.clone(), torch.cuda.Stream()))
    for _ in range(20):
        for args, kw, _, _, s in work:
            nv.linear_attention(*args, stream=s, **kw)
    torch.cuda.synchronize()
    assert nv.read_fault() == 0
    for _, kw, out, pool, _ in work:
        assert torch.equal(kw["out"], out) and torch.equal(kw["state"], pool)


@pytest.mark.parametrize("delta", [True, False])
def test_not_a_number_stays_in_its_sequence_and_head(nv, delta):
    lens, hk, hv, dk, dv = [100, 70, 130], 2, 4, 128, 64
    q, k, v, decay, beta = inputs(sum(lens), hk, hv, dk, dv, 50)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    state = torch.zeros(3, hv, dk, dv, device="cuda")
    beta = beta if delta else None
    want = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=state)
    want_state = state.clone()
    v[165, 2, 5] = float("nan")      # token 65 of the second sequence
    got = nv.linear_attention(q, k, v, decay, beta, cu_seqlens=cu, state=state)
    clean = torch.ones_like(got, dtype=torch.bool)
    clean[164:170, 2] = False        # its second chunk
    assert torch.equal(got[clean], want[clean])
    assert bool(torch.isnan(got[165:170, 2, 5]).all()) and bool(torch.isnan(state[1, 2, :, 5]).all())
    keep = torch.ones_like(state, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(state[keep], want_state[keep])


def test_binding_refuses_a_workspace_elsewhere(nv):
    args = inputs(70, 1, 1, 64, 32, 60)
    need = nv.linear_attention_workspace_bytes(70, 1, 1, 1, 64)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            nv.linear_attention(*args, workspace=ws)
    with pytest.raises(nv.NVFP4Error):
        nv.linear_attention(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("hv,dv", [(24, 128), (12, 128), (4, 64)])
@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("delta", [True, False])
def test_long_sequences(nv, dk, hv, dv, delta):
    """Many chunks in a row, with more chains than SMs, about as many, and few."""
    run_prompts(nv, [900, 1025], 2, hv, dk, dv, delta, True, dk + hv)
