"""What is measured of three operators around the W4A4 linear layer.

linear   y = act(W4A4(x, w) + bias) + residual, one call (nvfp4.linear with
         its epilogue): output projections that add the residual stream,
         biased and activated projections, from one token to a prefill.
prefill  linear attention with a decay for each head over packed prompts
         (nvfp4.linear_attention): the Gated DeltaNet update (delta rule) or,
         without beta, the plain decayed sum; states live in a pool of slots.
step     the same recurrence for single tokens (nvfp4.linear_attention_step),
         states updated in place.

``own`` False computes the plain forms in torch; True calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
# E2M1 values of the codes 0..15 (bit 3 is the sign)
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
CHUNK = 64


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decoding user: a GDN output projection (32 heads x 128) onto the
        # residual stream of width 5120
        dict(name="linear m1 out_proj", op="linear", m=1, n=5120, k=4096, act="none", bias=False, res=True),
        # a decode batch of odd size through a wide biased, activated projection
        dict(name="linear m37 up", op="linear", m=37, n=17408, k=5120, act="silu", bias=True, res=False),
        # a short chunk of prompt through the down projection (K is cut into slices)
        dict(name="linear m200 down", op="linear", m=200, n=5120, k=17408, act="none", bias=True, res=True),
        # prefill: the 8192-token projection of the benchmark with a full epilogue
        dict(name="linear m8192", op="linear", m=8192, n=5120, k=5120, act="gelu_tanh", bias=True, res=True),
        # one short prompt, few heads: latency
        dict(name="prefill 100", op="prefill", total=100, nseq=1, hk=4, hv=8, dk=128, dv=128, delta=True, resume=False),
        # one long prompt: 16 key heads shared by 32 value heads, as the qkv
        # group of width 8192 holds them
        dict(name="prefill 8192", op="prefill", total=8192, nseq=1, hk=16, hv=32, dk=128, dv=128, delta=True, resume=False),
        # a serving batch of ragged prompts, half of them continuing a state; 48 heads
        dict(name="prefill ragged", op="prefill", total=7777, nseq=23, hk=16, hv=48, dk=128, dv=128, delta=True, resume=True),
        # plain decayed linear attention (no delta rule), narrow keys
        dict(name="prefill plain", op="prefill", total=4096, nseq=3, hk=24, hv=24, dk=64, dv=128, delta=False, resume=True),
        # one decoding user
        dict(name="step b1", op="step", batch=1, hk=16, hv=32, dk=128, dv=128, delta=True),
        # a padded decode batch of odd size
        dict(name="step b37", op="step", batch=37, hk=16, hv=48, dk=128, dv=128, delta=True),
        # a large decode batch, plain decay
        dict(name="step b256 plain", op="step", batch=256, hk=24, hv=24, dk=64, dv=128, delta=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "prefill", "step"))
    if op == "linear":
        m = _log(rng, 1, 8192)
        n = 8 * _log(rng, 32, 2176)
        k = 32 * _log(rng, 8, 544)
        while m * n * k > 8192 * 5120 * 5120:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
                    bias=rng.random() < 0.6, res=rng.random() < 0.6)
    hk = rng.choice((1, 2, 4, 8, 16))
    heads = dict(hk=hk, hv=hk * rng.choice((1, 2, 3)), dk=rng.choice((64, 128, 128)),
                 dv=32 * rng.randint(1, 6), delta=rng.random() < 0.7)
    if op == "prefill":
        nseq = _log(rng, 1, 32)
        return dict(op=op, total=max(nseq, _log(rng, 1, 8192)), nseq=nseq, resume=rng.random() < 0.5, **heads)
    return dict(op=op, batch=_log(rng, 1, 256), **heads)


# ------------------------------------------------------------------ inputs --

def _swizzle(sf, rows, kb):
    """Row-major block scales [rows, kb] -> the 128x4 swizzled buffer."""
    kb4, r128 = -(-kb // 4) * 4, -(-rows // 128) * 128
    out = torch.zeros(r128 * kb4, dtype=torch.uint8, device=DEV)
    out[_sf_index(rows, kb)] = sf
    return out


def _sf_index(rows, kb):
    kb4 = -(-kb // 4) * 4
    r = torch.arange(rows, device=DEV)[:, None]
    c = torch.arange(kb, device=DEV)[None, :]
    return ((r // 128) * (kb4 // 4) + c // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4


def _lengths(case, seed):
    """Ragged lengths >= 1 that leave a few packed rows behind the last sequence."""
    total, nseq = case["total"], case["nseq"]
    used = total if nseq == 1 else max(nseq, total - total // 50)
    cuts = np.sort(np.random.RandomState(seed % (1 << 31)).permutation(used - 1)[: nseq - 1] + 1)
    return np.diff(np.concatenate(([0], cuts, [used]))).astype(np.int64)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = randn(m, k)
        x[:, torch.randint(k, (5,), generator=g, device=DEV)] *= 30.0  # outlier channels of the residual stream
        sf = torch.randint(0x58, 0x79, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8)
        return dict(case=case, x=x.bfloat16(),
                    codes=torch.randint(256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8),
                    sf=_swizzle(sf, n, k // 16),
                    w_global=torch.full((1,), 2688.0 / 0.1, device=DEV),
                    bias=randn(n).bfloat16() if case["bias"] else None,
                    res=randn(m, n).bfloat16() if case["res"] else None)

    prefill = case["op"] == "prefill"
    rows = case["total"] if prefill else case["batch"]
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    q = torch.nn.functional.normalize(randn(rows, hk, dk), dim=-1)
    k = torch.nn.functional.normalize(randn(rows, hk, dk), dim=-1)
    # q, k and v as a fused projection leaves them: columns of one [rows, ...] matrix
    qkv = torch.cat([q.flatten(1), k.flatten(1), randn(rows, hv * dv)], dim=1).bfloat16()
    # gates as Gated DeltaNet layers have them: A ~ U(1, 16), dt log-uniform in [1e-3, 0.1]
    a = 1.0 + 15.0 * torch.rand(hv, generator=g, device=DEV)
    dt = torch.exp(math.log(1e-3) + torch.rand(hv, generator=g, device=DEV) * math.log(100.0))
    decay = -a * torch.nn.functional.softplus(randn(rows, hv) + torch.log(torch.expm1(dt)))
    s = dict(case=case, q=qkv[:, : hk * dk].unflatten(1, (hk, dk)),
             k=qkv[:, hk * dk: 2 * hk * dk].unflatten(1, (hk, dk)),
             v=qkv[:, 2 * hk * dk:].unflatten(1, (hv, dv)), decay=decay,
             beta=torch.sigmoid(randn(rows, hv)) if case["delta"] else None,
             o=torch.zeros(rows, hv, dv, dtype=torch.bfloat16, device=DEV))
    n = case["nseq"] if prefill else rows
    pool = n + 2
    s["state"] = randn(pool, hv, dk, dv) * 0.3
    slots = torch.randperm(pool, generator=g, device=DEV)[:n].int()
    if prefill:
        lens = _lengths(case, seed)
        s["lens"] = lens
        s["cu"] = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device=DEV)
        s["resume"] = (torch.arange(n, device=DEV) % 2 == 0).int() if case["resume"] else None
    elif n >= 8:
        slots[n - n // 8:] = -1  # the padding rows of a captured batch
    s["slots"] = slots
    return s


# --------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        from nvfp4_w4a4_quantized_elem_b200 import nvfp4
        if op == "linear":
            c = s["case"]
            w = nvfp4.NVFP4Tensor(s["codes"], s["sf"], s["w_global"], c["n"], c["k"])
            if "ws" not in s:  # kept by the caller, as a serving loop keeps it
                s["ws"] = nvfp4.linear_workspace(c["m"], c["n"], c["k"])
            return nvfp4.linear(s["x"], w, bias=s["bias"], activation=c["act"], residual=s["res"],
                                workspace=s["ws"])
        if op == "prefill":
            o = nvfp4.linear_attention(s["q"], s["k"], s["v"], s["decay"], s["beta"], cu_seqlens=s["cu"],
                                       state=s["state"], slots=s["slots"], resume=s["resume"], out=s["o"])
        else:
            o = nvfp4.linear_attention_step(s["q"], s["k"], s["v"], s["decay"], s["beta"], state=s["state"],
                                            slots=s["slots"], out=s["o"])
        return {"o": o, "state": s["state"]}
    if op == "linear":
        return _plain_linear(s)
    (_plain_prefill if op == "prefill" else _plain_step)(s)
    return {"o": s["o"], "state": s["state"]}


def _round_e2m1(v):
    """Nearest E2M1 value, ties to the even code, saturating (torch.round is half-to-even)."""
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(torch.clamp_max(r, 6.0), v)


def _act(z, name):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    # quantize x: g = 2688 / amax; s = E4M3(amax_b / 6 * g); code = E2M1(x * (g / s)).
    # The divisors are tensors: torch divides by a number as a product with its inverse.
    x = s["x"].float()
    amax = x.abs().amax()
    g = torch.where(amax > 0, torch.full_like(amax, 2688.0) / amax, torch.ones_like(amax))
    xb = x.view(m, k // 16, 16)
    sx = torch.clamp_max(xb.abs().amax(-1) / torch.full_like(amax, 6.0) * g, 448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(sx > 0, g / sx, torch.zeros_like(sx))
    xq = (_round_e2m1(xb * r[..., None]) * sx[..., None]).view(m, k)
    grid = torch.tensor(GRID, device=DEV)
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).view(n, k).int()
    sw = s["sf"][_sf_index(n, k // 16)].view(torch.float8_e4m3fn).float()
    wq = (grid[codes].view(n, k // 16, 16) * sw[..., None]).view(n, k)
    y = (xq @ wq.T) / (g * s["w_global"])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.bfloat16()


def _plain_step(s):
    c = s["case"]
    group = c["hv"] // c["hk"]
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows].long()
    q = s["q"][rows].float().repeat_interleave(group, dim=1) * c["dk"] ** -0.5
    k = s["k"][rows].float().repeat_interleave(group, dim=1)
    v = s["v"][rows].float()
    S = s["state"][at] * torch.exp(s["decay"][rows])[..., None, None]
    u = v
    if s["beta"] is not None:
        u = s["beta"][rows][..., None] * (v - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["o"][rows] = (q[..., None] * S).sum(-2).bfloat16()
    s["state"][at] = S


def _plain_prefill(s):
    """The recurrence in chunks of 64 tokens: with G the running sum of the log
    decay in a chunk, U solves (I + L) U = beta (V - e^G K S0),
    L_tj = beta_t e^(G_t - G_j) k_t.k_j for j < t; O = e^G Q S0 + A U with
    A_tj = e^(G_t - G_j) q_t.k_j for j <= t; S = e^(G_end) S0 + K' U with
    K'_j = e^(G_end - G_j) k_j. Without beta, U = V."""
    c = s["case"]
    group, lens = c["hv"] // c["hk"], s["lens"]
    nch = -(-lens // CHUNK)
    first = np.concatenate(([0], np.cumsum(nch)[:-1]))
    start = np.concatenate(([0], np.cumsum(lens)[:-1]))
    seq = np.repeat(np.arange(len(lens)), nch)
    pos = np.arange(int(nch.sum())) - first[seq]
    tok = (start[seq] + pos * CHUNK)[:, None] + np.arange(CHUNK)
    ok = torch.from_numpy(tok < (start + lens)[seq][:, None]).to(DEV)
    tok = torch.from_numpy(np.minimum(tok, c["total"] - 1)).to(DEV)

    def chunks(x, rep=1):  # [T, H, d] -> [chunk, head, 64, d], rows past the end zero
        x = torch.where(ok[..., None, None], x[tok].float(), torch.zeros((), device=DEV))
        return x.repeat_interleave(rep, dim=2).transpose(1, 2)

    q, k, v = chunks(s["q"], group) * c["dk"] ** -0.5, chunks(s["k"], group), chunks(s["v"])
    gc = torch.cumsum(chunks(s["decay"][..., None])[..., 0].double(), -1)
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV))
    D = torch.exp(torch.where(low, gc[..., :, None] - gc[..., None, :], -math.inf)).float()
    eg, eend = torch.exp(gc).float()[..., None], torch.exp(gc[..., -1:]).float()[..., None]
    kd = (torch.exp(gc[..., -1:] - gc).float()[..., None] * k).transpose(-1, -2)
    A = (q @ k.transpose(-1, -2)) * D
    if s["beta"] is not None:
        beta = chunks(s["beta"][..., None])
        eye = torch.eye(CHUNK, device=DEV)
        N = -torch.tril((k @ k.transpose(-1, -2)) * D * beta, -1)
        T = eye + N
        for _ in range(5):  # (I - N)^-1 = (I + N)(I + N^2)(I + N^4)... ; N^64 = 0
            N = N @ N
            T = T + T @ N
        U0, W = T @ (beta * v), T @ (beta * eg * k)
    else:
        U0, W = v, None
    slots = s["slots"].long()
    S = s["state"][slots]
    S = S * (s["resume"] != 0)[:, None, None, None] if s["resume"] is not None else torch.zeros_like(S)
    o = torch.empty_like(v)
    for i in range(int(nch.max())):
        live = np.nonzero(nch > i)[0]
        at = torch.from_numpy(first[live] + i).to(DEV)
        live = torch.from_numpy(live).to(DEV)
        S0 = S[live]
        U = U0[at] if W is None else U0[at] - W[at] @ S0
        o[at] = eg[at] * (q[at] @ S0) + A[at] @ U
        S[live] = eend[at] * S0 + kd[at] @ U
    s["o"][tok[ok]] = o.transpose(1, 2)[ok].bfloat16()
    s["state"][slots] = S


# -------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        b = 2 * m * k + n * k // 2 + n * (k // 16) + 2 * m * n
        b += (2 * n if case["bias"] else 0) + (2 * m * n if case["res"] else 0)
        return {"bytes": b, "flops": 2 * m * n * k}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    per = 2 * (2 * hk * dk + 2 * hv * dv) + 4 * hv * (2 if case["delta"] else 1)
    state = 4 * hv * dk * dv
    # per token and head: the read-out and the rank-one update, and with the
    # delta rule the product with the key
    flops = hv * dk * dv * (6 if case["delta"] else 4)
    if case["op"] == "prefill":
        n, t = case["nseq"], case["total"]
        t = t if n == 1 else max(n, t - t // 50)
        reads = (n + 1) // 2 if case["resume"] else 0
        return {"bytes": t * per + (n + reads) * state, "flops": t * flops}
    b = case["batch"] if case["batch"] < 8 else case["batch"] - case["batch"] // 8
    return {"bytes": b * (per + 2 * state), "flops": b * flops}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"] == "linear" else _exact_recurrence(s)


def _exact_linear(s):
    """x quantized by the written convention (its FP32 steps are part of it),
    every product and sum in 64 bits."""
    c = s["case"]
    x = s["x"].float()
    amax = float(x.abs().max())
    g32 = np.float32(2688.0) / np.float32(amax) if amax > 0 else np.float32(1.0)
    blocks = x.reshape(c["m"], -1, 16)
    t = (blocks.abs().max(dim=-1).values / torch.tensor(6.0, device=DEV)) * torch.tensor(g32, device=DEV)
    # E4M3: 4 significant bits down to 2^-6, multiples of 2^-9 below
    t64 = t.double().clamp(max=448.0)
    e = torch.floor(torch.log2(t64.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > t64.clamp(min=2.0 ** -6), e - 1, e)
    unit = torch.exp2(e - 3)
    sc = (torch.round(t64 / unit) * unit).clamp(max=448.0)
    r = torch.where(sc == 0, torch.zeros_like(t), torch.tensor(g32, device=DEV) / sc.float())
    v = (blocks * r.unsqueeze(-1)).double()
    # nearest of the eight magnitudes, a tie to the even code
    mags = torch.tensor(GRID[:8], dtype=torch.float64, device=DEV)
    mids = (mags[1:] + mags[:-1]) / 2
    a = v.abs().contiguous()
    up, down = torch.bucketize(a, mids, right=True), torch.bucketize(a, mids, right=False)
    code = torch.where(up == down, up, torch.where(up % 2 == 0, up, down))
    xd = (mags[code] * torch.sign(v) * sc.unsqueeze(-1)).reshape(c["m"], c["k"])
    grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)
    wd = torch.empty(c["n"], c["k"], dtype=torch.float64, device=DEV)
    wd[:, 0::2] = grid[(s["codes"] % 16).long()]
    wd[:, 1::2] = grid[(s["codes"] // 16).long()]
    b = s["sf"][_sf_index(c["n"], c["k"] // 16)].int()
    ee, mm = (b >> 3).double(), (b & 7).double()
    ws = torch.where(ee == 0, mm * 2.0 ** -9, (1 + mm / 8) * torch.exp2(ee - 7))
    wd.view(c["n"], -1, 16).mul_(ws.unsqueeze(-1))
    z = xd @ wd.T / (float(g32) * float(s["w_global"]))
    if s["bias"] is not None:
        z += s["bias"].double()
    if c["act"] == "relu":
        z = z.clamp(min=0)
    elif c["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        z = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    elif c["act"] == "gelu_tanh":
        z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z if s["res"] is None else z + s["res"].double()


def _exact_recurrence(s):
    """Token by token: S <- e^g S; u = beta (v - S^T k), or v; S <- S + k u^T; o = scale S^T q."""
    c = s["case"]
    prefill = c["op"] == "prefill"
    rep = c["hv"] // c["hk"]
    if prefill:
        lens, first = s["lens"], s["cu"][:-1].long()
    else:
        lens, first = (s["slots"] >= 0).long().cpu().numpy(), torch.arange(c["batch"], device=DEV)
    order = torch.from_numpy(np.argsort(-lens, kind="stable")[: int((lens > 0).sum())]).to(DEV)
    first, slot = first[order], s["slots"].long()[order]
    sorted_lens = -np.sort(-lens)
    state = s["state"].double()
    S = state[slot].clone()
    if prefill:
        S = torch.zeros_like(S) if s["resume"] is None else torch.where((s["resume"][order] != 0)[:, None, None, None], S, 0.0)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    for t in range(int(sorted_lens[0])):
        n = int((sorted_lens > t).sum())
        at = first[:n] + t
        q = s["q"][at].double().repeat_interleave(rep, 1) / math.sqrt(c["dk"])
        k = s["k"][at].double().repeat_interleave(rep, 1)
        u = s["v"][at].double()
        cur = S[:n]
        cur *= torch.exp(s["decay"][at].double())[..., None, None]
        if s["beta"] is not None:
            u = s["beta"][at].double()[..., None] * (u - torch.einsum("nhk,nhkv->nhv", k, cur))
        cur += torch.einsum("nhk,nhv->nhkv", k, u)
        o[at] = torch.einsum("nhk,nhkv->nhv", q, cur)
    state[slot] = S
    return {"o": o, "state": state}
