"""One chunk (at most 64 tokens) of linear attention for one value head in FP64,
with a bound, element by element, on what the chunked kernels may be off by; and
an emulation of how they cut FP32 operands into bf16 pieces.

The bound, from the inputs alone (|.| element by element, first order; 1% on top
for the second). u24 = 2^-24 is FP32's half step.
- A sum on the tensor cores: bf16 products are exact, every addition is off by
  at most a step of a partial sum, so n nonzero terms give (n - 1) 2^-23 of the
  sum of their absolutes (one term: nothing). Column blocks of pieces are added
  in FP32, 2 u24 more.
- Pieces. Two rounded ones leave 2^-18 of the value (2^-9 twice): S, T, A, A T;
  of a product of two such operands the lower pieces' product is left out as
  well, 2^-18 again. Three truncated ones (24 bits) leave nothing: X and U~.
- e^x from two FP32 parts of x log2(e): their difference is rounded (2^-24 |x|),
  ex2 is off by 2^-22 of the value.
- T = (I + L)^-1: forward substitution in 16x16 blocks is off by 16 u24 |T||L||T|,
  each of the two doublings by two products on split tf32 tiles (three products
  of pieces with 10 bits, 2^-20 left, sums of up to 32 terms), and an error in
  the first reaches the second by way of |T||L|: eps = 2^-20 + 32 2^-23 in
  4 eps (W + |T||L| W), W = |T||L||T|. An error of L itself gives |T| dL |T|.
- Products and sums of single FP32 numbers: u24 each.
"""
import torch

U24, EX2 = 2.0 ** -24, 2.0 ** -22
LOG2E = 1.4426950408889634


def _mm(a, b, da=None, db=None, blocks=2):
    """(a @ b, bound on its error) for operands off by da and db."""
    terms = (a != 0).double() @ (b != 0).double()
    d = ((terms - 1).clamp(min=0) * 2.0 ** -23 + (blocks - 1) * 2 * U24) * (a.abs() @ b.abs())
    if da is not None:
        d = d + da @ b.abs()
    if db is not None:
        d = d + a.abs() @ db
    return a @ b, d


def _exp(x):
    """(e^x, bound), flushed to zero below 2^-126."""
    e = torch.exp(x)
    return e, e * (EX2 + U24 * x.abs() * LOG2E) + 2.0 ** -126


def pieces(x, n, rounded):
    """x as the sum of n bf16 pieces, rounded to nearest or cut off 8 bits at a time."""
    x = x.to(torch.float32)
    total = torch.zeros_like(x, dtype=torch.float64)
    for _ in range(n):
        if rounded:
            p = x.to(torch.bfloat16).to(torch.float32)
        else:
            p = (x.view(torch.int32) & -65536).view(torch.float32)
        total += p.double()
        x = x - p
    return total


def chunk(q, k, v, g, beta, S, scale, cut=None):
    """(o, S', bound of o, bound of S') of one chunk in FP64: q, k [n, d_k], v [n,
    d_v], g, beta [n] (None: plain), S [d_k, d_v]. With `cut`, how many pieces
    each operand keeps ("s", "t", "at", "a", "x", "u"), the results of the
    algorithm with operands in those pieces, and no bounds."""
    q, k, v, g, S = (t.double() for t in (q, k, v, g, S))
    n = q.shape[0]
    keep = (lambda x, what, rounded: x) if cut is None else (
        lambda x, what, rounded: pieces(x, cut[what], rounded))
    G = torch.cumsum(g.clamp(min=-1000.0), 0)
    low = torch.tril(torch.ones(n, n, dtype=torch.bool))
    D, dD = _exp(torch.where(low, G[:, None] - G[None, :], torch.zeros(())))
    D, dD = D * low, dD * low
    eg, deg = (t[:, None] for t in _exp(G))
    er, der = (t[:, None] for t in _exp(G[-1] - G))
    ea, dea = _exp(G[-1])

    Sp = keep(S, "s", True)
    KS, dKS = _mm(k, Sp, db=2.0 ** -18 * S.abs())
    QS, dQS = _mm(q, Sp, db=2.0 ** -18 * S.abs())
    P, dP = _mm(q, k.T, blocks=1)
    A, dA = D * P, D * dP + (dD + U24 * D) * P.abs()
    A2 = 2.0 ** -18 * A.abs()
    if beta is not None:
        b = beta.double()[:, None]
        KK, dKK = _mm(k, k.T, blocks=1)
        strict = torch.tril(low, -1)
        L = b * D * KK * strict
        dL = strict * b * (D * dKK + (dD + 2 * U24 * D) * KK.abs())
        T = torch.linalg.solve_triangular(torch.eye(n, dtype=torch.float64) + L,
                                          torch.eye(n, dtype=torch.float64), upper=False)
        aT, aL = T.abs(), L.abs()
        W = aT @ aL @ aT
        eps = 2.0 ** -20 + 32 * 2.0 ** -23
        dT = 16 * U24 * W + 4 * eps * (W + aT @ aL @ W) + aT @ dL @ aT
        # A T from pieces of both, itself in pieces
        AT, dAT = _mm(keep(A, "a", True), keep(T, "t", True), dA + A2, dT + 2.0 ** -18 * aT)
        dAT = dAT + 2.0 ** -18 * (A.abs() @ aT) + 2.0 ** -18 * AT.abs()
        X = b * (v - eg * KS)
        dX = b * (eg * dKS + deg * KS.abs()) + 3 * U24 * b * (v.abs() + eg * KS.abs())
        Xp = keep(X, "x", False)
        Ut, dU = _mm(keep(T, "t", True), Xp, dT + 2.0 ** -18 * aT, dX, blocks=4)
        AU, dAU = _mm(keep(AT, "at", True), Xp, dAT, dX, blocks=4)
    else:
        Ut, dU = v, torch.zeros_like(v)
        AU, dAU = _mm(keep(A, "a", True), v, dA + A2)
    Uw = er * Ut
    dUw = er * dU + (der + U24 * er) * Ut.abs()
    KU, dKU = _mm(k.T, keep(Uw, "u", False), db=dUw, blocks=3)
    o = scale * (eg * QS + AU)
    S1 = ea * S + KU
    if cut is not None:
        return o, S1
    do = abs(scale) * (eg * dQS + deg * QS.abs() + dAU + 3 * U24 * (eg * QS.abs() + AU.abs())) + U24 * o.abs()
    do = 1.01 * do * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-36   # rounded to bf16
    dS = 1.01 * (dea * S.abs() + dKU + 2 * U24 * (ea * S.abs() + KU.abs())) + 1e-36
    return o, S1, do, dS


def worst(got_o, got_S, ref):
    """The largest error of outputs and of states, in units of their bounds."""
    o, S1, do, dS = ref
    return (float(((got_o.double() - o).abs() / do).max()),
            float(((got_S.double() - S1).abs() / dS).max()))


# Inputs on which each piece shows, of one head: (q, k, v, g, beta, S).
def gates(n, gen):
    return (-torch.exp(torch.randn(n, generator=gen) - 2.0),
            torch.sigmoid(torch.randn(n, generator=gen)))


def usual(n, dk, dv, seed):
    """As a layer has them."""
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.nn.functional.normalize(torch.randn(n, dk, generator=gen), dim=-1).bfloat16()
            for _ in range(2))
    g, beta = gates(n, gen)
    return (q, k, torch.randn(n, dv, generator=gen).bfloat16(), g, beta,
            torch.randn(dk, dv, generator=gen) * 0.3)


def one_hot(n, dk, dv, seed):
    """Every key another unit vector, no state: each row of the state is one
    product, e^(G_end - G_t) beta_t v_t, and nothing is lost but FP32's own steps."""
    q, k, v, g, beta, S = usual(n, dk, dv, seed)
    k = torch.eye(dk)[torch.randperm(dk, generator=torch.Generator().manual_seed(seed))[:n]].bfloat16()
    return q, k, v, g, beta, torch.zeros(dk, dv)


def cancelling(n, dk, dv, seed):
    """Keys in pairs k and -k + a little, with equal values and little forgetting,
    and queries whose parts meet nearly equal rows of the state with opposite
    signs: outputs far smaller than the terms they are the sum of."""
    gen = torch.Generator().manual_seed(seed)
    q, k, v, g, beta, S = usual(n, dk, dv, seed)
    k, v, q, g = k.clone(), v.clone(), q.clone(), g * 2.0 ** -10
    m = n // 2
    small = (torch.randn(m, dk, generator=gen) * 2.0 ** -14).bfloat16()
    k[1:2 * m:2] = (small - k[0:2 * m:2]).bfloat16()
    v[1:2 * m:2] = v[0:2 * m:2]
    beta = beta * 0 + 2.0 ** -8
    q[:, 1::2] = -q[:, 0::2]
    S = S.clone()
    S[1::2] = S[0::2] * (1 + 2.0 ** -9 * torch.randn(dk // 2, dv, generator=gen))
    k[:, 1::2] = k[:, 0::2] * -1
    return q, k, v, g, beta, S
