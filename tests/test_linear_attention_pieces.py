"""The bound that the chunked kernels are held to (la_bound.py) tells whether they
keep every bf16 piece of their FP32 operands: an emulation with all of them is
within it, one that drops any single piece is not. Without a GPU."""
import pytest

import la_bound

ALL = dict(s=2, t=2, at=2, a=2, x=3, u=3)
SIZES = [(64, 128, 32), (64, 64, 32), (37, 128, 32)]


def run(make, n, dk, dv, delta, **cut):
    q, k, v, g, beta, S = make(n, dk, dv, 1)
    beta = beta if delta else None
    ref = la_bound.chunk(q, k, v, g, beta, S, dk ** -0.5)
    o, S1 = la_bound.chunk(q, k, v, g, beta, S, dk ** -0.5, {**ALL, **cut})
    return max(la_bound.worst(o.float().bfloat16(), S1.float(), ref))


MAKE = (la_bound.usual, la_bound.one_hot, la_bound.cancelling)


@pytest.mark.parametrize("n,dk,dv", SIZES)
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("make", MAKE)
def test_every_piece_kept(make, delta, n, dk, dv):
    assert run(make, n, dk, dv, delta) <= 1.0


@pytest.mark.parametrize("n,dk,dv", SIZES)
@pytest.mark.parametrize("delta,piece", [(True, p) for p in ("s", "t", "at", "a", "x", "u")]
                         + [(False, p) for p in ("s", "a", "u")])
def test_one_piece_dropped_shows(piece, delta, n, dk, dv):
    assert max(run(make, n, dk, dv, delta, **{piece: ALL[piece] - 1}) for make in MAKE) > 2.0
