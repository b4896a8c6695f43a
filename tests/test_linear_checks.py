"""The comparisons of linear_checks.py accept the chunked form with its documented
roundings and reject mistakes planted in it.  Host only: the chunked form below is
written here, in float64 with bf16 operands, and compared with the oracle."""
import numpy as np
import pytest
import torch

import oracle
from tests.linear_checks import CHUNK, OUT_BOUND, dw_bound, state_bound, worst_chunk, worst_state

D = 128


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def parts(x, n):
    """x as the sum of n bf16 parts, as far as they reach."""
    x = np.float32(x).astype(np.float64)
    out = np.zeros_like(x)
    for _ in range(n):
        out += bf16(x - out)
    return out


def make(T, seed=5):
    rng = np.random.default_rng(seed)
    return [bf16(rng.standard_normal((T, 1, D))) for _ in range(3)]


def chunked(q, k, v, g, *, value_parts=3, skip=None, stale=None, diagonal=None):
    """One head's outputs [T,1,D] and final state.  skip: that chunk's sum is lost;
    stale: that chunk reads the state of the one before; diagonal: only the
    diagonal of that chunk's scores is kept."""
    q, k, v = q[:, 0], k[:, 0], v[:, 0]
    scale, lam = D ** -0.5, np.exp(g)
    S, before, outs = np.zeros((D, D)), np.zeros((D, D)), []
    for c, t0 in enumerate(range(0, len(q), CHUNK)):
        qc, kc, vc = (x[t0:t0 + CHUNK] for x in (q, k, v))
        i = np.arange(len(qc))
        P = np.where(i[:, None] >= i, scale * lam ** np.maximum(i[:, None] - i, 0.0) * (qc @ kc.T), 0.0)
        if c == diagonal:
            P = np.diag(np.diag(P))
        image = bf16(before if c == stale else S)
        outs.append(bf16(bf16(P) @ vc + scale * lam ** (i[:, None] + 1.0) * (qc @ image.T)))
        before = S
        own = 0.0 if c == skip else parts(vc * lam ** (len(qc) - 1.0 - i)[:, None], value_parts).T @ kc
        S = np.float32(lam ** len(qc) * S + own).astype(np.float64)
    return np.concatenate(outs)[:, None], S[None, None]


T, G = 3000, -1e-4


@pytest.fixture(scope="module")
def case():
    q, k, v = make(T)
    return (q, k, v), oracle.linear_recurrent(q, k, v, np.array([G]), scale=D ** -0.5)


def test_the_documented_roundings_pass(case):
    x, (o_ref, s_ref) = case
    o, s = chunked(*x, G)
    assert worst_chunk(o, o_ref, [T]) <= OUT_BOUND
    assert worst_state(s, s_ref) <= state_bound(-(-T // CHUNK))


@pytest.mark.parametrize("mistake", [dict(skip=20), dict(skip=0), dict(stale=16), dict(stale=22), dict(stale=1),
                                     dict(diagonal=16), dict(diagonal=22)], ids=str)
def test_a_lost_or_stale_chunk_is_seen(case, mistake):
    x, (o_ref, _) = case
    o, _ = chunked(*x, G, **mistake)
    assert worst_chunk(o, o_ref, [T]) > 3 * OUT_BOUND


@pytest.mark.parametrize("n", [100, 300, 1500])
@pytest.mark.parametrize("g", [0.0, -0.01, -0.5])
def test_a_lost_third_part_of_the_values_is_seen(n, g):
    q, k, v = make(n, seed=n)
    _, s_ref = oracle.linear_recurrent(q, k, v, np.array([g]))
    chunks = -(-n // CHUNK)
    assert worst_state(chunked(q, k, v, g)[1], s_ref) <= state_bound(chunks)
    # Two parts leave each weighted value off by 40 u on average, but the newest token's, whose
    # weight is 1, by nothing: at exp(-0.5) a token that share is 1 - exp(-1) of the squares, and
    # sqrt(exp(-1)) 40 u = 24 u is within the bound.  Undecayed, a bf16 value is one part.
    if -0.2 < g < 0:
        assert worst_state(chunked(q, k, v, g, value_parts=2)[1], s_ref) > state_bound(chunks)


def test_a_lost_row_of_a_weight_gradient_is_seen():
    """Of 72,000 rows: one missing row is past the bound in most columns, 128 in nearly all."""
    rng = np.random.default_rng(8)
    dy, n = rng.standard_normal((2, 3000, 24, 64))
    bound = dw_bound(dy, n)
    one, block = dy[77, 5] * n[77, 5], (dy[40:, 3] * n[40:, 3])[:128].sum(0)
    assert (np.abs(one) > bound).mean() > 0.7 and (np.abs(block) > bound).mean() > 0.95
