"""Pins of the fp64 oracle of linear attention with a decay per head and of the
query/key norm with rotation: closed forms, invariances and central differences,
none of which types its formulas again."""
import numpy as np
import pytest

import oracle


def rnd(seed):
    return np.random.default_rng(seed)


def make(seed, lens, Hqk=2, Hv=6, Dk=5, Dv=4):
    r, T, N = rnd(seed), sum(lens), len(lens)
    x = dict(q=r.standard_normal((T, Hqk, Dk)), k=r.standard_normal((T, Hqk, Dk)), v=r.standard_normal((T, Hv, Dv)),
             s0=r.standard_normal((N, Hv, Dv, Dk)))
    return x, -np.linspace(0.0, 2.0, Hv), np.concatenate([[0], np.cumsum(lens)])


def test_a_single_token_and_its_orientation():
    """One token into a zero state: S = v k^T, read by q as scale (k . q) v."""
    x, g, _ = make(1, [1])
    o, S = oracle.linear_recurrent(x["q"], x["k"], x["v"], g, scale=0.5)
    for h in range(6):  # heads 0..2 share q/k head 0
        k, q, v = x["k"][0, h // 3], x["q"][0, h // 3], x["v"][0, h]
        np.testing.assert_allclose(S[0, h], np.outer(v, k), atol=1e-15)
        np.testing.assert_allclose(o[0, h], 0.5 * (k @ q) * v, atol=1e-14)


def test_closed_form_of_the_decayed_sum():
    """o_t = scale (lam^(t+1) S0 + sum_j lam^(t-j) v_j k_j^T) q_t, per sequence."""
    lens = [7, 0, 1, 12]
    x, g, cu = make(2, lens)
    o, S = oracle.linear_recurrent(x["q"], x["k"], x["v"], g, x["s0"], cu, scale=0.3)
    for n, L in enumerate(lens):
        for h in range(6):
            t = np.arange(L)
            kn, qn, vn = (x["k"][cu[n]:cu[n + 1], h // 3], x["q"][cu[n]:cu[n + 1], h // 3], x["v"][cu[n]:cu[n + 1], h])
            w = np.tril(np.exp(g[h] * np.tril(t[:, None] - t)))
            want = (w * (qn @ kn.T)) @ vn + np.exp(g[h] * (t + 1))[:, None] * (qn @ x["s0"][n, h].T)
            np.testing.assert_allclose(o[cu[n]:cu[n + 1], h], 0.3 * want, atol=1e-12)
            last = np.exp(g[h] * L) * x["s0"][n, h] + (np.exp(g[h] * (L - 1 - t))[:, None] * vn).T @ kn
            np.testing.assert_allclose(S[n, h], last, atol=1e-12)


def test_without_decay_order_does_not_matter_to_the_state():
    x, _, _ = make(3, [9])
    p = rnd(4).permutation(9)
    a = oracle.linear_recurrent(x["q"], x["k"], x["v"], np.zeros(6), x["s0"])[1]
    b = oracle.linear_recurrent(x["q"][p], x["k"][p], x["v"][p], np.zeros(6), x["s0"])[1]
    np.testing.assert_allclose(a, b, atol=1e-13)


def test_linear_gradients_by_central_differences():
    """The loss is linear in each input alone, so a central difference in one is exact
    but for rounding."""
    lens = [5, 0, 3]
    x, g, cu = make(5, lens)
    r = rnd(6)
    do, dsT = r.standard_normal(x["v"].shape), r.standard_normal(x["s0"].shape)

    def loss(y):
        o, S = oracle.linear_recurrent(y["q"], y["k"], y["v"], g, y["s0"], cu, scale=0.7)
        return (o * do).sum() + (S * dsT).sum()

    got = dict(zip(("q", "k", "v", "s0"), oracle.linear_backward(do, x["q"], x["k"], x["v"], g, x["s0"], cu, dsT=dsT,
                                                                scale=0.7)))
    for name, grad in got.items():
        assert grad.shape == x[name].shape
        for at in np.ndindex(*grad.shape):
            y = dict(x)
            y[name] = x[name].copy()
            y[name][at] += 0.5
            up = loss(y)
            y[name][at] -= 1.0
            assert abs(up - loss(y) - grad[at]) < 1e-10 * (1 + abs(grad[at])), (name, at)


ROPE = [dict(), dict(interleaved=True), dict(sections=[1, 3, 2]), dict(sections=[0, 6, 0], interleaved=True)]


def rope_case(seed, opts, T=6, H=3, D=16, R=12):
    r = rnd(seed)
    axes = len(opts.get("sections", [0]))
    pos = r.integers(-50, 1000, (axes, T))
    return r.standard_normal((T, H, D)), 1 + 0.3 * r.standard_normal(D), pos, 100.0 ** (-np.arange(R // 2) / 6.0)


@pytest.mark.parametrize("opts", ROPE, ids=str)
def test_rotation_keeps_lengths_and_turns_back(opts):
    x, w, pos, f = rope_case(11, opts)
    y = oracle.qk_norm_rope(x, w, 1e-6, None, None)
    z = oracle.qk_norm_rope(x, w, 1e-6, pos, f, **opts)
    np.testing.assert_allclose(np.linalg.norm(z, axis=-1), np.linalg.norm(y, axis=-1), rtol=1e-13)
    np.testing.assert_array_equal(z[..., 12:], y[..., 12:])  # what is not rotated
    back = oracle.qk_norm_rope(z, None, 1e-6, pos, f, inverse=True, norm=False, **opts)
    np.testing.assert_allclose(back, y, atol=1e-13)
    assert np.abs(z - y).max() > 0.1
    # unit weights: rows of root mean square 1, whatever their scale
    n = oracle.qk_norm_rope(1e3 * x, None, 1e-30, None, None)
    np.testing.assert_allclose((n * n).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("opts", ROPE[:2], ids=str)
def test_products_depend_on_relative_positions_only(opts):
    x, w, _, f = rope_case(12, opts, T=1)
    turn = lambda p: oracle.qk_norm_rope(x, w, 1e-6, np.array([p]), f, **opts)
    for far in (0, 5, 100000):
        np.testing.assert_allclose((turn(far + 9) * turn(far)).sum(), (turn(9) * turn(0)).sum(), rtol=1e-9)


def test_quarter_turns():
    """A frequency of pi / 2: at position 1 the pair (a, b) becomes (-b, a); every pair's
    place, in halves and interleaved, and each axis's frequencies."""
    x = rnd(13).standard_normal((2, 1, 16))
    for inter, pairs in ((False, [(i, i + 4) for i in range(4)]), (True, [(2 * i, 2 * i + 1) for i in range(4)])):
        for axis, mine in ((0, pairs[:1]), (1, pairs[1:])):
            pos = np.zeros((2, 2))
            pos[axis, 1] = 1
            z = oracle.qk_norm_rope(x, None, 1e-6, pos, np.full(4, np.pi / 2), sections=[1, 3], interleaved=inter,
                                    norm=False)
            want = x.copy()
            for a, b in mine:
                want[1, 0, a], want[1, 0, b] = -x[1, 0, b], x[1, 0, a]
            np.testing.assert_allclose(z, want, atol=1e-14)


@pytest.mark.parametrize("opts", ROPE, ids=str)
def test_rope_gradients_by_central_differences(opts):
    """Fourth-order differences: error of h^4 and of 1e-16 / h, both below 1e-10."""
    x, w, pos, f = rope_case(14, opts, T=3, H=2)
    dz = rnd(15).standard_normal(x.shape)
    loss = lambda y, u: (oracle.qk_norm_rope(y, u, 1e-3, pos, f, **opts) * dz).sum()
    dx, dw = oracle.qk_norm_rope_backward(dz, x, w, 1e-3, pos, f, **opts)

    def difference(of, at):
        def shifted(s):
            y, u = x.copy(), w.copy()
            (y if of == "x" else u)[at] += s
            return loss(y, u)
        h = 1e-3
        return (8 * (shifted(h) - shifted(-h)) - (shifted(2 * h) - shifted(-2 * h))) / (12 * h)

    for of, grad in (("x", dx), ("w", dw)):
        for at in np.ndindex(*grad.shape):
            assert abs(difference(of, at) - grad[at]) < 1e-8, (of, at)
