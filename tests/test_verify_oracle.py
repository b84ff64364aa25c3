"""The oracle of draft verification (CPU): what it draws is distributed as the
target, and it refuses and falls back where the rule says so."""
import numpy as np
import pytest

from oracle.speculation import dequantise, quantise, verify_drafts


def rows(rng, *shape):
    x = np.exp(1.5 * rng.standard_normal(shape))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def drawn_from(rng, row, n):
    return np.minimum(np.searchsorted(np.cumsum(row), rng.random(n) * row.sum()), len(row) - 1)


@pytest.mark.parametrize("real", [np.float32, np.float64])
@pytest.mark.parametrize("with_q", [True, False])
def test_first_token_follows_the_target(with_q, real):
    """Two siblings drawn from q (or two fixed proposals): the token after the root -- the
    accepted child's, or the next token -- has the frequencies of p.  A frequency of N draws
    is off by at most 5 sqrt(p (1 - p) / N) (5 sigma)."""
    rng = np.random.default_rng(1)
    N, V = 20000, 6
    P, Q = rows(rng, V), rows(rng, V)
    p = np.broadcast_to(P, (N, 3, V)).copy()
    q = np.broadcast_to(Q, (N, 3, V)).copy() if with_q else None
    tok = np.zeros((N, 3), np.int32)
    tok[:, 1:] = drawn_from(rng, Q, 2 * N).reshape(N, 2) if with_q else [2, 4]
    parent = np.broadcast_to(np.array([-1, 0, 0], np.int32), (N, 3))
    coins, u = rng.random((N, 3), np.float32), rng.random(N, np.float32)
    path, n, nxt, _ = verify_drafts(p, q, tok, parent, coins, u, 2, real)
    first = np.where(n > 1, tok[np.arange(N), np.maximum(path[:, 1], 0)], nxt)
    got = np.bincount(first, minlength=V) / N
    assert (np.abs(got - P) <= 5 * np.sqrt(P * (1 - P) / N)).all(), (got, P)


def test_rounded_and_real_rules_agree():
    """The float32 rule decides as the mathematics does wherever no decision is within 1e-5 of
    going the other way (a float32 mass of a row is off by a few 2^-24)."""
    rng = np.random.default_rng(2)
    B, T, V = 200, 12, 300
    p = rows(rng, B, T, V)
    q = rows(rng, B, T, V)
    q = (0.7 * p + 0.3 * q).astype(np.float32)
    parent = np.stack([np.r_[-1, [rng.integers(0, t) for t in range(1, T)]] for _ in range(B)])
    tok = np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(1, T):
            tok[b, t] = drawn_from(rng, q[b, parent[b, t]], 1)[0]
    coins, u = rng.random((B, T), np.float32), rng.random(B, np.float32)
    for qq in (q, None):
        a = verify_drafts(p, qq, tok, parent, coins, u, T, np.float32)
        c = verify_drafts(p, qq, tok, parent, coins, u, T, np.float64)
        sure = c[3] > 1e-5
        assert sure.mean() > 0.8
        for x, y in zip(a[:3], c[:3]):
            assert (x[sure] == y[sure]).all()


def test_rows_without_mass():
    V = 5
    p = np.zeros((1, 2, V), np.float32)
    par, tok = np.array([[-1, 0]]), np.array([[0, 3]], np.int32)
    coins, u = np.zeros((1, 2), np.float32), np.zeros(1, np.float32)
    path, n, nxt, _ = verify_drafts(p, None, tok, par, coins, u, 2)
    assert n[0] == 1 and nxt[0] == -1 and (path == [[0, -1]]).all()
    p[0, 0, 3] = 1.0   # all mass on the child, whose coin refuses it: the row as it was
    path, n, nxt, _ = verify_drafts(p, None, tok, par, np.ones((1, 2), np.float32), u, 2)
    assert n[0] == 1 and nxt[0] == 3


def test_quantise_is_within_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((2, 3, 32, 64)) * np.exp(3 * rng.standard_normal((2, 3, 32, 1))))
    x = x.astype(np.float32)
    codes, scale = quantise(x)
    assert np.abs(codes).max() == 127
    # half a step, and the rounding of the product and of the scale (127 * 3 * 2^-24 steps)
    err = np.abs(dequantise(codes, scale).astype(np.float64) - x)
    assert (err <= scale[..., None].astype(np.float64) * (0.5 + 127 * 3 * 2.0 ** -24)).all()
