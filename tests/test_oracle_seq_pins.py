"""Pins of the fp64 oracles of the language-model operators: closed forms, and gradients against
central differences (float64, step 1e-6: truncation and rounding leave about 1e-8)."""
import numpy as np
import pytest

from oracle.seq_oracle import gated_delta, qk_norm_rope


def test_norm_has_unit_mean_square_and_rotation_keeps_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 4, 32))
    pos = rng.integers(0, 7, (2, 3))
    ang = rng.standard_normal((7, 16))
    for il in (False, True):
        y = qk_norm_rope(x, 2, 1, None, None, np.cos(ang), np.sin(ang), pos, 0.0, il)
        assert np.allclose((y[:, :, :3] ** 2).mean(-1), 1.0)
        assert np.array_equal(y[:, :, 3], x[:, :, 3])
    # by position 0 with angle 0 nothing turns
    y = qk_norm_rope(x, 2, 1, None, None, np.ones((1, 16)), np.zeros((1, 16)), np.zeros((2, 3), int), 0.0, False)
    assert np.allclose(y[:, :, :3], x[:, :, :3] / np.sqrt((x[:, :, :3] ** 2).mean(-1, keepdims=True)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradient_against_differences(interleaved):
    rng = np.random.default_rng(1)
    x, wq, wk = rng.standard_normal((1, 3, 3, 32)), rng.standard_normal(32), rng.standard_normal(32)
    ang, pos = rng.standard_normal((5, 8)), np.array([[4, -1, 2]])
    dout = rng.standard_normal(x.shape)
    args = (np.cos(ang), np.sin(ang), pos, 1e-3, interleaved)
    f = lambda x, wq, wk: (qk_norm_rope(x, 1, 1, wq, wk, *args) * dout).sum()  # noqa: E731
    got = qk_norm_rope(x, 1, 1, wq, wk, *args, dout=dout)
    for i, t in enumerate((x, wq, wk)):
        flat = t.reshape(-1)
        for j in rng.integers(0, flat.size, 25):
            old, e = flat[j], 1e-6
            flat[j] = old + e
            up = f(x, wq, wk)
            flat[j] = old - e
            down = f(x, wq, wk)
            flat[j] = old
            assert abs((up - down) / (2 * e) - got[i].reshape(-1)[j]) < 1e-7


def _delta_inputs(rng, N, Hk, Hv, d):
    q, k = rng.standard_normal((2, N, Hk, d))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return q, k, rng.standard_normal((N, Hv, d)), -rng.random((N, Hv)), rng.random((N, Hv))


def test_delta_closed_forms():
    rng = np.random.default_rng(2)
    q, k, v, g, beta = _delta_inputs(rng, 6, 1, 2, 4)
    # full write strength and unit keys: reading the last key back gives its value
    out, S = gated_delta(k, k, v, g, np.ones_like(beta), 1.0)
    assert np.allclose(out, v)
    # an emptied state: the tokens before the reset do not matter
    g2 = g.copy()
    g2[3] = -np.inf
    a, Sa = gated_delta(q, k, v, g2, beta, 0.5)
    b, Sb = gated_delta(q[3:], k[3:], v[3:], g[3:], beta[3:], 0.5)
    assert np.allclose(a[3:], b) and np.allclose(Sa, Sb)
    # no write: the state only decays
    S0 = rng.standard_normal((2, 4, 4))
    _, S = gated_delta(q, k, v, g, 0 * beta, 1.0, S0)
    assert np.allclose(S, np.exp(g.sum(0))[:, None, None] * S0)
    # orthogonal keys, no decay: linear attention
    eye = np.broadcast_to(np.eye(4)[:, None], (4, 1, 4))
    out, _ = gated_delta(q[:4], eye, v[:4], 0 * g[:4], np.ones((4, 2)), 1.0)
    w = np.tril(q[:4, 0] @ eye[:, 0].T)
    assert np.allclose(out, np.einsum("ij,jhd->ihd", w, v[:4]))


def test_delta_gradient_against_differences():
    rng = np.random.default_rng(3)
    N, Hk, Hv, d = 5, 1, 2, 3
    q, k, v, g, beta = _delta_inputs(rng, N, Hk, Hv, d)
    S0 = rng.standard_normal((Hv, d, d))
    do, dS = rng.standard_normal((N, Hv, d)), rng.standard_normal((Hv, d, d))

    def f(*t):
        out, S = gated_delta(*t[:5], 0.7, t[5])
        return (out * do).sum() + (S * dS).sum()

    ins = [q.copy(), k.copy(), v, g, beta, S0]
    got = gated_delta(*ins[:5], 0.7, S0, grads=(do, dS))[2]
    for i, t in enumerate(ins):
        flat = t.reshape(-1)
        for j in range(flat.size):
            old, e = flat[j], 1e-6
            flat[j] = old + e
            up = f(*ins)
            flat[j] = old - e
            down = f(*ins)
            flat[j] = old
            assert abs((up - down) / (2 * e) - got[i].reshape(-1)[j]) < 1e-7, (i, j)
