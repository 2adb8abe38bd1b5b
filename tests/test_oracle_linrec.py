"""Pins of the fp64 elementwise recurrence: closed forms, and the gradients against differences."""
import numpy as np

from oracle import linrec as O


def test_constant_gate_is_a_geometric_sum():
    T, a = 12, 0.75
    y, s = O.replay(np.ones((T, 2)), np.full((T, 2), np.log(a)), [0, T])
    want = (1 - a ** np.arange(1, T + 1)) / (1 - a)
    assert np.allclose(y, want[:, None], rtol=1e-13, atol=0)
    assert np.allclose(s, want[-1], rtol=1e-13, atol=0)


def test_a_closed_gate_forgets_and_empty_sequences_keep_h0():
    x = np.arange(10.0).reshape(5, 2)
    g = np.zeros((5, 2))
    g[3] = -np.inf
    h0 = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    y, s = O.replay(x, g, [0, 2, 2, 5], h0)
    assert np.array_equal(s[1], h0[1])
    assert np.array_equal(y[3], x[3]) and np.array_equal(s[2], x[3] + x[4])
    assert np.array_equal(s[0], h0[0] + x[0] + x[1])


def test_gradients_are_the_differences():
    rng = np.random.default_rng(5)
    cu = [0, 3, 3, 4, 11]
    x, dy = rng.normal(size=(11, 3)), rng.normal(size=(11, 3))
    g = -rng.uniform(0.01, 2, size=(11, 3))
    h0, ds = rng.normal(size=(4, 3)), rng.normal(size=(4, 3))

    def loss(x, g, h0):
        y, s = O.replay(x, g, cu, h0)
        return (y * dy).sum() + (s * ds).sum()

    y, _ = O.replay(x, g, cu, h0)
    grads = O.backward(g, y, dy, cu, h0, ds)
    eps = 1e-5
    for k, grad in enumerate(grads):
        for _ in range(6):
            u = [np.zeros_like(x), np.zeros_like(g), np.zeros_like(h0)]
            u[k] = rng.normal(size=u[k].shape)
            up = loss(x + eps * u[0], g + eps * u[1], h0 + eps * u[2])
            down = loss(x - eps * u[0], g - eps * u[1], h0 - eps * u[2])
            # central differences: eps^2 of the third derivative, and 2^-52 of the loss over eps
            assert abs((up - down) / (2 * eps) - (grad * u[k]).sum()) < 1e-7
