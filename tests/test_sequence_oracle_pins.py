"""Pins of the sequence oracle: its recurrence against the written-out sums, its gradients against
differences, its rotation against complex multiplication."""
import math

import numpy as np

from oracle import sequence_oracle as SO


def problem(n=7, D=4, seed=0):
    r = np.random.default_rng(seed)
    return [r.standard_normal((n, D)) for _ in range(4)] + [r.standard_normal((D, D)) for _ in range(2)]


def test_recurrence_is_the_written_out_sum():
    q, k, v, _, S0, _ = problem()
    g, scale = math.log(0.8), 0.5
    out, S = SO.decay_forward(q, k, v, g, S0, scale)
    n = len(q)
    for i in range(n):
        want = sum(0.8 ** (i - j) * (q[i] @ k[j]) * v[j] for j in range(i + 1))
        want = scale * (want + 0.8 ** (i + 1) * (q[i] @ S0))
        assert np.allclose(out[i], want, rtol=0, atol=1e-13)
    want = 0.8 ** n * S0 + sum(0.8 ** (n - 1 - j) * np.outer(k[j], v[j]) for j in range(n))
    assert np.allclose(S, want, rtol=0, atol=1e-13)


def test_gradients_are_the_differences():
    q, k, v, do, S0, dS = problem(seed=1)
    g, scale = math.log(0.7), 0.5

    def loss(q, k, v, S0):
        out, S = SO.decay_forward(q, k, v, g, S0, scale)
        return (out * do).sum() + (S * dS).sum()

    got = SO.decay_backward(q, k, v, g, do, S0, dS, scale)
    args = [q, k, v, S0]
    for n, grad in enumerate(got):
        for idx in [(0, 0), (2, 3), (grad.shape[0] - 1, 1)]:
            e = 1e-5
            up, dn = [x.copy() for x in args], [x.copy() for x in args]
            up[n][idx] += e
            dn[n][idx] -= e
            # the loss is linear in each argument: the difference has no truncation error
            assert abs((loss(*up) - loss(*dn)) / (2 * e) - grad[idx]) < 1e-7


def test_rotation_is_complex_multiplication():
    r = np.random.default_rng(2)
    x, freq, pos = r.standard_normal((3, 5, 10)), np.array([1.0, 0.1, 0.01]), np.arange(5) * 7
    z = np.exp(1j * pos[:, None] * freq) * 1.5
    half = SO.rotary(x, pos, freq, 1.5)
    w = (x[..., 0:3] + 1j * x[..., 3:6]) * z
    assert np.allclose(half[..., 0:3], w.real) and np.allclose(half[..., 3:6], w.imag)
    inter = SO.rotary(x, pos, freq, 1.5, interleaved=True)
    w = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) * z
    assert np.allclose(inter[..., 0:6:2], w.real) and np.allclose(inter[..., 1:6:2], w.imag)
    for y in (half, inter):
        assert (y[..., 6:] == x[..., 6:]).all()
    back = SO.rotary(SO.rotary(x, pos, freq, interleaved=True), pos, freq, interleaved=True,
                     inverse=True)
    assert np.allclose(back, x)
