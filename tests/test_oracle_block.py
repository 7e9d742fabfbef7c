"""Pins of the fp64 oracles of the transformer block's operators (CPU)."""
import math

import numpy as np
import pytest

from oracle import unet_ops

torch = pytest.importorskip("torch")


@pytest.fixture
def ln_case():
    rng = np.random.default_rng(7)
    return (rng.normal(0.3, 2.0, (5, 12)), rng.normal(size=(5, 12)), 1 + 0.3 * rng.normal(size=12), rng.normal(size=12))


def test_layer_norm_brute_force(ln_case):
    x, _, gamma, beta = ln_case
    y, stats = unet_ops.layer_norm(x, gamma, beta, 1e-5)
    for t in range(5):
        m = math.fsum(x[t]) / 12
        v = math.fsum((a - m) ** 2 for a in x[t]) / 12
        assert stats[t, 0] == pytest.approx(m, rel=1e-13) and stats[t, 1] == pytest.approx(1 / math.sqrt(v + 1e-5), rel=1e-13)
        for c in range(12):
            assert y[t, c] == pytest.approx((x[t, c] - m) / math.sqrt(v + 1e-5) * gamma[c] + beta[c], rel=1e-11, abs=1e-12)


def test_layer_norm_gradients_are_torchs(ln_case):
    x, dy, gamma, beta = ln_case
    tx, tg, tb = (torch.tensor(a, dtype=torch.float64, requires_grad=True) for a in (x, gamma, beta))
    y = torch.nn.functional.layer_norm(tx, (12,), tg, tb, 1e-5)
    y.backward(torch.tensor(dy))
    ref, stats = unet_ops.layer_norm(x, gamma, beta, 1e-5)
    np.testing.assert_allclose(ref, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for got, want in zip(unet_ops.layer_norm_backward(dy, x, stats, gamma), (tx.grad, tg.grad, tb.grad)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-11, atol=1e-12)


def test_geglu_backward_against_differences():
    rng = np.random.default_rng(11)
    x, w, b, dy = rng.normal(size=(5, 6)), rng.normal(size=(8, 6)), rng.normal(size=8), rng.normal(size=(5, 4))
    got = unet_ops.geglu_backward(dy, x, w, b)
    f = lambda v: (unet_ops.geglu(v[0] @ v[1].T + v[2]) * dy).sum()   # noqa: E731
    at, step = [x, w, b], 1e-6
    for k, grad in enumerate(got):
        for i in np.ndindex(at[k].shape):
            d = np.zeros(at[k].shape)
            d[i] = step
            num = (f([a + d if j == k else a for j, a in enumerate(at)])
                   - f([a - d if j == k else a for j, a in enumerate(at)])) / (2 * step)
            # the differences' own error: step^2 of third derivatives and 2^-52 |f| / step, both below 1e-7 here
            assert abs(num - grad[i]) <= 1e-6 * max(1.0, abs(grad[i]))
    assert np.array_equal(unet_ops.geglu_backward(dy, x, w)[0], unet_ops.geglu_backward(dy, x, w, np.zeros(8))[0])
