"""Pins of the fp64 definitions of the distillation operators: gradients
against central differences, closed forms, and torch's own operators."""
import numpy as np
import pytest
import torch

from oracle import distill_oracle as D


def _gen(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_rmsnorm_closed_form():
    # a row of equal values v has rms |v|: y = sign(v)·γ for eps = 0
    _, rstd, y = D.rmsnorm(np.array([[2.0, 2.0], [-3.0, -3.0]]), None, np.array([1.0, 5.0]), 0.0)
    assert np.allclose(rstd, [0.5, 1 / 3]) and np.allclose(y, [[1, 5], [-1, -5]])
    h, _, _ = D.rmsnorm(np.array([[1.0, 2.0]]), np.array([[3.0, -1.0]]), None, 1e-6)
    assert np.array_equal(h, [[4.0, 1.0]])
    assert D.rmsnorm_q8_scale(np.array([[1.0, -254.0], [0.0, 0.0]])).tolist() == [2.0, 0.0]


def test_rmsnorm_grad_against_differences():
    gen = _gen(1)
    x, g, w = gen.standard_normal((3, 7)), gen.standard_normal(7), gen.standard_normal((3, 7))
    v = gen.standard_normal((3, 7))      # gradient that reaches h by another way: f adds Σ v·h

    def f(x, g):
        h, _, y = D.rmsnorm(x, None, g, 1e-3)
        return np.sum(w * y) + np.sum(v * h)

    _, rstd, _ = D.rmsnorm(x, None, g, 1e-3)
    dx, dg = D.rmsnorm_grad(w, x, rstd, g, v)
    e = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((f(x + d, g) - f(x - d, g)) / (2 * e) - dx[i]) < 1e-8
    for j in range(7):
        d = np.zeros(7)
        d[j] = e
        assert abs((f(x, g + d) - f(x, g - d)) / (2 * e) - dg[j]) < 1e-8


def test_q8_matmul_is_the_integer_product():
    gen = _gen(2)
    a, w = gen.integers(-128, 128, (5, 33)).astype(np.int8), gen.integers(-128, 128, (4, 33)).astype(np.int8)
    want = a.astype(object) @ w.astype(object).T
    got = D.q8_matmul(a, np.full(5, 0.5), w, np.full(4, 2.0))
    assert np.array_equal(got, want.astype(np.float64))


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_against_torch_and_differences(tau):
    gen = _gen(3)
    T, V, k = 4, 11, 5
    z, t = gen.standard_normal((T, V)) * 2, gen.standard_normal((T, k)) * 2
    index = np.stack([gen.permutation(V)[:k] for _ in range(T)])
    index[1, 3] = -1                      # absent
    index[2, 4] = index[2, 0]             # twice
    index[3, :] = -1                      # no entries
    up = gen.standard_normal(T)
    loss, lse, dz = D.distill_topk(z, index, t, tau, up)
    assert loss[3] == 0 and not dz[3].any()
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(z) / tau, 1).numpy(), rtol=1e-13)
    # row 0 is an ordinary KL divergence of dense distributions
    dense = torch.full((V,), -np.inf, dtype=torch.float64)
    dense[torch.from_numpy(index[0])] = torch.from_numpy(t[0])
    kl = torch.nn.functional.kl_div(torch.log_softmax(torch.from_numpy(z[0]) / tau, 0),
                                    torch.softmax(dense / tau, 0), reduction="sum")
    assert abs(loss[0] - tau ** 2 * float(kl)) < 1e-12
    e = 1e-6
    for i in np.ndindex(T, V):
        d = np.zeros((T, V))
        d[i] = e
        diff = (D.distill_topk(z + d, index, t, tau)[0] - D.distill_topk(z - d, index, t, tau)[0]) / (2 * e)
        assert abs(up[i[0]] * diff[i[0]] - dz[i]) < 1e-7


def test_distill_minus_infinity():
    z = np.array([[0.0, -np.inf, 1.0]])
    loss, _, dz = D.distill_topk(z, np.array([[0, 2]]), np.array([[0.0, -np.inf]]), 1.0)
    assert np.isclose(loss[0], np.log(1 + np.e)) and dz[0, 1] == 0
    loss, _, dz = D.distill_topk(z, np.array([[0, 2]]), np.array([[-np.inf, -np.inf]]), 1.0)
    assert loss[0] == 0 and not dz.any()
