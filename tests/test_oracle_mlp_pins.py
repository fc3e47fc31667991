"""Pins of the MLP-branch oracle: its gradients against central differences of its
own forward, its forward against torch in fp64, and the 8-bit format's stated
properties. CPU only."""

import numpy as np
import pytest
import torch

import oracle

MOD = np.array([0, 0, 1, 0, 1, 1, 0])


def _loss_grad(f, a, g, h=1e-6):
    """Central differences of sum(f(a) * g) with respect to a."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        p, m = a.copy(), a.copy()
        p[i] += h
        m[i] -= h
        out[i] = ((f(p) - f(m)) * g).sum() / (2 * h)
    return out


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_gradients_against_differences(act):
    rng = np.random.default_rng(11)
    T, K, N = len(MOD), 5, 4
    x, W, b = rng.standard_normal((T, K)), rng.standard_normal((2, N, K)), rng.standard_normal((2, N))
    r, g = rng.standard_normal((T, N)), rng.standard_normal((T, N))
    _, z = oracle.linear_fused(x, W, b, r, MOD, act)
    dx, dW, db, _ = oracle.linear_fused_bwd(g, x, W, z, MOD, act)
    # central differences at h = 1e-6: truncation h^2 f'''/6 and rounding eps/h, both ~1e-9
    for got, at, f in ((dx, x, lambda a: oracle.linear_fused(a, W, b, r, MOD, act)[0]),
                       (dW, W, lambda a: oracle.linear_fused(x, a, b, r, MOD, act)[0]),
                       (db, b, lambda a: oracle.linear_fused(x, W, a, r, MOD, act)[0])):
        np.testing.assert_allclose(got, _loss_grad(f, at, g), atol=2e-8)


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(12)
    T, n, eps = len(MOD), 6, 1e-6
    x, g = rng.standard_normal((T, n)), rng.standard_normal((T, n))
    gamma, beta = rng.standard_normal((2, n)), rng.standard_normal((2, n))
    resid = rng.standard_normal((T, n))
    _, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, MOD, eps)
    dx, dgamma, dbeta = oracle.layer_norm_affine_bwd(g, x, gamma, np.stack([mean, rstd], 1), MOD)
    for got, at, f in ((dx, x, lambda a: oracle.layer_norm_affine(a, gamma, beta, MOD, eps)[0]),
                       (dgamma, gamma, lambda a: oracle.layer_norm_affine(x, a, beta, MOD, eps)[0]),
                       (dbeta, beta, lambda a: oracle.layer_norm_affine(x, gamma, a, MOD, eps)[0])):
        np.testing.assert_allclose(got, _loss_grad(f, at, g), atol=5e-8)
    with_resid = oracle.layer_norm_affine_bwd(g, x, gamma, np.stack([mean, rstd], 1), MOD, resid)[0]
    np.testing.assert_allclose(with_resid, dx + resid, rtol=1e-14)


def test_layer_norm_against_torch():
    rng = np.random.default_rng(13)
    x, gamma, beta = rng.standard_normal((7, 24)), rng.standard_normal((2, 24)), rng.standard_normal((2, 24))
    y, _, _ = oracle.layer_norm_affine(x, gamma, beta, MOD, 1e-6)
    for t in range(7):
        ref = torch.nn.functional.layer_norm(torch.tensor(x[t]), (24,), torch.tensor(gamma[MOD[t]]),
                                             torch.tensor(beta[MOD[t]]), 1e-6)
        np.testing.assert_allclose(y[t], ref.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("act,fn", [("gelu", lambda z: torch.nn.functional.gelu(z, approximate="tanh")),
                                    ("silu", torch.nn.functional.silu)])
def test_activations_against_torch(act, fn):
    z = torch.linspace(-9, 9, 401, dtype=torch.float64, requires_grad=True)
    out = fn(z)
    out.sum().backward()
    np.testing.assert_allclose(oracle.mlp_act(z.detach().numpy(), act), out.detach().numpy(), atol=1e-14)
    np.testing.assert_allclose(oracle.mlp_act_grad(z.detach().numpy(), act), z.grad.numpy(), atol=1e-14)


def test_act8_format():
    rng = np.random.default_rng(14)
    x = (rng.standard_normal((5, 300)) * 10.0 ** rng.integers(-8, 8, (5, 1))).astype(np.float32)
    x[1, 128:256] = 0
    x[2, 256:] = 1e-35          # below 2^-100
    x[3, 7], x[4, 299] = np.inf, np.nan
    q, s = oracle.act8_quantize(x)
    v = oracle.act8_values(q, s)
    assert q.shape == (5, 300) and s.shape == (5, 3)
    assert np.isnan(v[3, :128]).all() and np.isfinite(v[3, 128:]).all()
    assert np.isnan(v[4, 256:]).all() and np.isfinite(v[4, :256]).all()
    assert (v[1, 128:256] == 0).all() and (v[2, 256:] == 0).all()
    ok = np.isfinite(v)
    ok[2, 256:] = False
    half = np.asarray(s, np.float64)[:, np.arange(300) // 128] / 2
    assert (np.abs(v - np.asarray(x, np.float64))[ok] <= half[ok] * (1 + 2.0 ** -15)).all()
    assert np.abs(q[0]).max() == 127
