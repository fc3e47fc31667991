"""Plain fp64 NumPy definitions of the MLP-branch operators: the modality-specific
layer norm with weights, the linear layer with bias, activation and residual, their
gradients, and activation checkpoints in 8 bits.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): slow, obviously correct.

Sources (page title, then section): [norm], [fuse], [train] of
``oracle/__init__.py``. The pages name modality-specific weights and fused chains,
not these forms; the forms are the usual ones, written out below. ``mod[t]`` is the
token's modality (0 image, 1 text). Inputs arrive as float32 arrays holding exact
bf16 or fp32 values; every computation is float64 except where a definition is in
fp32 (the checkpoint's scale and code).
"""

from __future__ import annotations

import numpy as np

ACT8_BLOCK = 128


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def mlp_act(z, act: str) -> np.ndarray:
    """none; gelu: 0.5 z (1 + tanh(sqrt(2/pi)(z + 0.044715 z^3))); silu: z sigma(z)."""
    z = np.asarray(z, dtype=np.float64)
    if act == "none":
        return z
    if act == "gelu":
        return 0.5 * z * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    raise ValueError(act)


def mlp_act_grad(z, act: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if act == "none":
        return np.ones_like(z)
    if act == "gelu":
        c = np.sqrt(2.0 / np.pi)
        th = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    raise ValueError(act)


def layer_norm_affine(x, gamma, beta, mod, eps: float):
    """(y, mean, rstd): each row normalised with the population variance."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    return xhat * _f64(gamma)[mod] + _f64(beta)[mod], mean, rstd


def layer_norm_affine_bwd(dy, x, gamma, stats, mod, resid=None):
    """(dx, dgamma, dbeta) from the forward's stats [T][2] = (mean, rstd)."""
    dy, x, stats = (np.asarray(a, dtype=np.float64) for a in (dy, x, stats))
    n = x.shape[1]
    rstd = stats[:, 1:]
    xhat = (x - stats[:, :1]) * rstd
    g = dy * _f64(gamma)[mod]
    dx = (g - g.sum(1, keepdims=True) / n - xhat * ((g * xhat).sum(1, keepdims=True) / n)) * rstd
    if resid is not None:
        dx = dx + _f64(resid)
    dgamma = np.stack([(dy * xhat)[mod == m].sum(0) for m in (0, 1)])
    dbeta = np.stack([dy[mod == m].sum(0) for m in (0, 1)])
    return dx, dgamma, dbeta


def linear_fused(x, W, bias, resid, mod, act: str):
    """(out, z): z[t] = x[t] W[m]^T + bias[m], out = act(z) + resid."""
    x, W = np.asarray(x, dtype=np.float64), np.asarray(W, dtype=np.float64)
    z = np.empty((x.shape[0], W.shape[1]))
    for m in (0, 1):
        z[mod == m] = x[mod == m] @ W[m].T
        if bias is not None:
            z[mod == m] += _f64(bias)[m]
    out = mlp_act(z, act)
    return (out if resid is None else out + _f64(resid)), z


def linear_fused_bwd(dout, x, W, z, mod, act: str):
    """(dx, dW, db, dz)."""
    dout, x, W = (np.asarray(a, dtype=np.float64) for a in (dout, x, W))
    dz = dout if act == "none" else dout * mlp_act_grad(z, act)
    dx = np.empty_like(x)
    for m in (0, 1):
        dx[mod == m] = dz[mod == m] @ W[m]
    dW = np.stack([dz[mod == m].T @ x[mod == m] for m in (0, 1)])
    db = np.stack([dz[mod == m].sum(0) for m in (0, 1)])
    return dx, dW, db, dz


def act8_quantize(x):
    """(codes int8 [T][C], scale fp32 [T][ceil(C / 128)]): fp32 arithmetic by
    definition, scale = amax / 127, code = round-half-even(x * (127 / amax)); blocks
    below 2^-100 are zero, blocks with a non-finite value have a NaN scale."""
    x = np.asarray(x, dtype=np.float32)
    T, C = x.shape
    nb = -(-C // ACT8_BLOCK)
    q = np.zeros((T, C), dtype=np.int8)
    scale = np.zeros((T, nb), dtype=np.float32)
    for b in range(nb):
        blk = x[:, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK]
        bad = ~np.isfinite(blk).all(axis=1)
        amax = np.where(bad, np.float32(0), np.abs(np.where(bad[:, None], 0, blk)).max(axis=1))
        amax = amax.astype(np.float32)
        zero = amax < np.float32(2.0 ** -100)
        safe = np.where(zero, np.float32(1), amax).astype(np.float32)
        code = np.rint(np.where(bad[:, None], np.float32(0), blk) * (np.float32(127) / safe)[:, None])
        q[:, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK] = np.where(zero[:, None], 0, code).astype(np.int8)
        scale[:, b] = np.where(zero, np.float32(0), amax / np.float32(127))
        scale[bad, b] = np.nan
    return q, scale


def act8_values(q, scale) -> np.ndarray:
    """The values a checkpoint stands for, code * scale of its block."""
    C = q.shape[1]
    return _f64(q) * _f64(scale)[:, np.arange(C) // ACT8_BLOCK]
