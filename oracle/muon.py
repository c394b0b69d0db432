"""Muon's update, plain NumPy. The two element passes follow the kernels'
definition (fp32, one rounding per operation); the orthogonalisation is the
iteration itself in float64."""

import numpy as np

from .zero_step import narrow, widen

QUINTIC = (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-7


def muon_momentum(grads, dtype, m, grad_scale, mu, nesterov, update_dtype):
    """(new m fp32, update) from grads (bit patterns of dtype, or fp32)."""
    f = np.float32
    mu = f(mu)
    omu = f(1.0) - mu
    g = widen(grads, dtype) * f(grad_scale)
    t = omu * g
    m = mu * m + t
    u = mu * m + t if nesterov else m
    return m, (u.astype(f) if update_dtype == "fp32" else narrow(u, update_dtype))


def newton_schulz(g, steps=5, coef=None):
    """Float64 iteration on one matrix (rows x cols, float64)."""
    x = g / (np.sqrt((g * g).sum()) + NORM_EPS)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for k in range(steps):
        a, b, c = np.float32(QUINTIC if coef is None else coef[k]).astype(np.float64)
        w = x @ x.T
        x = a * x + (b * w + c * (w @ w)) @ x
    return x.T if tall else x


def muon_scale(rows, cols, mode):
    if mode == "aspect":
        return np.float32(np.sqrt(max(1.0, rows / cols)))
    return np.float32(0.2 * np.sqrt(max(rows, cols))) if mode == "rms" else np.float32(1.0)


def muon_apply(update, update_dtype, p, rows, cols, lr, wd, mode, param_dtype):
    """(new master fp32, params bit patterns) of one matrix, flat arrays."""
    f = np.float32
    lr = np.float64(f(lr))
    decay = f(1.0 - lr * np.float64(f(wd)))
    fac = f(lr * np.float64(muon_scale(rows, cols, mode)))
    p = p * decay
    p = p - fac * widen(update, update_dtype)
    return p, narrow(p, param_dtype)
