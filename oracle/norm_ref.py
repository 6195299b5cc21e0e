"""TEST INFRASTRUCTURE ONLY: fp64 layer normalisation of [tokens, H, d] and
its gradients, from the definition.  Pinned in tests/test_linear_norm_host.py
by the mean and variance of its output and by central differences."""
from __future__ import annotations

import numpy as np


def _stats(x, eps):
    x = np.asarray(x, np.float64)
    c = x - x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c, rstd


def layer_norm(x, weight, bias, eps):
    c, rstd = _stats(x, eps)
    y = c * rstd
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y


def layer_norm_grads(x, weight, d_out, eps):
    """dict of dx [n, H, d], dweight and dbias [H, d]."""
    c, rstd = _stats(x, eps)
    dy = np.asarray(d_out, np.float64)
    xh = c * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(-1, keepdims=True)
                 - xh * (g * xh).mean(-1, keepdims=True))
    return dict(dx=dx, dweight=(dy * xh).sum(0), dbias=dy.sum(0))
