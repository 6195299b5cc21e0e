"""TEST INFRASTRUCTURE ONLY: fp64 token loop of the gated linear recurrence
and of its gradients, written from the definition

    h_t = alpha_t h_{t-1} + x_t,   out_t = h_t,   alpha = e^{log_alpha}

per sequence and channel, with alpha = 1, one per token and head, or one per
token and channel.  Pinned in tests/test_linear_norm_host.py by closed forms
(a prefix sum, a geometric series), by splitting a sequence, and, the
gradients, by central differences of the forward loop.
"""
from __future__ import annotations

import numpy as np


def _arrays(x, log_alpha, initial_state, cu_seqlens):
    """Tokens flattened to [n, H, d]; alpha [n, H, d or 1]; the offsets."""
    x = np.asarray(x, np.float64)
    B, T, H, d = x.shape
    cu = (np.arange(B + 1) * T if cu_seqlens is None
          else np.asarray(cu_seqlens, np.int64))
    x = x.reshape(B * T, H, d)
    if log_alpha is None:
        a = np.ones((B * T, 1, 1))
    else:
        a = np.exp(np.asarray(log_alpha, np.float64))
        a = a.reshape(B * T, H, d if a.ndim == 4 else 1)
    n = len(cu) - 1
    s0 = (np.zeros((n, H, d)) if initial_state is None
          else np.asarray(initial_state, np.float64))
    return x, a, s0, cu


def linear_fwd(x, log_alpha=None, initial_state=None, cu_seqlens=None):
    """(out [B, T, H, d], final state [N, H, d], alpha_t h_{t-1} of every
    token [B, T, H, d]); rows outside every sequence are 0."""
    shape = np.shape(x)
    x, a, s0, cu = _arrays(x, log_alpha, initial_state, cu_seqlens)
    out, ah = np.zeros_like(x), np.zeros_like(x)
    final = s0.copy()
    for n in range(len(cu) - 1):
        h = s0[n]
        for t in range(cu[n], cu[n + 1]):
            ah[t] = a[t] * h
            h = ah[t] + x[t]
            out[t] = h
        final[n] = h
    return out.reshape(shape), final, ah.reshape(shape)


def linear_grads(x, log_alpha, initial_state, d_out, d_final_state=None,
                 cu_seqlens=None):
    """dict of dx, dlog_alpha (None without a decay) and dinitial_state."""
    shape = np.shape(x)
    _, _, ah = linear_fwd(x, log_alpha, initial_state, cu_seqlens)
    xf, a, s0, cu = _arrays(x, log_alpha, initial_state, cu_seqlens)
    ah = ah.reshape(xf.shape)
    dout = np.asarray(d_out, np.float64).reshape(xf.shape)
    G = np.zeros_like(xf)
    ds0 = np.zeros_like(s0)
    for n in range(len(cu) - 1):
        c = (np.zeros_like(s0[n]) if d_final_state is None
             else np.asarray(d_final_state, np.float64)[n])
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G[t] = dout[t] + c
            c = a[t] * G[t]
        ds0[n] = c
    dla = None
    if log_alpha is not None:
        dla = G * ah
        if np.ndim(log_alpha) == 3:
            dla = dla.sum(-1)
        dla = dla.reshape(np.shape(log_alpha))
    return dict(dx=G.reshape(shape), dlog_alpha=dla, dinitial_state=ds0)
