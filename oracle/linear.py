"""FP64 oracle of linear attention with one fixed decay per head, and of its
gradients: the rule token by token, nothing chunked.

  S_t = a S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a = exp(g_h)

Arrays: q, k (B, T, H, dk); v (B, T, H, dv); g (H,); h0 (B, H, dk, dv) or
None.  Packed sequences are the caller's: one call a sequence.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def fwd(q, k, v, g, h0=None):
    """(out, hT)."""
    q, k, v, g = (_f64(x) for x in (q, k, v, g))
    B, T, H, dk = q.shape
    S = np.zeros((B, H, dk, v.shape[-1])) if h0 is None else _f64(h0).copy()
    a = np.exp(g)[None, :, None, None]
    out = np.zeros(v.shape)
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out[:, t] = np.matmul(q[:, t, :, None, :], S)[:, :, 0]
    return out, S


def bwd(q, k, v, g, dout, h0=None, dhT=None):
    """Gradients of <dout, out> + <dhT, hT> as a dict: dq, dk, dv, dh0."""
    q, k, v, g, dout = (_f64(x) for x in (q, k, v, g, dout))
    B, T, H, dk = q.shape
    shape = (B, H, dk, v.shape[-1])
    a = np.exp(g)[None, :, None, None]
    S = np.zeros(shape) if h0 is None else _f64(h0).copy()
    G = np.zeros(shape) if dhT is None else _f64(dhT).copy()
    r = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        r["dq"][:, t] = np.matmul(S, dout[:, t, :, :, None])[..., 0]
    for t in reversed(range(T)):
        G = G + q[:, t, :, :, None] * dout[:, t, :, None, :]
        r["dk"][:, t] = np.matmul(G, v[:, t, :, :, None])[..., 0]
        r["dv"][:, t] = np.matmul(k[:, t, :, None, :], G)[:, :, 0]
        G = a * G
    r["dh0"] = G
    return r


def delta(q, k, v, g, beta, h0):
    """(out, hT) of the gated delta rule; g, beta (B, T, H)."""
    q, k, v, g, beta = (_f64(x) for x in (q, k, v, g, beta))
    S = _f64(h0).copy()
    out = np.zeros(v.shape)
    for t in range(q.shape[1]):
        S = np.exp(g[:, t])[..., None, None] * S
        u = beta[:, t][..., None] * (v[:, t] - np.matmul(k[:, t, :, None, :], S)[:, :, 0])
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = np.matmul(q[:, t, :, None, :], S)[:, :, 0]
    return out, S
