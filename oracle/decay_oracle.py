"""Plain float64 oracle of linear attention with a decay per head, its gradients, and rotary positions.

The recurrences are run one token at a time, as written:
  S_t = lambda S_{t-1} + k_t v_t^T,  out_t = S_t^T q_t
  G_t = lambda G_{t+1} + q_t dout_t^T,  dq_t = S_t dout_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t
Arrays are [B, H, L, d], states [B, H, d, d], g = log lambda [H] (-inf: lambda = 0), lengths [B] or None.
Rows at and past a sequence's length come back as zero. Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _lam(g):
    return np.exp(np.asarray(g, dtype=np.float64))[None, :, None, None]


def _inside(B, L, lengths):
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    return n, np.arange(L)[None, :] < n[:, None]


def decay_attention(q, k, v, g, state=None, lengths=None):
    B, H, L, d = q.shape
    lam = _lam(g)
    n, inside = _inside(B, L, lengths)
    S = np.zeros((B, H, d, d)) if state is None else np.array(state, dtype=np.float64)
    out = np.zeros((B, H, L, d))
    with np.errstate(invalid="ignore"):
        for t in range(L):
            live = inside[:, t]
            if not live.any():
                break
            S[live] = lam * S[live] + k[live, :, t, :, None] * v[live, :, t, None, :]
            out[live, :, t] = np.einsum("bhm,bhmn->bhn", q[live, :, t], S[live])
    return out, S


def decay_backward(q, k, v, g, dout, state=None, dstate=None, lengths=None):
    B, H, L, d = q.shape
    lam = _lam(g)
    n, inside = _inside(B, L, lengths)
    S = np.zeros((B, H, d, d)) if state is None else np.array(state, dtype=np.float64)
    dq, dk, dv = np.zeros((3, B, H, L, d))
    for t in range(L):
        live = inside[:, t]
        S[live] = lam * S[live] + k[live, :, t, :, None] * v[live, :, t, None, :]
        dq[live, :, t] = np.einsum("bhmn,bhn->bhm", S[live], dout[live, :, t])
    G = np.zeros((B, H, d, d)) if dstate is None else np.array(dstate, dtype=np.float64)
    for t in reversed(range(L)):
        live = inside[:, t]
        # G arrives here decayed by the step it crossed; beyond the last token it is dstate itself
        G[live] = G[live] + q[live, :, t, :, None] * dout[live, :, t, None, :]
        dk[live, :, t] = np.einsum("bhmn,bhn->bhm", G[live], v[live, :, t])
        dv[live, :, t] = np.einsum("bhmn,bhm->bhn", G[live], k[live, :, t])
        G[live] = lam * G[live]
    return dq, dk, dv, G


def decay_quadratic_head(q, k, v, lam, state=None):
    """One head by the explicit masked matrix: out_i = sum_{j<=i} lam^(i-j) (q_i.k_j) v_j + lam^(i+1) state^T q_i."""
    L = q.shape[0]
    gap = np.arange(L)[:, None] - np.arange(L)[None, :]
    w = np.where(gap >= 0, float(lam) ** np.maximum(gap, 0), 0.0)
    out = (w * (q @ k.T)) @ v
    if state is not None:
        out = out + (float(lam) ** np.arange(1, L + 1))[:, None] * (q @ state)
    return out


def rotary(x, freq, pos, interleaved=False, inverse=False, scale=1.0, rot_scale=1.0):
    """x [B, H, L, d], freq [rot/2], pos [B, L]: each pair as a complex number times e^(i pos freq)."""
    h = len(freq)
    y = np.array(x, dtype=np.float64)
    lo, hi = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if interleaved else (y[..., :h], y[..., h:2 * h])
    a = np.asarray(pos, dtype=np.float64)[:, None, :, None] * np.asarray(freq, dtype=np.float64)
    z = (lo + 1j * hi) * np.exp(-1j * a if inverse else 1j * a) * rot_scale
    if interleaved:
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = z.real, z.imag
    else:
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    return scale * y
