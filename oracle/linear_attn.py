"""fp64 oracle of linear attention with a decay for each head and of rotary positions
(test infrastructure, numpy on the host): the recursions token by token, as written down,
with none of the chunk algebra of the CUDA path.

    S_t = gamma S_{t-1} + k_t^T v_t,   z_t = scale q_t S_t,   gamma = exp(log_decay[head])

Arrays are [B, H, T, d] (q, k, v), [H] (log_decay), [B, H, d, d] (states), [B] (lengths)."""
from __future__ import annotations

import numpy as np


def _ends(B, T, lengths):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, T)


def forward(q, k, v, log_decay, scale, S0=None, lengths=None):
    """(Z [B,H,T,d], S [B,H,d,d]): rows of Z behind a sequence's end are zeros."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, T, d = q.shape
    gamma = np.exp(np.asarray(log_decay, np.float64))
    Z = np.zeros((B, H, T, d))
    S = np.zeros((B, H, d, d)) if S0 is None else np.array(S0, np.float64)
    for b, n in enumerate(_ends(B, T, lengths)):
        for t in range(n):
            S[b] = gamma[:, None, None] * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            Z[b, :, t] = scale * np.einsum("hi,hij->hj", q[b, :, t], S[b])
    return Z, S


def backward(q, k, v, log_decay, scale, dZ, S0=None, dS_T=None, lengths=None):
    """Gradients of <dZ, Z> + <dS_T, S>: {"dQ", "dK", "dV", "dS0"}, by the chain rule along the
    recursion (states kept, the tokens of each sequence from its end)."""
    q, k, v, dZ = (np.asarray(x, np.float64) for x in (q, k, v, dZ))
    B, H, T, d = q.shape
    gamma = np.exp(np.asarray(log_decay, np.float64))
    out = {n: np.zeros((B, H, T, d)) for n in ("dQ", "dK", "dV")}
    out["dS0"] = np.zeros((B, H, d, d))
    for b, n in enumerate(_ends(B, T, lengths)):
        S = np.zeros((H, d, d)) if S0 is None else np.array(S0[b], np.float64)
        for t in range(n):
            S = gamma[:, None, None] * S + k[b, :, t, :, None] * v[b, :, t, None, :]
            out["dQ"][b, :, t] = scale * np.einsum("hij,hj->hi", S, dZ[b, :, t])
        G = np.zeros((H, d, d)) if dS_T is None else np.array(dS_T[b], np.float64)
        for t in range(n - 1, -1, -1):
            G = G + scale * q[b, :, t, :, None] * dZ[b, :, t, None, :]
            out["dK"][b, :, t] = np.einsum("hij,hj->hi", G, v[b, :, t])
            out["dV"][b, :, t] = np.einsum("hi,hij->hj", k[b, :, t], G)
            G = gamma[:, None, None] * G
        out["dS0"][b] = G
    return out


def rope(x, positions, inv_freq, mscale=1.0, interleaved=False, inverse=False):
    """Rows x [B, H, T, d] turned at positions [B, T]: pairs as complex numbers."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    if not half:
        return x
    angle = np.asarray(positions, np.float64)[:, None, :, None] * np.asarray(inv_freq, np.float64)
    turn = mscale * np.exp((-1j if inverse else 1j) * angle)
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    w = (x[..., first] + 1j * x[..., second]) * turn
    x[..., first], x[..., second] = w.real, w.imag
    return x
