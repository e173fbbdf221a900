"""CPU oracle of streaming attention: plain numpy in fp64, one head at a time.

Visibility of key j to the query at position i, in a sequence of n tokens:
causal: j <= i and (i - j < window or j < sinks); not causal: |i - j| < window or j < sinks.
Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def visible(i, n, window, sinks, causal):
    """Rows of the mask for the query positions `i` over n keys."""
    i = np.asarray(i)[:, None]
    j = np.arange(n)[None, :]
    near = (np.abs(i - j) < window) | (j < sinks)
    return near & (j <= i) if causal else near & (j < n)


def weights(Q, K, mask, scale):
    """Softmax over the visible keys and the logarithm of its sum; a row that sees nothing has no weight."""
    x = np.where(mask, Q @ K.T * scale, -np.inf)
    top = x.max(axis=1, keepdims=True, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(x - safe)
    s = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (safe + np.log(s))[:, 0]
    return e / np.where(s > 0, s, 1.0), lse


def window_head(Q, K, V, window, sinks, causal, scale):
    """O and lse of one head, all of the sequence's tokens."""
    n = Q.shape[0]
    P, lse = weights(Q, K, visible(np.arange(n), n, window, sinks, causal), scale)
    return P @ V, lse, P


def window_head_backward(Q, K, V, dO, window, sinks, causal, scale):
    """dQ, dK, dV of one head."""
    O, _, P = window_head(Q, K, V, window, sinks, causal, scale)
    dP = dO @ V.T
    dS = P * (dP - (dO * O).sum(axis=1, keepdims=True)) * scale
    return dS @ K, dS.T @ Q, P.T @ dO


def round_to(x, dtype):
    """fp64 -> fp32 -> the 16-bit type, each to nearest even, back in fp64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.float64).astype(np.float32)))
    return t.to(dtype).double().numpy()


def rotate(x, cos, sin, interleaved, dtype):
    """A row [d] turned by the angles of its position (cos, sin: [rope_dim / 2]), rounded to dtype."""
    y = np.array(x, np.float64)
    half = len(cos)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    p, q = y[a].copy(), y[b].copy()
    y[a], y[b] = p * cos - q * sin, q * cos + p * sin
    return round_to(y, dtype)


def append_rows(codes, scale, filled, rows):
    """One page of one head: `filled` tokens hold codes of the given scale, `rows` [n, d] follow them.
    Returns the page's codes and its scale (fp32)."""
    rows = np.asarray(rows, np.float64)
    codes = np.array(codes, np.int8)
    old = np.float32(scale) if filled else np.float32(0)
    if not np.isfinite(rows).all() or np.isnan(old):
        return codes, np.float32(np.nan)
    new = np.maximum(old, np.float32(np.float32(np.abs(rows).max()) / np.float32(127)))
    if new > old and filled:
        codes[:filled] = np.rint(codes[:filled].astype(np.float64) * (np.float64(old) / np.float64(new)))
    q = rows / np.float64(new) if new > 0 else np.zeros_like(rows)
    codes[filled:filled + len(rows)] = np.clip(np.rint(q), -127, 127)
    return codes, new
