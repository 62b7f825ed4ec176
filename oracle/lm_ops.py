"""float64 NumPy oracle of the language-model attention operators.

Written from the operators' formulas alone (per-head RMS norm and rotation,
softmax attention of packed sequences and of single tokens), shared by no code
of the library.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, w, offset, eps, positions, axis, freq):
    """x [tokens, heads, dh] -> rotated heads; w [dh] or None; positions [axes, tokens]."""
    x = np.asarray(x, dtype=np.float64)
    dh = x.shape[-1]
    half = dh // 2
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (offset + np.asarray(w, dtype=np.float64))
    phi = np.asarray(positions, dtype=np.float64)[np.asarray(axis)].T * np.asarray(freq)  # [tokens, half]
    z = (x[..., :half] + 1j * x[..., half:]) * np.exp(1j * phi)[:, None, :]
    return np.concatenate([z.real, z.imag], axis=-1)


def ladder(theta, dh):
    return theta ** (-2.0 * np.arange(dh // 2) / dh)


def attend(q, k, v, seen, scale):
    """One head: q [n, dh], k / v [m, dh], seen [n, m] -> (out, sum_j p_j |v_j|), zeros without keys."""
    n, m = q.shape[0], k.shape[0]
    if m == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = np.where(seen, q @ k.T * scale, -np.inf)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    l = p.sum(-1, keepdims=True)
    p = p / np.where(l > 0, l, 1.0)
    return p @ v, p @ np.abs(v)


def packed_attention(q, k, v, hq, hkv, cu_q, row0, lens, mask=None, causal=True, scale=None):
    """q [rows, hq dh], k / v [cache rows, hkv dh] float64 -> (out, weighted |v|) [rows, hq dh]."""
    dh = q.shape[1] // hq
    scale = 1.0 / np.sqrt(dh) if not scale else scale
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for b in range(len(cu_q) - 1):
        q0, q1, r, m = cu_q[b], cu_q[b + 1], row0[b], lens[b]
        n = q1 - q0
        seen = np.ones((n, m), dtype=bool)
        if causal:
            seen = np.arange(m)[None, :] <= (m - n + np.arange(n))[:, None]
        kb, vb = k[r:r + m].copy(), v[r:r + m].copy()
        if mask is not None:
            on = mask[r:r + m] != 0
            seen = seen & on[None, :]
            kb[~on] = 0.0  # never read: whatever they hold
            vb[~on] = 0.0
        for h in range(hq):
            c = slice(h * dh, (h + 1) * dh)
            g = slice((h // (hq // hkv)) * dh, (h // (hq // hkv) + 1) * dh)
            out[q0:q1, c], mag[q0:q1, c] = attend(q[q0:q1, c], kb[:, g], vb[:, g], seen, scale)
    return out, mag
