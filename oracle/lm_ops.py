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


def prefill_prompts(dims, w, emb, cu, positions, axis, freq, causal=True, mask=None, q_norm=None, k_norm=None,
                    offset=0.0):
    """Per-layer K and V of a VLM prefill over packed prompts (the layer of
    ``ae_oracle.prefill_request`` with per-head norms, several rotary axes and
    a causal or bidirectional attention within each prompt).
    emb [tokens, D] -> (K, V) [L, tokens, hkv * dh]."""
    from .ae_oracle import ada_rms, gelu_tanh, modulation
    n, D = emb.shape
    L, hq, hkv, dh = dims.layers, dims.n_q_heads, dims.n_kv_heads, dims.head_dim
    f = lambda x: np.asarray(x, dtype=np.float64)  # noqa: E731
    ks, vs = np.empty((L, n, hkv * dh)), np.empty((L, n, hkv * dh))
    lens = [cu[b + 1] - cu[b] for b in range(len(cu) - 1)]
    h = f(emb)
    for l in range(L):
        s1, sh1, g1 = modulation(np.zeros(D), w["w_mod1"][l], w["b_mod1"][l], 3)
        s2, sh2, g2 = modulation(np.zeros(D), w["w_mod2"][l], w["b_mod2"][l], 3)
        y = ada_rms(h, s1, sh1, dims.rms_eps)
        q, k, v = y @ f(w["wq"][l]).T, y @ f(w["wk"][l]).T, y @ f(w["wv"][l]).T
        rot = lambda x, heads, nw: norm_rope(x.reshape(n, heads, dh), None if nw is None else nw[l], offset,  # noqa
                                             dims.rms_eps, positions, axis, freq).reshape(n, heads * dh)
        q, k = rot(q, hq, q_norm), rot(k, hkv, k_norm)
        ks[l], vs[l] = k, v
        o, _ = packed_attention(q, k, v, hq, hkv, cu, cu[:-1], lens, mask, causal)
        h = h + g1 * (o @ f(w["wo"][l]).T)
        y2 = ada_rms(h, s2, sh2, dims.rms_eps)
        h = h + g2 * ((gelu_tanh(y2 @ f(w["wg"][l]).T) * (y2 @ f(w["wu"][l]).T)) @ f(w["wd"][l]).T)
    return ks, vs
