"""Pins of the language-model operators' oracle against independent forms."""
import numpy as np
import torch

from oracle import lm_ops


def test_norm_rope_matches_complex_rotation_and_torch_rms_norm():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 3, 8)), rng.standard_normal(8)
    pos = np.array([[0, 1, 7, 1000, -3], [4, 4, 0, 2, 9]])
    axis, freq = [0, 1, 0, 1], lm_ops.ladder(100.0, 8)
    got = lm_ops.norm_rope(x, w, 0.0, 1e-6, pos, axis, freq)
    y = torch.nn.functional.rms_norm(torch.from_numpy(x), (8,), torch.from_numpy(w), 1e-6).numpy()
    for t in range(5):
        for j in range(4):
            a = pos[axis[j], t] * 100.0 ** (-2.0 * j / 8)
            r = np.array([[np.cos(a), -np.sin(a)], [np.sin(a), np.cos(a)]])
            np.testing.assert_allclose(got[t][:, [j, j + 4]], y[t][:, [j, j + 4]] @ r.T, atol=1e-12)


def test_rotation_keeps_relative_scores():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    f = lm_ops.ladder(10000.0, 16)

    def score(i, j):
        a = lm_ops.norm_rope(q, None, 0, 0, [[i]], [0] * 8, f)
        b = lm_ops.norm_rope(k, None, 0, 0, [[j]], [0] * 8, f)
        return float((a * b).sum())
    assert abs(score(5, 2) - score(1005, 1002)) < 1e-9


def test_packed_attention_matches_torch():
    rng = np.random.default_rng(2)
    hq, hkv, dh = 4, 2, 8
    cu, row0, lens = [0, 3, 3, 8], [2, 0, 6], [3, 0, 9]
    q = rng.standard_normal((8, hq * dh))
    k, v = rng.standard_normal((15, hkv * dh)), rng.standard_normal((15, hkv * dh))
    got, _ = lm_ops.packed_attention(q, k, v, hq, hkv, cu, row0, lens)
    for b in (0, 2):
        n, m = cu[b + 1] - cu[b], lens[b]
        bias = torch.full((n, m), 0.0, dtype=torch.float64)
        bias.masked_fill_(~torch.ones(n, m, dtype=torch.bool).tril(m - n), -torch.inf)
        tq = torch.from_numpy(q[cu[b]:cu[b + 1]]).view(n, hq, dh).transpose(0, 1)
        tk = torch.from_numpy(k[row0[b]:row0[b] + m]).view(m, hkv, dh).transpose(0, 1).repeat_interleave(2, 0)
        tv = torch.from_numpy(v[row0[b]:row0[b] + m]).view(m, hkv, dh).transpose(0, 1).repeat_interleave(2, 0)
        ref = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=bias)
        np.testing.assert_allclose(got[cu[b]:cu[b + 1]], ref.transpose(0, 1).reshape(n, hq * dh).numpy(), atol=1e-12)


def test_rows_without_keys_are_zero():
    q, k, v = np.ones((2, 8)), np.full((2, 8), np.nan), np.full((2, 8), np.nan)
    out, _ = lm_ops.packed_attention(q, k, v, 1, 1, [0, 2], [0], [2], mask=np.zeros(2, np.uint8))
    assert (out == 0).all()
