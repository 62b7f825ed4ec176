"""Further calls of the language-model attention operators on the GPU, against the 64-bit oracle
and against other forms of the same call.

Tolerances of the rotation: outputs are fp32 results rounded once to bf16 (half a step, 2^-8
relative); the fp32 part is within 2^-18 of the pair's magnitude (a few roundings of 2^-24, an
angle of at most half a turn held in fp32, so within 2^-26 turns).
"""
import numpy as np
import pytest

from oracle import lm_ops

from .test_gpu_lm_ops import _expert, check_rope, experts, f64, generator, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (12, 4, 64), (32, 8, 128)])
@pytest.mark.parametrize("tokens", [1, 2])
def test_rotation_in_place_of_single_tokens(experts, hq, hkv, dh, tokens):  # noqa: F811
    """The queries of a decoding step over the projection's own columns, through the binding."""
    import torch
    ex, g = experts(hq, hkv, dh), generator(60 + tokens)
    qkv = normal(g, tokens, (hq + 2 * hkv) * dh)
    pos = torch.arange(70, 70 + tokens, dtype=torch.int32, device="cuda")
    w = normal(g, dh)
    q = torch.empty((tokens, hq * dh), dtype=torch.bfloat16, device="cuda")
    k, v = [torch.zeros((4, hkv * dh), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    ex.qk_norm_rope(qkv, pos, q, k, v, q_norm=w, k_norm=w)
    over = qkv.clone()
    ex.qk_norm_rope(over, pos, over[:, :hq * dh], k2, v2, q_norm=w, k_norm=w)
    ex.synchronize()
    assert torch.equal(over[:, :hq * dh], q) and torch.equal(over[:, hq * dh:], qkv[:, hq * dh:])
    assert torch.equal(k, k2) and torch.equal(v, v2)
    x = f64(qkv).reshape(tokens, hq + 2 * hkv, dh)
    ref = lm_ops.norm_rope(x[:, :hq], f64(w), 0, 1e-6, f64(pos)[None], [0] * (dh // 2), lm_ops.ladder(10000.0, dh))
    check_rope(f64(q).reshape(tokens, hq, dh), ref, "q")


@pytest.mark.parametrize("hq,hkv,dh", [(4, 1, 64), (12, 4, 64), (5, 5, 128), (8, 1, 256)])
@pytest.mark.parametrize("axes,norm,offset,in_place", [(3, True, 1.0, False), (1, False, 0.0, True),
                                                       (2, True, 0.0, True)])
def test_rotation_of_more_tokens_than_warps(experts, hq, hkv, dh, axes, norm, offset, in_place):  # noqa: F811
    """Every warp of the launch (24 a SM) goes on to a second and some to a third token: the next token's pieces,
    positions and cache row are fetched under this one's; rows scattered, some not stored."""
    import torch
    ex, g = experts(hq, hkv, dh), generator(70 + dh + axes)
    tokens = 2 * 24 * ex.info()["sm_count"] + 37
    heads, n_rows = hq + 2 * hkv, tokens + 1001
    qkv = normal(g, tokens, heads * dh, std=2.0)
    w = normal(g, 2, dh)
    pos = torch.randint(-50, 70000, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.randperm(n_rows, generator=g, device="cuda")[:tokens]
    skipped = torch.rand(tokens, generator=g, device="cuda") < 0.1
    rows = torch.where(skipped, torch.full_like(rows, -1), rows)
    over = qkv.clone()
    q = over[:, :hq * dh] if in_place else torch.zeros((tokens, hq * dh), dtype=torch.bfloat16, device="cuda")
    k = torch.full((n_rows, hkv * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 5.0)
    axis = [j % axes for j in range(dh // 2)]
    ex.qk_norm_rope(over, pos, q, k, v, q_norm=w[0] if norm else None, k_norm=w[1] if norm else None,
                    norm_offset=offset, pair_axis=bytes(axis), kv_rows=rows)
    ex.synchronize()
    assert torch.equal(over[:, hq * dh:], qkv[:, hq * dh:])
    kept = np.flatnonzero(~skipped.cpu().numpy())
    where = rows.cpu().numpy()[kept]
    p, f = f64(pos), lm_ops.ladder(10000.0, dh)
    got_q, got_k, got_v = f64(q).reshape(tokens, hq, dh), f64(k), f64(v)
    x = f64(qkv).reshape(tokens, heads, dh)
    check_rope(got_q, lm_ops.norm_rope(x[:, :hq], f64(w[0]) if norm else None, offset, 1e-6, p, axis, f), "q")
    check_rope(got_k[where].reshape(-1, hkv, dh),
               lm_ops.norm_rope(x[kept, hq:hq + hkv], f64(w[1]) if norm else None, offset, 1e-6, p[:, kept], axis, f),
               "k")
    assert (got_v[where].reshape(-1, hkv, dh) == x[kept, hq + hkv:]).all()
    rest = np.setdiff1d(np.arange(n_rows), where)
    assert (got_k[rest] == 7.0).all() and (got_v[rest] == 5.0).all()


def test_rotation_without_a_cache_row(experts):  # noqa: F811
    """Queries alone are rotated: no token has a cache row, and there is no cache."""
    import torch
    hq, hkv, dh, n = 12, 4, 64, 19
    ex, g = experts(hq, hkv, dh), generator(80)
    qkv = normal(g, n, (hq + 2 * hkv) * dh)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    want, q = [torch.empty((n, hq * dh), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k = torch.zeros((n, hkv * dh), dtype=torch.bfloat16, device="cuda")
    ex.qk_norm_rope(qkv, pos, want, k, torch.empty_like(k))
    none = k[:0]
    ex.qk_norm_rope(qkv, pos, q, none, none, kv_rows=torch.full((n,), -1, dtype=torch.int64, device="cuda"))
    ex.synchronize()
    assert torch.equal(q, want)
