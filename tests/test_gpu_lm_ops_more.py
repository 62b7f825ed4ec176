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
