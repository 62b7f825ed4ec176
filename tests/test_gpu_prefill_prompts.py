"""ae_prefill_prompts against the oracle: packed prompts of different lengths,
causal or bidirectional, per-head norms, several rotary axes, masked tokens;
every layer's K and V within relative L2 1e-2 (the bf16 tolerance of the
prefill's hidden values), and the chain prefill -> bind -> sample.
"""
import dataclasses

import numpy as np
import pytest

from flow_matching_action_gb300 import synth
from oracle import ae_oracle, lm_ops

from .helpers import GpuRunner, device_weights, oracle_actions

pytestmark = pytest.mark.gpu


def rel_l2(a, b):
    return float(np.sqrt(((a - b) ** 2).sum()) / np.sqrt((b ** 2).sum()))


def bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Prefill:
    def __init__(self, dims, w, batch, fp8_weights=False):
        from flow_matching_action_gb300 import ae
        self.d, self.ex = dims, ae.ActionExpert(dims, device_weights(w, "bf16"), batch, 0, dtype="bf16",
                                                fp8_weights=fp8_weights)

    def __call__(self, emb, cu, positions, mask=None, q_norm=None, k_norm=None, **kw):
        import torch
        n = emb.shape[0]
        k = torch.empty((self.d.layers, n, self.d.kv_dim), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        self.ex.prefill_prompts(emb, cu, torch.from_numpy(np.asarray(positions, dtype=np.int32)).cuda(), k, v,
                                token_mask=None if mask is None else torch.from_numpy(mask).cuda(),
                                q_norm=q_norm, k_norm=k_norm, **kw)
        self.ex.synchronize()
        return k, v


def check(got, ref, rows=None):
    for l in range(ref.shape[0]):
        a, b = f64(got[l]), ref[l]
        if rows is not None:
            a, b = a[rows], b[rows]
        assert rel_l2(a, b) <= 1e-2, (l, rel_l2(a, b))


TINY = dataclasses.replace(synth.TINY_VLM, dtype="bf16")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("norm", [False, True])
def test_packed_prompts_match_oracle(causal, norm):
    w = synth.make_vlm_weights(TINY, 3)
    emb = synth.prefix_embeddings(TINY, 3, 2)[:89]
    cu = [0, 17, 17, 18, 61, 89]
    rng = np.random.default_rng(0)
    pos = rng.integers(0, 500, (3, 89))
    half = TINY.head_dim // 2
    axis = [j % 3 for j in range(half)]
    qn, kn = ([synth.round_to_bf16(0.3 * rng.standard_normal(TINY.head_dim).astype(np.float32))
               for _ in range(TINY.layers)] for _ in range(2))
    p = Prefill(TINY, w, 2)
    try:
        kw = dict(norm_offset=1.0, pair_axis=bytes(axis), causal=causal)
        k, v = p(bf16(emb), cu, pos, q_norm=[bf16(x) for x in qn] if norm else None,
                 k_norm=[bf16(x) for x in kn] if norm else None, **kw)
    finally:
        p.ex.close()
    rk, rv = lm_ops.prefill_prompts(TINY, w, emb, cu, pos, axis, lm_ops.ladder(TINY.rope_theta, TINY.head_dim), causal,
                                    None, qn if norm else None, kn if norm else None, 1.0)
    check(k, rk)
    check(v, rv)


@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 1, 2], [0, 7, 7]])
def test_shortest_prompts(cu):
    w = synth.make_vlm_weights(TINY, 9)
    n, half = cu[-1], TINY.head_dim // 2
    emb = synth.prefix_embeddings(TINY, 9, 1)[:n]
    pos = np.arange(n)[None]
    p = Prefill(TINY, w, 1)
    try:
        k, v = p(bf16(emb), cu, pos)
    finally:
        p.ex.close()
    rk, rv = lm_ops.prefill_prompts(TINY, w, emb, cu, pos, [0] * half, lm_ops.ladder(TINY.rope_theta, TINY.head_dim))
    check(k, rk)
    check(v, rv)


def test_equal_bidirectional_prompts_match_the_prefill_oracle():
    """Prompts of one length, bidirectional, one axis, no norms: the values of ae_prefill."""
    w = synth.make_vlm_weights(TINY, 4)
    emb = synth.prefix_embeddings(TINY, 4, 2)
    n = TINY.horizon
    p = Prefill(TINY, w, 2)
    try:
        k, v = p(bf16(emb), [0, n, 2 * n], np.concatenate([np.arange(n)] * 2), causal=False)
    finally:
        p.ex.close()
    ref = [ae_oracle.prefill_request(TINY, w, emb[b * n:(b + 1) * n]) for b in (0, 1)]
    check(k, np.concatenate([r[0] for r in ref], 1))
    check(v, np.concatenate([r[1] for r in ref], 1))


def test_masked_tokens_reach_nothing():
    """Masked tokens' embeddings are NaN; the other rows are those of the oracle."""
    w = synth.make_vlm_weights(TINY, 5)
    emb = synth.prefix_embeddings(TINY, 5, 2)[:70]
    mask = np.ones(70, dtype=np.uint8)
    mask[[0, 1, 30, 31, 32, 50, 69]] = 0
    cu, half = [0, 40, 70], TINY.head_dim // 2
    pos = np.concatenate([np.cumsum(mask[:40]) - 1, np.cumsum(mask[40:]) - 1])[None]
    bad = emb.copy()
    bad[mask == 0] = np.nan
    p = Prefill(TINY, w, 2)
    try:
        k, v = p(bf16(bad), cu, pos, mask=mask, causal=True)
    finally:
        p.ex.close()
    rk, rv = lm_ops.prefill_prompts(TINY, w, emb, cu, pos, [0] * half, lm_ops.ladder(TINY.rope_theta, TINY.head_dim),
                                    True, mask)
    check(k, rk, mask != 0)
    check(v, rv, mask != 0)


def test_pi05_vlm_widths_ragged():
    """The widths of Pi0.5's VLM, two ragged causal prompts in the room of one 712-token request."""
    d = synth.PI05_VLM_2L
    w = synth.make_vlm_weights(d, 0)
    emb = synth.prefix_embeddings(d, 0, 1)[:700]
    cu = [0, 411, 700]
    pos = np.concatenate([np.arange(411), np.arange(289)])[None]
    p = Prefill(d, w, 1)
    try:
        k, v = p(bf16(emb), cu, pos)
    finally:
        p.ex.close()
    rk, rv = lm_ops.prefill_prompts(d, w, emb, cu, pos, [0] * (d.head_dim // 2),
                                    lm_ops.ladder(d.rope_theta, d.head_dim))
    check(k, rk)
    check(v, rv)


def test_fp8_weights():
    w = synth.make_vlm_weights(TINY, 6)
    emb = synth.prefix_embeddings(TINY, 6, 1)
    n = TINY.horizon
    cu, pos = [0, 20, n], np.concatenate([np.arange(20), np.arange(n - 20)])[None]
    p = Prefill(TINY, w, 1, fp8_weights=True)
    try:
        k, v = p(bf16(emb), cu, pos)
    finally:
        p.ex.close()
    w8 = ae_oracle.fp8_expert_weights(w)[0]
    rk, rv = lm_ops.prefill_prompts(TINY, w8, emb, cu, pos, [0] * (TINY.head_dim // 2),
                                    lm_ops.ladder(TINY.rope_theta, TINY.head_dim))
    check(k, rk)
    check(v, rv)


def test_prefilled_prompts_drive_the_action_expert_and_keep_the_binding():
    """Ragged prefill -> bind_prefix -> sample against the oracle's chain; a prefill on a bound
    context leaves its binding in place."""
    import torch
    from flow_matching_action_gb300 import ae
    de = dataclasses.replace(synth.TINY, dtype="bf16")
    wv, we = synth.make_vlm_weights(TINY, 7), synth.make_weights(de, 7)
    cu = [0, 31, 75]
    emb = synth.prefix_embeddings(TINY, 7, 2)[:75]
    pos = np.concatenate([np.arange(31), np.arange(44)])[None]
    p = Prefill(TINY, wv, 2)
    try:
        k, v = p(bf16(emb), cu, pos)
    finally:
        p.ex.close()
    rk, rv = lm_ops.prefill_prompts(TINY, wv, emb, cu, pos, [0] * (TINY.head_dim // 2),
                                    lm_ops.ladder(TINY.rope_theta, TINY.head_dim))
    wl = synth.build_workload("prompts", de, 2, [[("v", 31)], [("v", 44)]], seed=7)
    wl_ref = dataclasses.replace(wl, prefix_k=rk, prefix_v=rv)
    ref = oracle_actions(wl_ref, we)
    r = GpuRunner(de, we, dtype="bf16", max_batch=5, max_rows=64)
    try:
        noise = torch.from_numpy(wl.noise).cuda()
        r.expert.bind_prefix(k, v, cu)
        got = r.expert.sample(noise, wl.n_steps)
        r.expert.synchronize()
        assert np.abs(f64(got) - ref).max() <= 1e-2
        # the expert's own context runs a prefill over other prompts in between
        kk = torch.empty((de.layers, 75, de.kv_dim), dtype=torch.bfloat16, device="cuda")
        r.expert.prefill_prompts(bf16(emb), cu, torch.from_numpy(pos.astype(np.int32)).cuda(), kk, torch.empty_like(kk))
        again = r.expert.sample(noise, wl.n_steps)
        r.expert.synchronize()
        assert torch.equal(got, again)
    finally:
        r.close()


def test_too_many_tokens_are_refused():
    import torch
    from flow_matching_action_gb300 import ae
    w = synth.make_vlm_weights(TINY, 8)
    p = Prefill(TINY, w, 1)
    try:
        n = TINY.horizon + 1
        with pytest.raises(ae.AEError) as e:
            p(torch.zeros((n, TINY.width), dtype=torch.bfloat16, device="cuda"), [0, n], np.zeros((1, n)))
        assert e.value.status == -2
    finally:
        p.ex.close()
