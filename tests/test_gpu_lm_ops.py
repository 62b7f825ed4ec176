"""Language-model attention operators on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic of the operators:
* rotation: outputs are fp32 results rounded once to bf16 (half a step, 2^-8
  relative); the fp32 part is within 2^-18 of the pair's magnitude (a few
  roundings of 2^-24, an angle error of 2^-33 turns).
* attention: the softmax weights are rounded to bf16 before they meet V (2^-8
  of each term, so 2^-8 sum_j p_j |v_j| at most), the output once more (2^-8 of
  itself); fp32 scores, exponentials and sums add less than
  2^-12 sum_j p_j |v_j| at these sizes.
"""
import ctypes

import numpy as np
import pytest

from flow_matching_action_gb300 import ae, synth
from oracle import lm_ops

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def _expert(hq, hkv, dh, theta=10000.0, stream=None):
    import torch
    dims = synth.ExpertDims(layers=1, width=128, mlp=128, n_q_heads=hq, n_kv_heads=hkv, head_dim=dh, horizon=1,
                            action_dim=8, dtype="bf16", rope_theta=theta)
    w = {n: torch.zeros(s, dtype=torch.bfloat16, device="cuda") for n, s in synth.global_weight_shapes(dims)}
    for n, s in synth.layer_weight_shapes(dims):
        w[n] = [torch.zeros(s, dtype=torch.bfloat16, device="cuda")]
    return ae.ActionExpert(dims, w, 1, 0, stream=stream)


@pytest.fixture(scope="module")
def experts():
    made = {}

    def get(hq, hkv, dh, theta=10000.0):
        key = (hq, hkv, dh, theta)
        if key not in made:
            made[key] = _expert(*key)
        return made[key]
    yield get
    for e in made.values():
        e.close()


def normal(gen, *shape, std=1.0):
    import torch
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def generator(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def f64(t):
    return t.double().cpu().numpy()


def strided(t, pad):
    """The same rows inside wider rows of NaN."""
    import torch
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


# ---------------------------------------------------------------- norm + rotation

def check_rope(got, ref, what):
    half = ref.shape[-1] // 2
    amp = np.sqrt(ref[..., :half] ** 2 + ref[..., half:] ** 2)
    tol = HALF * np.abs(ref) + 2.0 ** -18 * np.concatenate([amp, amp], -1) * 2
    bad = np.abs(got - ref) - tol
    assert bad.max() <= 0, (what, bad.max())


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (4, 1, 64), (12, 4, 64), (5, 5, 128), (32, 8, 128), (16, 2, 128)])
@pytest.mark.parametrize("tokens,axes,norm,offset,scatter", [
    (1, 1, True, 0.0, False), (3, 2, True, 1.0, True), (37, 3, False, 0.0, True), (1301, 4, True, 0.0, False)])
def test_qk_norm_rope(experts, hq, hkv, dh, tokens, axes, norm, offset, scatter):
    import torch
    ex, g = experts(hq, hkv, dh), generator(tokens + dh)
    qkv = normal(g, tokens, (hq + 2 * hkv) * dh, std=2.0)
    qn, kn = normal(g, dh), normal(g, dh)
    pos = torch.randint(-50, 70000, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.randperm(2 * tokens + 5, generator=g, device="cuda")[:tokens] if scatter else None
    n_rows = 2 * tokens + 5
    q_out = torch.full((tokens, hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    k_cache = torch.full((n_rows, hkv * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.full_like(k_cache, 5.0)
    axis = [j % axes for j in range(dh // 2)]
    ex.qk_norm_rope(qkv, pos, q_out, k_cache, v_cache, q_norm=qn if norm else None, k_norm=kn if norm else None,
                    norm_offset=offset, pair_axis=bytes(axis), kv_rows=rows)
    ex.synchronize()
    x = f64(qkv).reshape(tokens, hq + 2 * hkv, dh)
    args = (offset, 1e-6, f64(pos), axis, lm_ops.ladder(10000.0, dh))
    check_rope(f64(q_out).reshape(tokens, hq, dh), lm_ops.norm_rope(x[:, :hq], f64(qn) if norm else None, *args), "q")
    where = rows.cpu().numpy() if scatter else np.arange(tokens)
    check_rope(f64(k_cache)[where].reshape(tokens, hkv, dh),
               lm_ops.norm_rope(x[:, hq:hq + hkv], f64(kn) if norm else None, *args), "k")
    assert (f64(v_cache)[where].reshape(tokens, hkv, dh) == x[:, hq + hkv:]).all()
    rest = np.setdiff1d(np.arange(n_rows), where)  # rows no token names are left alone
    assert (f64(k_cache)[rest] == 7.0).all() and (f64(v_cache)[rest] == 5.0).all()


def test_rope_far_positions_and_given_frequencies(experts):
    """int32 positions up to the ends of their range, frequencies given by the caller (one of them 0)."""
    import torch
    hq, hkv, dh = 4, 1, 64
    ex, g = experts(hq, hkv, dh), generator(3)
    pos = torch.tensor([[0, 1, 2 ** 31 - 1, -2 ** 31, 16777217, 999999937]], dtype=torch.int32, device="cuda")
    n = pos.shape[1]
    # frequencies with few bits, so that pos * freq is exact in the oracle's 64 bits
    freq = [0.0] + [2.0 ** -(j % 12) for j in range(1, dh // 2)]
    qkv = normal(g, n, (hq + 2 * hkv) * dh)
    q = torch.empty((n, hq * dh), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((n, hkv * dh), dtype=torch.bfloat16, device="cuda")
    ex.qk_norm_rope(qkv, pos, q, k, torch.empty_like(k), pair_freq=freq)
    ex.synchronize()
    x = f64(qkv).reshape(n, hq + 2 * hkv, dh)
    ref = lm_ops.norm_rope(x[:, :hq], None, 0, 0, f64(pos), [0] * (dh // 2), freq)
    got = f64(q).reshape(n, hq, dh)
    assert (got[..., 0] == x[:, :hq, 0]).all()  # frequency 0: not rotated
    # a frequency is held as a 64-bit fraction of a turn made from a double: 2^-54 of it
    # times 2^31 positions is 2^-23 turns, 2^-20 radians
    half = dh // 2
    amp = np.sqrt(ref[..., :half] ** 2 + ref[..., half:] ** 2)
    tol = HALF * np.abs(ref) + 2.0 ** -17 * np.concatenate([amp, amp], -1)
    assert (np.abs(got - ref) <= tol).all()


def test_rope_frequencies_above_one_turn(experts):
    """Frequencies of many turns a position, at far positions: the angle modulo one turn in exact
    arithmetic (80 digits of pi).  Its fp32 sine and cosine are good to 2^-18."""
    import torch
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)
    hq, hkv, dh = 4, 1, 64
    ex, g = experts(hq, hkv, dh), generator(4)
    positions = [1, -7, 2 ** 31 - 1, -2 ** 31, 1234567891]
    pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
    half = dh // 2
    freq = [(-1) ** j * 1.0001 * 1.9 ** j for j in range(half)]
    n = len(positions)
    qkv = normal(g, n, (hq + 2 * hkv) * dh)
    q = torch.empty((n, hq * dh), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((n, hkv * dh), dtype=torch.bfloat16, device="cuda")
    ex.qk_norm_rope(qkv, pos, q, k, torch.empty_like(k), pair_freq=freq)
    ex.synchronize()
    phi = np.array([[float(p * Fraction(f) / two_pi % 1) for f in freq] for p in positions])[:, None] * 2 * np.pi
    x = f64(qkv).reshape(n, hq + 2 * hkv, dh)[:, :hq]
    lo, hi = x[..., :half], x[..., half:]
    ref = np.concatenate([lo * np.cos(phi) - hi * np.sin(phi), hi * np.cos(phi) + lo * np.sin(phi)], -1)
    check_rope(f64(q).reshape(n, hq, dh), ref, "q")


def test_rope_in_place_strides_and_skipped_rows(experts):
    """q written over the projection's own columns, wide rows, tokens without a cache row, a row
    beyond the cache reported and skipped."""
    import torch
    hq, hkv, dh, n = 12, 4, 64, 21
    ex, g = _expert(hq, hkv, dh), generator(4)
    try:
        qkv = normal(g, n, (hq + 2 * hkv) * dh)
        wide, view = strided(qkv, 40)
        kw, kview = strided(torch.zeros((n, hkv * dh), dtype=torch.bfloat16, device="cuda"), 24)
        vw, vview = strided(torch.zeros((n, hkv * dh), dtype=torch.bfloat16, device="cuda"), 24)
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        rows = torch.arange(n, dtype=torch.int64, device="cuda")
        rows[5] = -1
        # in place: q_out is the same memory with the same stride
        a = ae.ae_qk_norm_rope_args(tokens=n, n_axes=1, qkv=wide.data_ptr(), qkv_stride=wide.stride(0),
                                    positions=pos.data_ptr(), kv_rows=rows.data_ptr(), cache_rows=n,
                                    q_out=wide.data_ptr(), q_stride=wide.stride(0), k_cache=kw.data_ptr(),
                                    v_cache=vw.data_ptr(), kv_stride=kw.stride(0))
        ae.ae_qk_norm_rope(ex.ctx, a)
        ex.synchronize()
        x = f64(qkv).reshape(n, hq + 2 * hkv, dh)
        args = (0, 0, f64(pos)[None], [0] * (dh // 2), lm_ops.ladder(10000.0, dh))
        check_rope(f64(view)[:, :hq * dh].reshape(n, hq, dh), lm_ops.norm_rope(x[:, :hq], None, *args), "q")
        assert (f64(view)[:, hq * dh:] == f64(qkv)[:, hq * dh:]).all()
        assert torch.isnan(wide[:, qkv.shape[1]:]).all() and torch.isnan(kw[:, hkv * dh:]).all()
        kept = [i for i in range(n) if i != 5]
        check_rope(f64(kview)[kept].reshape(-1, hkv, dh), lm_ops.norm_rope(x[kept, hq:hq + hkv], None, *args[:2],
                                                                         f64(pos)[None][:, kept], *args[3:]), "k")
        assert (f64(kview)[5] == 0).all() and (f64(vview)[5] == 0).all()
        # a row beyond the cache: not stored, and the context says so
        rows[7] = n
        before = kw.clone()
        ae.ae_qk_norm_rope(ex.ctx, ae.ae_qk_norm_rope_args(
            tokens=n, n_axes=1, qkv=qkv.data_ptr(), qkv_stride=qkv.stride(0), positions=pos.data_ptr(),
            kv_rows=rows.data_ptr(), cache_rows=n, q_out=torch.empty_like(qkv).data_ptr(), q_stride=qkv.stride(0),
            k_cache=kw.data_ptr(), v_cache=vw.data_ptr(), kv_stride=kw.stride(0)))
        with pytest.raises(ae.AEError) as e:
            ex.synchronize()
        assert e.value.status == -5
        assert (before[7].view(torch.int16) == kw[7].view(torch.int16)).all()
        with pytest.raises(ae.AEError):
            ae.ae_qk_norm_rope(ex.ctx, a)
    finally:
        ex.close()


# ---------------------------------------------------------------- prompt attention

def check_attention(got, ref, mag, what=""):
    assert np.isfinite(got).all(), what
    tol = HALF * np.abs(ref) + (HALF + 2.0 ** -12) * mag
    bad = np.abs(got - ref) - tol
    assert bad.max() <= 0, (what, bad.max(), np.unravel_index(bad.argmax(), bad.shape))


def run_prompt(ex, hq, hkv, dh, new, cached, masked=None, causal=True, scale=0.0, seed=0, gap=0, nan_outside=True,
               std=1.5, packed=False):
    """Packed prompts whose cache rows lie `gap` rows apart, everything that is not theirs NaN."""
    import torch
    g = generator(seed)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    lens = [n + c for n, c in zip(new, cached)]
    row0, r = [], 0 if packed else gap
    for m in lens:
        row0.append(r)
        r += m + (0 if packed else gap)
    rows = max(r, 1)
    q = normal(g, cu[-1] + 3, hq * dh, std=std)
    k, v = normal(g, rows, hkv * dh), normal(g, rows, hkv * dh)
    mask = None
    if masked is not None:
        mask = torch.ones(rows, dtype=torch.uint8, device="cuda")
        for m, r0 in zip(lens, row0):
            on = torch.rand(m, generator=g, device="cuda") >= masked if isinstance(masked, float) else \
                torch.tensor([masked(i, m) for i in range(m)], dtype=torch.bool, device="cuda")
            mask[r0:r0 + m] = on.to(torch.uint8) * 3  # any non-zero byte is valid
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for m, r0 in zip(lens, row0):
        own[r0:r0 + m] = True
    if mask is not None:
        own &= mask != 0
    ref, mag = lm_ops.packed_attention(f64(q)[:cu[-1]], f64(k), f64(v), hq, hkv, cu, row0, lens,
                                       None if mask is None else mask.cpu().numpy(), causal, scale)
    if nan_outside:
        k[~own] = float("nan")
        v[~own] = float("nan")
        q[cu[-1]:] = float("nan")
    out = torch.full_like(q, 9.0)
    ex.prompt_attention(q, k, v, cu, kv_row0=None if packed else row0, kv_len=None if packed else lens, key_mask=mask,
                        causal=causal, scale=scale, out=out)
    ex.synchronize()
    check_attention(f64(out)[:cu[-1]], ref, mag, (new, cached))
    assert (out[cu[-1]:] == 9.0).all()  # rows behind the last sequence
    return q, k, v, out


LAYOUTS = [(8, 1, 256), (4, 1, 64), (12, 4, 64), (5, 5, 128), (32, 8, 128), (16, 2, 128), (14, 2, 128), (3, 1, 256)]


@pytest.mark.parametrize("hq,hkv,dh", LAYOUTS)
@pytest.mark.parametrize("new,cached", [
    ([1], [0]), ([2, 1, 3], [0, 0, 0]), ([63, 64, 65], [0, 0, 0]), ([127, 128, 129], [0, 0, 0]),
    ([300], [0]), ([5, 0, 17], [250, 0, 128]), ([1, 33], [511, 63]), ([0, 130], [40, 1])])
def test_prompt_attention(experts, hq, hkv, dh, new, cached):
    run_prompt(experts(hq, hkv, dh), hq, hkv, dh, new, cached, gap=3, seed=sum(new))


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (12, 4, 64), (32, 8, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_attention_packed_keys(experts, hq, hkv, dh, causal):
    run_prompt(experts(hq, hkv, dh), hq, hkv, dh, [70, 1, 200, 31], [0] * 4, causal=causal, packed=True)


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (4, 1, 64), (16, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("masked", [0.3, 0.95, lambda i, m: False, lambda i, m: i >= m - 1, lambda i, m: i >= 200,
                                    lambda i, m: i < 64, lambda i, m: not 64 <= i < 192],
                         ids=["third", "most", "all", "last-only", "first-200", "beyond-64", "slot"])
def test_prompt_attention_masks(experts, hq, hkv, dh, causal, masked):
    """Masked rows hold NaN; a mask may leave rows without any key (zeros)."""
    run_prompt(experts(hq, hkv, dh), hq, hkv, dh, [40, 260, 1], [0, 70, 200], masked=masked, causal=causal, gap=1)


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (12, 4, 64), (32, 8, 128)])
def test_prompt_attention_long(experts, hq, hkv, dh):
    run_prompt(experts(hq, hkv, dh), hq, hkv, dh, [1500, 700], [0, 1301], gap=5, seed=11)
    run_prompt(experts(hq, hkv, dh), hq, hkv, dh, [9, 3], [4000, 3000], gap=5, seed=12)


def test_prompt_attention_masked_key_ranges_of_any_length(experts):
    """Masked caches whose share of a CTA is beyond the room of its tile list, and well within it."""
    for dh, n in ((256, 300000), (64, 70000)):
        run_prompt(experts(8, 1, 256) if dh == 256 else experts(4, 1, 64), 8 if dh == 256 else 4, 1, dh, [5], [n - 5],
                   masked=lambda i, m: (i // 100) % 3 != 1 and i % 7 != 0, gap=1, seed=n)


def test_prompt_attention_masked_keys_beyond_the_list(experts):
    """One CTA's key range longer than its tile list: 64 one-token sequences that share 60000 masked
    rows fill the GPU, so their keys are not split."""
    import torch
    hq, hkv, dh, rows, batch = 12, 4, 64, 60000, 64
    ex, g = experts(hq, hkv, dh), generator(60)
    q, k, v = normal(g, batch, hq * dh), normal(g, rows, hkv * dh), normal(g, rows, hkv * dh)
    mask = (torch.rand(rows, generator=g, device="cuda") < 0.5).to(torch.uint8)
    mask[1000:3000] = 0
    lens = [rows - 37 * (b % 5) for b in range(batch)]
    cu, row0 = list(range(batch + 1)), [0] * batch
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, cu, row0, lens, mask.cpu().numpy())
    k[mask == 0] = float("nan")
    v[mask == 0] = float("nan")
    out = ex.prompt_attention(q, k, v, cu, row0, lens, key_mask=mask)
    ex.synchronize()
    check_attention(f64(out), ref, mag)


@pytest.mark.parametrize("hq,hkv,dh", [(4, 1, 64), (12, 4, 64), (6, 6, 64), (8, 1, 256), (32, 8, 128)])
@pytest.mark.parametrize("keys", [95, 96, 97, 191, 192, 193, 288, 385])
def test_prompt_attention_key_tile_ends(experts, hq, hkv, dh, keys):
    """Lengths around whole key tiles (96 keys at head_dim 64, 128 above), causal diagonals and masks
    that end at them."""
    ex = experts(hq, hkv, dh)
    run_prompt(ex, hq, hkv, dh, [keys, 3], [0, keys - 3], gap=2, seed=keys)
    run_prompt(ex, hq, hkv, dh, [2, 50], [keys - 2, keys], gap=1, seed=keys + 1, causal=False)
    for cut in (lambda i, m: i < 96, lambda i, m: i >= 96, lambda i, m: not 96 <= i < 192, lambda i, m: i == m - 1):
        run_prompt(ex, hq, hkv, dh, [4, 30], [keys - 4, keys - 30], masked=cut, gap=1, seed=keys + 2)


@pytest.mark.parametrize("hq,hkv,dh,new,cached", [
    (8, 1, 256, [700], [0]), (32, 8, 128, [700, 300], [0, 0]), (32, 8, 128, [64], [1000]), (12, 4, 64, [700], [0]),
    (32, 8, 128, [64] * 40, [0] * 40), (4, 1, 64, [10], [4000])])
def test_prompt_attention_rows_without_keys_are_zero_every_time(experts, hq, hkv, dh, new, cached):
    """Query tiles all of whose keys are masked write their zeros where the queries land: many calls,
    the copies cold and warm, all the same bits."""
    import torch
    ex, g = experts(hq, hkv, dh), generator(61)
    cu, lens = [0] + [int(x) for x in np.cumsum(new)], [a + b for a, b in zip(new, cached)]
    row0 = [0] + [int(x) for x in np.cumsum(lens)[:-1]]
    rows = sum(lens)
    q, k, v = normal(g, cu[-1], hq * dh), normal(g, rows, hkv * dh), normal(g, rows, hkv * dh)
    mask = torch.zeros(rows, dtype=torch.uint8, device="cuda")
    for r0, m in zip(row0, lens):
        mask[r0 + m // 2:r0 + m] = 1  # a sequence's first half is masked
    if len(new) > 2 or cached[0] > 3000:
        mask[:] = 0
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, cu, row0, lens, mask.cpu().numpy())
    want = ex.prompt_attention(q, k, v, cu, row0, lens, key_mask=mask)
    ex.synchronize()
    check_attention(f64(want), ref, mag)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(60):
        if i % 3 == 0:
            flush.fill_(i)
        outs.append(ex.prompt_attention(q, k, v, cu, row0, lens, key_mask=mask, out=torch.full_like(q, 3.0)))
    ex.synchronize()
    assert all(torch.equal(want, o) for o in outs)


@pytest.mark.parametrize("std,scale", [(30.0, 0.0), (1.0, 3.0), (1e-3, 0.0), (1.0, 1e-4)])
def test_prompt_attention_score_ranges(experts, std, scale):
    """Peaked and flat softmaxes (scores of several hundred, scores near zero)."""
    run_prompt(experts(16, 2, 128), 16, 2, 128, [200, 65], [0, 300], std=std, scale=scale, gap=2)


def test_prompt_attention_rising_scores(experts):
    """Keys whose scores rise along the row: every tile raises the running maximum."""
    import torch
    for hq, hkv, dh in ((4, 1, 64), (8, 1, 256), (16, 2, 128)):
        ex, n = experts(hq, hkv, dh), 700
        g = generator(5)
        q = torch.ones((n, hq * dh), dtype=torch.bfloat16, device="cuda")
        ramp = torch.linspace(-20, 20, n, device="cuda")[:, None].expand(n, hkv * dh)
        k, v = (ramp / dh ** 0.5).to(torch.bfloat16).contiguous(), normal(g, n, hkv * dh)
        for a, b in ((k, "up"), (k.flip(0).contiguous(), "down")):
            out = ex.prompt_attention(q, a, v, [0, n], causal=False)
            ex.synchronize()
            ref, mag = lm_ops.packed_attention(f64(q), f64(a), f64(v), hq, hkv, [0, n], [0], [n], causal=False)
            check_attention(f64(out), ref, mag, b)


def test_prompt_attention_strides(experts):
    """q, k and v read from the columns of wider rows (a merged projection), out into wider rows."""
    import torch
    hq, hkv, dh, n = 12, 4, 64, 150
    ex, g = experts(hq, hkv, dh), generator(6)
    qkv = normal(g, n, (hq + 2 * hkv) * dh)
    q, k, v = qkv[:, :hq * dh], qkv[:, hq * dh:(hq + hkv) * dh], qkv[:, (hq + hkv) * dh:]
    wide = torch.full((n, hq * dh + 16), 9.0, dtype=torch.bfloat16, device="cuda")
    ex.prompt_attention(q, k, v, [0, 90, n], out=wide[:, :hq * dh])
    ex.synchronize()
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, [0, 90, n], [0, 90], [90, 60])
    check_attention(f64(wide)[:, :hq * dh], ref, mag)
    assert (wide[:, hq * dh:] == 9.0).all()


def test_prompt_attention_most_sequences(experts):
    """The largest batch, lengths from zero up, some sharing one cached beginning."""
    import torch
    hq, hkv, dh = 4, 1, 64
    ex, g = experts(hq, hkv, dh), generator(7)
    new = [i % 5 for i in range(64)]
    cu = [0] + [int(x) for x in np.cumsum(new)]
    lens = [100 if i % 2 else 100 - i for i in range(64)]
    row0 = [0 if i % 2 else i for i in range(64)]
    q, k, v = normal(g, cu[-1], hq * dh), normal(g, 100, hkv * dh), normal(g, 100, hkv * dh)
    out = ex.prompt_attention(q, k, v, cu, kv_row0=row0, kv_len=lens)
    ex.synchronize()
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, cu, row0, lens)
    check_attention(f64(out), ref, mag)


@pytest.mark.parametrize("hq,hkv,dh", [(130, 1, 64), (262, 2, 64), (200, 1, 64), (66, 2, 128), (130, 1, 128), (33, 1, 256)])
def test_prompt_attention_wide_groups(hq, hkv, dh):
    """Groups of more heads than a query tile has rows, and just above half of them."""
    ex = _expert(hq, hkv, dh)
    try:
        run_prompt(ex, hq, hkv, dh, [1, 5, 40], [0, 130, 3], gap=2)
        run_token(ex, hq, hkv, dh, [1, 77, 300])
    finally:
        ex.close()


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (12, 4, 64), (32, 8, 128)])
def test_attention_in_place_of_the_queries(experts, hq, hkv, dh):
    import torch
    ex, g = experts(hq, hkv, dh), generator(50)
    cu, row0, lens = [0, 90, 107], [0, 1300], [1300, 400]
    q, k, v = normal(g, 107, hq * dh), normal(g, 1700, hkv * dh), normal(g, 1700, hkv * dh)
    want = ex.prompt_attention(q, k, v, cu, row0, lens)
    got = q.clone()
    ex.prompt_attention(got, k, v, cu, row0, lens, out=got)
    r, n = torch.tensor(row0, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    token = ex.token_attention(q[:2], k, v, r, n, 1300)
    over = q[:2].clone()
    ex.token_attention(over, k, v, r, n, 1300, out=over)
    ex.synchronize()
    assert torch.equal(want, got) and torch.equal(token, over)


@pytest.mark.parametrize("new,cached", [
    ([1200, 63, 65, 1, 900, 257], [0, 0, 5, 300, 0, 1]), ([100, 64, 128, 33, 65, 129, 1, 32] * 2, [0] * 16),
    ([64, 60, 64], [3936, 4000, 3900]), ([64, 50, 33, 64, 64, 64, 64, 61], [0] * 8), ([128] * 4, [0] * 4)])
def test_prompt_attention_two_tiles_a_cta(experts, new, cached):
    """Calls at head_dim 128 that fill the SMs with pairs of query tiles, and one that does not."""
    ex = experts(32, 8, 128)
    run_prompt(ex, 32, 8, 128, new, cached, gap=1, seed=90)
    run_prompt(ex, 32, 8, 128, new, cached, gap=1, seed=91, causal=False, masked=0.5)
    run_prompt(ex, 32, 8, 128, new, cached, gap=1, seed=92, masked=lambda i, m: i // 150 % 2 == 1)


def test_prompt_attention_two_tiles_over_split_keys(experts):
    """Pairs of query tiles whose long key ranges are split over eight CTAs."""
    ex = experts(5, 5, 128)
    run_prompt(ex, 5, 5, 128, [520], [59480], gap=1, seed=95)
    run_prompt(ex, 5, 5, 128, [520], [59480], gap=1, seed=96, masked=0.5)


@pytest.mark.parametrize("hq,hkv,dh,new,cached", [
    (4, 1, 64, [2048], [0]), (4, 1, 64, [100] * 8 + [2100], [0] * 9), (2, 1, 64, [900, 2500, 1], [0, 300, 2000]),
    (6, 6, 64, [64] * 4, [1500, 1700, 900, 1601])])
def test_prompt_attention_two_split_ctas_a_sm(experts, hq, hkv, dh, new, cached):
    """Split key ranges of more CTAs than SMs, whole and masked, causal and not."""
    ex = experts(hq, hkv, dh)
    run_prompt(ex, hq, hkv, dh, new, cached, gap=1, seed=80)
    run_prompt(ex, hq, hkv, dh, new, cached, gap=1, seed=81, causal=False, masked=0.5)
    run_prompt(ex, hq, hkv, dh, new, cached, gap=1, seed=82, masked=lambda i, m: i // 200 % 2 == 1)


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (3, 1, 256), (16, 2, 128), (5, 5, 128)])
def test_prompt_attention_idle_sms(experts, hq, hkv, dh):
    """Small calls, whose value dims two CTAs share, against the same calls over their queries, which
    they do not share: whole and cut tiles, split keys, masks, wide output rows."""
    import torch
    ex, g = experts(hq, hkv, dh), generator(70)
    for new, cached in (([16], [0]), ([5], [0]), ([1], [4000]), ([16], [1008]), ([130], [7]), ([33, 1], [90, 700])):
        q, k, v, out = run_prompt(ex, hq, hkv, dh, new, cached, gap=2, seed=sum(new))
        run_prompt(ex, hq, hkv, dh, new, cached, masked=0.4, gap=2, seed=1 + sum(new))
        n = sum(new)
        cu, lens = [0] + [int(x) for x in np.cumsum(new)], [a + b for a, b in zip(new, cached)]
        row0 = [2 + sum(lens[:i]) + 2 * i for i in range(len(new))]
        wide, view = strided(out[:n], 8)
        wide.fill_(5.0)
        ex.prompt_attention(q[:n], k, v, cu, row0, lens, out=view)
        over = q[:n].clone()
        ex.prompt_attention(over, k, v, cu, row0, lens, out=over)
        ex.synchronize()
        assert torch.equal(over, out[:n]) and torch.equal(view, out[:n]) and (wide[:, hq * dh:] == 5.0).all()


# ---------------------------------------------------------------- token attention

def run_token(ex, hq, hkv, dh, lens, max_len=None, masked=None, seed=0, room=7, scale=0.0):
    import torch
    g = generator(seed)
    cap = max(lens) + room
    rows = cap * len(lens)
    perm = np.random.default_rng(seed).permutation(len(lens))
    row0 = [int(p) * cap + 2 for p in perm]
    q = normal(g, len(lens), hq * dh, std=1.5)
    k, v = normal(g, rows, hkv * dh), normal(g, rows, hkv * dh)
    mask = None
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for m, r0 in zip(lens, row0):
        own[r0:r0 + m] = True
    if masked is not None:
        mask = (torch.rand(rows, generator=g, device="cuda") >= masked).to(torch.uint8)
        own &= mask != 0
    cu = list(range(len(lens) + 1))
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, cu, row0, lens,
                                       None if mask is None else mask.cpu().numpy(), False, scale)
    k[~own] = float("nan")
    v[~own] = float("nan")
    r, n = torch.tensor(row0, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    ex.token_attention(q, k, v, r, n, max_len or max(lens), key_mask=mask, scale=scale, out=out)
    ex.synchronize()
    check_attention(f64(out), ref, mag, lens)
    return q, k, v, r, n, mask, out


@pytest.mark.parametrize("hq,hkv,dh", LAYOUTS + [(40, 2, 64), (17, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [15, 16, 17, 31], [64, 65, 127, 128, 129], [1000, 1, 333], [3000]])
def test_token_attention(experts, hq, hkv, dh, lens):
    run_token(experts(hq, hkv, dh), hq, hkv, dh, lens, seed=len(lens))


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (12, 4, 64), (32, 8, 128)])
@pytest.mark.parametrize("masked", [0.3, 0.97, 1.0])
def test_token_attention_masks(experts, hq, hkv, dh, masked):
    run_token(experts(hq, hkv, dh), hq, hkv, dh, [1, 40, 700, 129], masked=masked, max_len=5000)


def test_token_attention_many_requests(experts):
    run_token(experts(4, 1, 64), 4, 1, 64, [(37 * i) % 90 for i in range(700)], seed=3)


def test_token_attention_without_cache_rows(experts):
    import torch
    ex = experts(4, 1, 64)
    q = torch.ones((3, 256), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    r, n = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for max_len in (0, 500):
        out = torch.full_like(q, 9.0)
        ex.token_attention(q, k, k, r, n, max_len, out=out)
        ex.synchronize()
        assert (out == 0).all()


def test_token_attention_scales(experts):
    run_token(experts(16, 2, 128), 16, 2, 128, [500, 80], scale=2.0)
    run_token(experts(16, 2, 128), 16, 2, 128, [500, 80], scale=1e-3)


def test_token_attention_rows_beyond_32_bits():
    """Cache rows whose element offsets pass 2^31 and 2^32."""
    import torch
    hq, hkv, dh = 8, 1, 256
    ex, g = _expert(hq, hkv, dh), generator(8)
    try:
        stride, rows = 1 << 16, 70000  # 4.6e9 elements of rows, one buffer shared by k and v
        buf = torch.zeros(stride * rows, dtype=torch.bfloat16, device="cuda")
        k = buf.as_strided((rows, dh), (stride, 1))
        v = buf.as_strided((rows, dh), (stride, 1), dh)
        lens, row0 = [300, 100], [rows - 300, 40000]
        for m, r in zip(lens, row0):
            k[r:r + m], v[r:r + m] = normal(g, m, dh), normal(g, m, dh)
        q = normal(g, 2, hq * dh)
        ks, vs = [np.concatenate([f64(t[r:r + m]) for m, r in zip(lens, row0)]) for t in (k, v)]
        ref, mag = lm_ops.packed_attention(f64(q), ks, vs, hq, hkv, [0, 1, 2], [0, 300], lens, None, False)
        r, n = torch.tensor(row0, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = ex.token_attention(q, k, v, r, n, 300)
        ex.synchronize()
        check_attention(f64(out), ref, mag)
        got = ex.prompt_attention(q, k, v, [0, 1, 2], kv_row0=row0, kv_len=lens)
        ex.synchronize()
        check_attention(f64(got), ref, mag)
    finally:
        ex.close()


def test_token_attention_bad_rows_are_cut_and_reported():
    import torch
    hq, hkv, dh = 4, 1, 64
    g = generator(9)
    q, k, v = normal(g, 5, hq * dh), normal(g, 50, dh), normal(g, 50, dh)
    bad_row0, bad_len = [40, -3, 10, 60, 1 << 40], [20, 10, 31, 5, 1]
    cut_row0, cut_len = [40, 0, 10, 0, 0], [10, 7, 30, 0, 0]  # max_len 30
    ref, mag = lm_ops.packed_attention(f64(q), f64(k), f64(v), hq, hkv, list(range(6)), cut_row0, cut_len, None, False)
    ex = _expert(hq, hkv, dh)
    try:
        out = ex.token_attention(q, k, v, torch.tensor(bad_row0, device="cuda"),
                                 torch.tensor(bad_len, dtype=torch.int32, device="cuda"), 30)
        with pytest.raises(ae.AEError) as e:
            ex.synchronize()
        assert e.value.status == -5
        check_attention(f64(out), ref, mag)
    finally:
        ex.close()


# ---------------------------------------------------------------- as they are used

def _layer(ex, qkv, pos, k, v, rows, cu, row0, lens, out):
    import torch
    q = torch.empty((qkv.shape[0], out.shape[1]), dtype=torch.bfloat16, device="cuda")
    ex.qk_norm_rope(qkv, pos, q, k, v, kv_rows=rows)
    ex.prompt_attention(q, k, v, cu, kv_row0=row0, kv_len=lens, out=out)
    return q


@pytest.mark.parametrize("hq,hkv,dh", [(8, 1, 256), (32, 8, 128)])
def test_prompt_then_tokens_equals_one_prompt(experts, hq, hkv, dh):
    """Prefill, a continued chunk and single tokens over one cache give each row the same attention
    as one prompt of the whole sequence."""
    import torch
    ex, g = experts(hq, hkv, dh), generator(10)
    total, room = [140, 77], 160
    qkv = [normal(g, t, (hq + 2 * hkv) * dh) for t in total]
    k = torch.full((2 * room, hkv * dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    done, outs = [0, 0], [[], []]
    row0 = torch.tensor([0, room], device="cuda")
    for step in ([100, 40], [38, 30], None, None):
        n = step or [1, 1]
        if step is None and done[1] + 1 > total[1]:
            break
        x = torch.cat([qkv[b][done[b]:done[b] + n[b]] for b in (0, 1)])
        pos = torch.cat([torch.arange(done[b], done[b] + n[b]) for b in (0, 1)]).to(torch.int32).cuda()
        rows = torch.cat([torch.arange(done[b], done[b] + n[b]) + b * room for b in (0, 1)]).cuda()
        lens = [done[b] + n[b] for b in (0, 1)]
        out = torch.empty((x.shape[0], hq * dh), dtype=torch.bfloat16, device="cuda")
        if step is not None:
            _layer(ex, x, pos, k, v, rows, [0, n[0], n[0] + n[1]], [0, room], lens, out)
        else:
            q = torch.empty_like(out)
            ex.qk_norm_rope(x, pos, q, k, v, kv_rows=rows)
            ex.token_attention(q, k, v, row0, torch.tensor(lens, dtype=torch.int32, device="cuda"), room, out=out)
        outs[0].append(out[:n[0]])
        outs[1].append(out[n[0]:])
        done = lens
    ex.synchronize()
    f = lm_ops.ladder(10000.0, dh)
    for b in (0, 1):
        t = done[b]
        q = torch.empty((t, hq * dh), dtype=torch.bfloat16, device="cuda")
        kk, vv = torch.empty((t, hkv * dh), dtype=torch.bfloat16, device="cuda"), None
        vv = torch.empty_like(kk)
        ex.qk_norm_rope(qkv[b][:t].contiguous(), torch.arange(t, dtype=torch.int32, device="cuda"), q, kk, vv)
        ex.synchronize()
        # the rotated rows do not depend on the call they were written by
        assert torch.equal(kk, k[b * room:b * room + t]) and torch.equal(vv, v[b * room:b * room + t])
        x = f64(qkv[b][:t]).reshape(t, hq + 2 * hkv, dh)
        check_rope(f64(q).reshape(t, hq, dh),
                   lm_ops.norm_rope(x[:, :hq], None, 0, 0, [np.arange(t)], [0] * (dh // 2), f), "q")
        ref, mag = lm_ops.packed_attention(f64(q), f64(kk), f64(vv), hq, hkv, [0, t], [0], [t])
        check_attention(f64(torch.cat(outs[b])), ref, mag, b)


def test_decode_graph_follows_growing_lengths():
    """One captured decoding step (rotation + cache write + attention) replayed while the lengths on
    the device grow; another graph of the same context replays beside it on a second stream."""
    import torch
    hq, hkv, dh, room = 32, 8, 128, 300
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ex = _expert(hq, hkv, dh)
    try:
        states = []
        for i, st in enumerate((s1, s2)):
            g = generator(20 + i)
            s = dict(qkv=normal(g, 2, (hq + 2 * hkv) * dh), k=normal(g, 2 * room, hkv * dh),
                     v=normal(g, 2 * room, hkv * dh), row0=torch.tensor([0, room], device="cuda"),
                     n=torch.tensor([200 + i, 31], dtype=torch.int32, device="cuda"))
            s["pos"] = s["n"] - 1
            s["rows"] = s["row0"] + s["pos"]
            s["q"] = torch.empty((2, hq * dh), dtype=torch.bfloat16, device="cuda")
            s["out"] = torch.empty_like(s["q"])
            states.append(s)
        torch.cuda.synchronize()
        graphs = []
        for s, st in zip(states, (s1, s2)):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                ae.ae_set_stream(ex.ctx, ctypes.c_void_p(st.cuda_stream))
                ex.qk_norm_rope(s["qkv"], s["pos"], s["q"], s["k"], s["v"], kv_rows=s["rows"])
                ex.token_attention(s["q"], s["k"], s["v"], s["row0"], s["n"], room, out=s["out"])
            graphs.append(graph)
        for step in range(3):
            for s, st, graph in zip(states, (s1, s2), graphs):
                with torch.cuda.stream(st):
                    graph.replay()
            torch.cuda.synchronize()
            for s in states:
                lens, row0 = s["n"].tolist(), s["row0"].tolist()
                ref, mag = lm_ops.packed_attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), hq, hkv, [0, 1, 2], row0,
                                                   lens, None, False)
                check_attention(f64(s["out"]), ref, mag, step)
                x = f64(s["qkv"]).reshape(2, hq + 2 * hkv, dh)
                ref = lm_ops.norm_rope(x[:, hq:hq + hkv], None, 0, 0, [np.array(lens) - 1], [0] * (dh // 2),
                                       lm_ops.ladder(10000.0, dh))
                check_rope(f64(s["k"][s["rows"]]).reshape(2, hkv, dh), ref, "k")
                s["n"] += 1
                s["pos"] += 1
                s["rows"] += 1
            torch.cuda.synchronize()
    finally:
        ex.close()


def test_prompt_graph_and_repeat_are_bitwise_equal(experts):
    """Eager calls, repeated calls and graph replays (two streams at once) give the same bits."""
    import torch
    hq, hkv, dh = 16, 2, 128
    ex = _expert(hq, hkv, dh)
    try:
        g = generator(30)
        cu, row0, lens = [0, 20, 150], [0, 2100], [2000, 333]
        q, k, v = normal(g, 150, hq * dh), normal(g, 2500, hkv * dh), normal(g, 2500, hkv * dh)
        want = ex.prompt_attention(q, k, v, cu, row0, lens)
        again = ex.prompt_attention(q, k, v, cu, row0, lens)
        torch.cuda.synchronize()
        assert torch.equal(want, again)
        outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
        for st in streams:
            out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                ae.ae_set_stream(ex.ctx, ctypes.c_void_p(st.cuda_stream))
                ex.prompt_attention(q, k, v, cu, row0, lens, out=out)
            outs.append(out)
            graphs.append(graph)
        for _ in range(3):
            for st, graph in zip(streams, graphs):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want, o) for o in outs)
        ex.synchronize()
    finally:
        ex.close()


def test_binding_refuses_wrong_tensors(experts):
    import torch
    hq, hkv, dh = 4, 1, 64
    ex, g = experts(hq, hkv, dh), generator(40)
    q, k, v = normal(g, 4, hq * dh), normal(g, 4, dh), normal(g, 4, dh)
    for bad in (dict(q=q.float()), dict(q=q[:, ::2]), dict(k=k[:3]), dict(v=v.cpu()), dict(q=q[:2]),
                dict(key_mask=torch.ones(3, dtype=torch.uint8, device="cuda")), dict(kv_row0=[0, 1], kv_len=[4, 4]),
                dict(out=torch.empty((4, hq * dh), device="cuda")), dict(q=q.t().contiguous().t())):
        args = dict(q=q, k=k, v=v, cu_q=[0, 4])
        args.update(bad)
        with pytest.raises(ValueError):
            ex.prompt_attention(**args)


def test_binding_refuses_tensors_of_another_device(experts):
    """A tensor's device index is compared with the context's (here a context that says it lives
    elsewhere: one GPU is enough)."""
    import torch
    hq, hkv, dh = 4, 1, 64
    ex, g = experts(hq, hkv, dh), generator(41)
    q, k, v = normal(g, 2, hq * dh), normal(g, 2, dh), normal(g, 2, dh)
    ex._device += 1
    try:
        with pytest.raises(ValueError, match="cuda:"):
            ex.prompt_attention(q, k, v, [0, 2])
        with pytest.raises(ValueError, match="cuda:"):
            ex.token_attention(q, k, v, torch.zeros(2, dtype=torch.int64, device="cuda"),
                               torch.ones(2, dtype=torch.int32, device="cuda"), 2)
        with pytest.raises(ValueError, match="cuda:"):
            ex.qk_norm_rope(normal(g, 2, (hq + 2 * hkv) * dh), torch.zeros(2, dtype=torch.int32, device="cuda"), q, k, v)
    finally:
        ex._device -= 1
