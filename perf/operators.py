"""Timed cases of the language-model attention operators.

Three operators of a decoder layer's attention, as a vision-language prefill and
its language requests use them:

* ``rope``    per-head RMS norm of queries and keys, rotary positions on one or
              several axes, keys and values written into the cache
              (``ActionExpert.qk_norm_rope``)
* ``prompt``  attention of packed prompts of different lengths, causal, grouped
              heads, optionally continuing cached rows (``ActionExpert.prompt_attention``)
* ``token``   attention of one new token per request over its cached rows
              (``ActionExpert.token_attention``)

``run`` computes them by elementary torch operations in 32 bits, or, with
``own`` set, by the framework's calls.  Head layouts are written "query heads /
KV heads / head size".
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6
SLOT = 256  # rows of one camera's image tokens; an empty second slot is masked


# ---------------------------------------------------------------- cases

def _text(lens):
    return ",".join(str(int(n)) for n in lens)


def _lens(text):
    return [int(n) for n in text.split(",")]


def _rope(name, heads, tokens, axes, norm, scatter):
    return {"name": name, "op": "rope", "heads": heads, "tokens": tokens, "axes": axes, "norm": norm,
            "scatter": scatter}


def _prompt(name, heads, new, cached=None, masked=False):
    return {"name": name, "op": "prompt", "heads": heads, "new": _text(new),
            "cached": _text(cached if cached is not None else [0] * len(new)), "masked": masked}


def _token(name, heads, lens, masked=False):
    return {"name": name, "op": "token", "heads": heads, "lens": _text(lens), "masked": masked}


def listed():
    return [
        # one decoding step of twelve language requests: the smallest call
        _rope("rope-12-tokens", "8/1/256", 12, 1, True, True),
        # image patches of a vision tower: two axes, no norm, an odd count, heads of 64
        _rope("rope-5003-patches", "12/4/64", 5003, 2, False, False),
        # a long video and text prompt: time, height, width; rows scattered into the cache
        _rope("rope-32k-video", "32/8/128", 32768, 3, True, True),
        # an instruction alone
        _prompt("prompt-50", "8/1/256", [50]),
        # two cameras and an instruction, the batch-1 prefix of the benchmark
        _prompt("prompt-712", "8/1/256", [712]),
        # sixteen requests of 600 to 2048 rows, the range of the batch-16 benchmark, one camera slot empty
        _prompt("prompt-16-ragged", "8/1/256",
                [600, 1811, 712, 2048, 968, 1333, 1601, 777, 2000, 651, 1224, 1480, 905, 1999, 1111, 1719],
                masked=True),
        # a packed batch of text prompts from one token up, heads of 64 in groups of three
        _prompt("prompt-mixed-64", "12/4/64", [1, 17, 300, 63, 1025, 2, 129, 511, 4097, 64]),
        # the next turn of four conversations: few new rows over long cached ones
        _prompt("prompt-chunk", "32/8/128", [48, 7, 64, 33], cached=[8000, 8191, 6001, 7777]),
        # one long document
        _prompt("prompt-32k", "32/8/128", [32768]),
        # one language request decoding over the two-camera prefix
        _token("token-1", "8/1/256", [712]),
        # twelve requests decoding over prefixes with an empty camera slot
        _token("token-12-frames", "8/1/256",
               [713, 1969, 730, 2048, 968, 1, 1601, 777, 2000, 651, 257, 1480], masked=True),
        # a full serving batch over long caches
        _token("token-64-8k", "32/8/128", [8192 - 61 * (i % 7) for i in range(64)]),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ("8/1/256", "4/1/64", "12/4/64", "16/2/128", "32/8/128", "5/5/128", "16/16/64")
PROMPT_FLOPS = 4.0 * 32 * 128 * 32768 * 32769 / 2
TOKEN_BYTES = 64 * 8000 * 8 * 128 * 4


def draw(rng):
    op = rng.choice(("rope", "prompt", "prompt", "token", "token"))
    heads = rng.choice(HEADS)
    hq, _, dh = _heads(heads)
    if op == "rope":
        hkv = _heads(heads)[1]
        most = 32768 * 48 * 128 // ((hq + 2 * hkv) * dh)
        return {"op": op, "heads": heads, "tokens": _log(rng, 1, min(32768, most)), "axes": rng.randint(1, 3),
                "norm": rng.random() < 0.75, "scatter": rng.random() < 0.5}
    if op == "prompt":
        n = _log(rng, 1, 24)
        top = _log(rng, 8, 16384)
        new = [_log(rng, 1, top) for _ in range(n)]
        cached = [_log(rng, 1, 8192) if rng.random() < 0.3 else 0 for _ in range(n)]
        case = {"op": op, "heads": heads, "new": _text(new), "cached": _text(cached), "masked": rng.random() < 0.3}
        while work(case)["flops"] > PROMPT_FLOPS / 4 and len(new) > 1:
            new, cached = new[:-1], cached[:-1]
            case["new"], case["cached"] = _text(new), _text(cached)
        return case
    n = _log(rng, 1, 96)
    top = _log(rng, 16, 16384)
    lens = [_log(rng, 1, top) for _ in range(n)]
    case = {"op": op, "heads": heads, "lens": _text(lens), "masked": rng.random() < 0.3}
    while work(case)["bytes"] > TOKEN_BYTES and len(lens) > 1:
        lens = lens[:-1]
        case["lens"] = _text(lens)
    return case


def _heads(text):
    return tuple(int(n) for n in text.split("/"))


def _unmasked(n, masked):
    """Keys of the first n rows that an empty second camera slot leaves."""
    return n - max(0, min(n, 2 * SLOT) - SLOT) if masked else n


def work(case):
    hq, hkv, dh = _heads(case["heads"])
    if case["op"] == "rope":
        t, elems = case["tokens"], case["tokens"] * (hq + 2 * hkv) * dh
        side = t * (4 * case["axes"] + (8 if case["scatter"] else 0)) + (4 * dh if case["norm"] else 0)
        per = 3 + (4 if case["norm"] else 0)  # rotation; square, sum, two products
        return {"bytes": 4 * elems + side, "flops": float(per * t * (hq + hkv) * dh)}
    if case["op"] == "prompt":
        pairs = rows = kept = 0
        for n, c in zip(_lens(case["new"]), _lens(case["cached"])):
            j = np.arange(c + 1, c + n + 1, dtype=np.int64)  # rows a query sees
            if case["masked"]:
                j = j - np.clip(j - SLOT, 0, SLOT)
            pairs += int(j.sum())
            rows += n
            kept += _unmasked(c + n, case["masked"])
        side = sum(n + c for n, c in zip(_lens(case["new"]), _lens(case["cached"]))) if case["masked"] else 0
        return {"bytes": 4 * rows * hq * dh + 4 * kept * hkv * dh + side, "flops": 4.0 * dh * hq * pairs}
    lens = _lens(case["lens"])
    kept = sum(_unmasked(n, case["masked"]) for n in lens)
    side = 12 * len(lens) + (sum(lens) if case["masked"] else 0)
    return {"bytes": 4 * len(lens) * hq * dh + 4 * kept * hkv * dh + side, "flops": 4.0 * dh * hq * kept}


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = x.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda") * std
    return x


def _pair_axis(axes, half):
    """Axis of every rotation pair: axes in turn, as interleaved time/height/width positions use them."""
    return bytes(i % axes for i in range(half))


def _slot_mask(lens, rows, row0):
    m = torch.ones(rows, dtype=torch.uint8, device="cuda")
    for n, r in zip(lens, row0):
        m[r + min(n, SLOT):r + min(n, 2 * SLOT)] = 0
    return m


def _inputs(case, seed):
    hq, hkv, dh = _heads(case["heads"])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "hq": hq, "hkv": hkv, "dh": dh}
    if case["op"] == "rope":
        t, ax = case["tokens"], case["axes"]
        s["qkv"] = _normal(gen, (t, (hq + 2 * hkv) * dh), 1.5)
        if case["norm"]:
            s["q_norm"] = (1.0 + 0.2 * torch.randn(dh, generator=gen, device="cuda")).to(torch.bfloat16)
            s["k_norm"] = (1.0 + 0.2 * torch.randn(dh, generator=gen, device="cuda")).to(torch.bfloat16)
        else:
            s["q_norm"] = s["k_norm"] = None
        i = torch.arange(t, device="cuda")
        pos = [i] if ax == 1 else [i // 64, i % 64] if ax == 2 else [i // 1024, (i // 32) % 32, i % 32]
        if case["scatter"]:
            start = torch.randint(0, 1 << 16, (1,), generator=gen, device="cuda")
            pos[0] = pos[0] + start
            rows = t + t // 2 + 1
            s["kv_rows"] = torch.randperm(rows, generator=gen, device="cuda")[:t].sort().values
        else:
            rows, s["kv_rows"] = t, None
        s["positions"] = torch.stack(pos).to(torch.int32)
        s["pair_axis"] = _pair_axis(ax, dh // 2)
        s["q_out"] = torch.zeros((t, hq * dh), dtype=torch.bfloat16, device="cuda")
        s["k_cache"] = torch.zeros((rows, hkv * dh), dtype=torch.bfloat16, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        return s
    if case["op"] == "prompt":
        new, cached = _lens(case["new"]), _lens(case["cached"])
        s["cu_q"] = [0] + [int(n) for n in np.cumsum(new)]
        s["kv_len"] = [n + c for n, c in zip(new, cached)]
        s["kv_row0"] = [0] + [int(n) for n in np.cumsum(s["kv_len"])[:-1]]
        rows = sum(s["kv_len"])
        s["q"] = _normal(gen, (s["cu_q"][-1], hq * dh), 1.5)
        s["mask"] = _slot_mask(s["kv_len"], rows, s["kv_row0"]) if case["masked"] else None
    else:
        lens = _lens(case["lens"])
        room = max(lens) + 32  # rows reserved for each request
        rows = room * len(lens)
        s["max_len"] = max(lens)
        row0 = [room * b for b in range(len(lens))]
        s["row0"] = torch.tensor(row0, dtype=torch.int64, device="cuda")
        s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal(gen, (len(lens), hq * dh), 1.5)
        s["mask"] = _slot_mask(lens, rows, row0) if case["masked"] else None
    s["k"] = _normal(gen, (rows, hkv * dh))
    s["v"] = _normal(gen, (rows, hkv * dh))
    s["out"] = torch.zeros_like(s["q"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from flow_matching_action_gb300 import ae, synth
        dims = synth.ExpertDims(layers=1, width=128, mlp=128, n_q_heads=s["hq"], n_kv_heads=s["hkv"],
                                head_dim=s["dh"], horizon=1, action_dim=8, dtype="bf16", rms_eps=EPS,
                                rope_theta=THETA)
        weights = {}
        for name, shape in synth.global_weight_shapes(dims):
            weights[name] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        for name, shape in synth.layer_weight_shapes(dims):
            weights[name] = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda")]
        s["expert"] = ae.ActionExpert(dims, weights, 1, 0, stream=torch.cuda.current_stream().cuda_stream)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_rope(s):
    s["expert"].qk_norm_rope(s["qkv"], s["positions"], s["q_out"], s["k_cache"], s["v_cache"], q_norm=s["q_norm"],
                             k_norm=s["k_norm"], pair_axis=s["pair_axis"], kv_rows=s["kv_rows"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_prompt(s):
    return s["expert"].prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], kv_row0=s["kv_row0"], kv_len=s["kv_len"],
                                        key_mask=s["mask"], out=s["out"])


def _own_token(s):
    return s["expert"].token_attention(s["q"], s["k"], s["v"], s["row0"], s["len"], s["max_len"],
                                       key_mask=s["mask"], out=s["out"])


def _turned(x, weight, cos, sin):
    """[tokens, heads, dh] 32-bit: RMS norm of every head, then the rotation of pairs (j, j + dh / 2)."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_rope(s):
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    t = s["qkv"].shape[0]
    x = s["qkv"].float().view(t, hq + 2 * hkv, dh)
    half = dh // 2
    freq = THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    pos = s["positions"].double()  # angles of far positions need 64 bits
    axes = pos.shape[0]
    which = torch.arange(half, device="cuda") % axes
    ang = pos.t()[:, which] * freq
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    s["q_out"].copy_(_turned(x[:, :hq], s["q_norm"], cos, sin).reshape(t, hq * dh))
    k = _turned(x[:, hq:hq + hkv], s["k_norm"], cos, sin).reshape(t, hkv * dh).to(torch.bfloat16)
    v = x[:, hq + hkv:].reshape(t, hkv * dh).to(torch.bfloat16)
    if s["kv_rows"] is None:
        s["k_cache"].copy_(k)
        s["v_cache"].copy_(v)
    else:
        s["k_cache"][s["kv_rows"]] = k
        s["v_cache"][s["kv_rows"]] = v
    return s["q_out"], s["k_cache"], s["v_cache"]


def _weights_times_values(score, v):
    """softmax(score) v over the last axis of score; a row without keys gives zeros."""
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s):
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(dh)
    for b, (row0, n_keys) in enumerate(zip(s["kv_row0"], s["kv_len"])):
        q0, q1 = s["cu_q"][b], s["cu_q"][b + 1]
        n_new = q1 - q0
        k = s["k"][row0:row0 + n_keys].float().view(n_keys, hkv, dh)
        v = s["v"][row0:row0 + n_keys].float().view(n_keys, hkv, dh)
        q = s["q"][q0:q1].float().view(n_new, hkv, g, dh)
        key = torch.arange(n_keys, device="cuda")
        step = max(1, (1 << 27) // (g * n_keys))
        for i in range(0, n_new, step):
            j = min(i + step, n_new)
            hi = n_keys - n_new + j  # keys any query of the block sees
            last = n_keys - n_new + torch.arange(i, j, device="cuda")
            seen = key[None, :hi] <= last[:, None]
            if s["mask"] is not None:
                seen = seen & (s["mask"][row0:row0 + hi] != 0)
            for h in range(hkv):
                score = torch.matmul(q[i:j, h], k[:hi, h].t()) * scale  # [block, g, keys]
                score = score.masked_fill(~seen[:, None], -math.inf)
                o = _weights_times_values(score, v[:hi, h])
                s["out"][q0 + i:q0 + j, h * g * dh:(h + 1) * g * dh] = o.reshape(j - i, g * dh).to(torch.bfloat16)
    return s["out"]


def _plain_token(s):
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(dh)
    key = torch.arange(s["max_len"], device="cuda")
    for b in range(s["q"].shape[0]):
        rows = (s["row0"][b] + key).clamp(max=s["k"].shape[0] - 1)
        seen = key < s["len"][b]
        if s["mask"] is not None:
            seen = seen & (s["mask"][rows] != 0)
        k = s["k"][rows].float().view(-1, hkv, dh).permute(1, 2, 0)
        v = s["v"][rows].float().view(-1, hkv, dh).permute(1, 0, 2)
        score = torch.matmul(s["q"][b].float().view(hkv, g, dh), k) * scale
        o = _weights_times_values(score.masked_fill(~seen, -math.inf), v)
        s["out"][b] = o.reshape(hq * dh).to(torch.bfloat16)
    return s["out"]


_OWN = {"rope": _own_rope, "prompt": _own_prompt, "token": _own_token}
_PLAIN = {"rope": _plain_rope, "prompt": _plain_prompt, "token": _plain_token}


# ---------------------------------------------------------------- 64-bit values

def _exact_rope(s):
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    half, axes = dh // 2, s["positions"].shape[0]
    t = s["qkv"].shape[0]
    pos = s["positions"].double()
    z = torch.empty((t, half), dtype=torch.complex128, device="cuda")
    for j in range(half):  # a unit complex number for every pair
        a = pos[j % axes] * THETA ** (-2.0 * j / dh)
        z[:, j] = torch.polar(torch.ones_like(a), a)

    def head(col, weight):
        x = s["qkv"][:, col:col + dh].double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / dh + EPS) * weight.double()
        y = torch.complex(x[:, :half], x[:, half:]) * z
        return torch.cat((y.real, y.imag), 1)

    q = torch.empty((t, hq * dh), dtype=torch.float64, device="cuda")
    for h in range(hq):
        q[:, h * dh:(h + 1) * dh] = head(h * dh, s["q_norm"])
    k, v = s["k_cache"].double(), s["v_cache"].double()
    rows = s["kv_rows"] if s["kv_rows"] is not None else torch.arange(t, device="cuda")
    for h in range(hkv):
        k[rows, h * dh:(h + 1) * dh] = head((hq + h) * dh, s["k_norm"])
    v[rows] = s["qkv"][:, (hq + hkv) * dh:].double()
    return q, k, v


def _exact_rows(q, k, v, seen, dh):
    """One head: queries [n, dh] over keys [m, dh], a row without keys giving zeros."""
    e = torch.einsum("nd,md->nm", q, k) / math.sqrt(dh)
    e[~seen] = -math.inf
    w = torch.nan_to_num(torch.softmax(e, dim=1), nan=0.0)
    return w @ v


def exact(case, seed):
    if case["op"] != "rope" and work(case)["flops"] > 1.5e12:
        return None
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        spans = [(s["cu_q"][b], s["cu_q"][b + 1], r, n) for b, (r, n) in enumerate(zip(s["kv_row0"], s["kv_len"]))]
    else:
        spans = [(b, b + 1, r, n) for b, (r, n) in enumerate(zip(s["row0"].tolist(), s["len"].tolist()))]
    for q0, q1, r, n in spans:
        for h in range(hkv):
            k = s["k"][r:r + n, h * dh:(h + 1) * dh].double()
            v = s["v"][r:r + n, h * dh:(h + 1) * dh].double()
            for i in range(q0, q1, 2048):
                j = min(i + 2048, q1)
                m = n - q1 + j
                place = torch.arange(m, device="cuda")
                seen = place.unsqueeze(0) <= (torch.arange(i, j, device="cuda") + (n - q1)).unsqueeze(1)
                if s["mask"] is not None:
                    seen = seen & s["mask"][r:r + m].bool().unsqueeze(0)
                for c in range(h * g * dh, (h + 1) * g * dh, dh):
                    out[i:j, c:c + dh] = _exact_rows(s["q"][i:j, c:c + dh].double(), k[:m], v[:m], seen, dh)
    return out
