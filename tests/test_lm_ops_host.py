"""Refusals of the language-model operators: every bad argument is answered on
the host, before any CUDA call (these run without a GPU, on fake pointers)."""
import ctypes
import os
import subprocess

import pytest

from flow_matching_action_gb300 import ae
from flow_matching_action_gb300 import build as ae_build

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 0x10000  # a non-NULL, aligned address nothing reads
INVALID, SHAPE, UNSUPPORTED = -1, -2, -7


@pytest.fixture(scope="module")
def make_context(tmp_path_factory):
    ae_build.build()
    so = str(tmp_path_factory.mktemp("hostctx") / "libhostctx.so")
    r = subprocess.run([ae_build._nvcc()] + ae_build.NVCC_FLAGS +
                       ["-shared", "-o", so, os.path.join(HERE, "host_context.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    h = ctypes.CDLL(so)
    h.host_context.restype = ctypes.c_void_p
    h.host_context_free.argtypes = [ctypes.c_void_p]
    made = []

    def make(hq=8, hkv=2, dh=64, bf16=1):
        c = h.host_context(hq, hkv, dh, bf16)
        made.append(c)
        return c
    yield make
    for c in made:
        h.host_context_free(c)


def i32(*v):
    return (ctypes.c_int32 * len(v))(*v)


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rope_args(**kw):
    a = ae.ae_qk_norm_rope_args(tokens=4, n_axes=2, qkv=FAKE, qkv_stride=768, q_norm=FAKE, k_norm=FAKE,
                                positions=FAKE, kv_rows=FAKE, cache_rows=8, q_out=2 * FAKE, q_stride=512,
                                k_cache=3 * FAKE, v_cache=4 * FAKE, kv_stride=128)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def prompt_args(cu=(0, 3, 7), row0=(0, 10), lens=(3, 9), **kw):
    a = ae.ae_prompt_attention_args(batch=len(cu) - 1, causal=1, cache_rows=20, q=FAKE, q_stride=512, k=FAKE, v=FAKE,
                                    kv_stride=128, out=FAKE, out_stride=512)
    a._keep = (i32(*cu), i64(*row0) if row0 else None, i32(*lens) if lens else None)
    a.cu_q, a.kv_row0, a.kv_len = [ae._addr(x) for x in a._keep]
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def token_args(**kw):
    a = ae.ae_token_attention_args(batch=3, max_len=10, kv_row0=FAKE, kv_len=FAKE, cache_rows=40, q=FAKE, q_stride=512,
                                   k=FAKE, v=FAKE, kv_stride=128, out=FAKE, out_stride=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def prefill_args(cu=(0, 2, 4), **kw):
    a = ae.ae_prefill_prompts_args(batch=len(cu) - 1, causal=1, embeddings=FAKE, n_axes=1, positions=FAKE, out_k=FAKE,
                                   out_v=FAKE)
    a._keep = i32(*cu)
    a.cu_lens = ae._addr(a._keep)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(call, ctx, args, status):
    with pytest.raises(ae.AEError) as e:
        call(ctx, args)
    assert e.value.status == status, e.value



@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE),
    (dict(norm_offset=float("nan")), INVALID), (dict(cache_rows=-1), SHAPE), (dict(cache_rows=1 << 31), SHAPE),
    (dict(pair_axis=bytes([0, 1, 2] + [0] * 29)), INVALID),
    (dict(qkv=None), INVALID), (dict(qkv=FAKE + 8), INVALID), (dict(qkv_stride=760), SHAPE),
    (dict(qkv_stride=772), INVALID), (dict(q_out=None), INVALID), (dict(q_stride=504), SHAPE),
    (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 4), INVALID), (dict(kv_stride=64), SHAPE),
    (dict(kv_stride=-128), SHAPE), (dict(kv_stride=1 << 40), SHAPE), (dict(positions=None), INVALID),
    (dict(positions=FAKE + 2), INVALID), (dict(kv_rows=FAKE + 4), INVALID), (dict(q_norm=FAKE + 2), INVALID),
    (dict(kv_rows=None, cache_rows=3), SHAPE), (dict(q_out=FAKE, qkv_stride=776), INVALID)])
def test_qk_norm_rope_refuses(make_context, kw, status):
    refused(ae.ae_qk_norm_rope, make_context(), rope_args(**kw), status)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_qk_norm_rope_refuses_frequencies(make_context, bad):
    f = (ctypes.c_double * 32)(*([1.0] * 31 + [bad]))
    refused(ae.ae_qk_norm_rope, make_context(), rope_args(pair_freq=ctypes.addressof(f)), INVALID)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(batch=65), SHAPE), (dict(cu_q=None), INVALID), (dict(kv_len=None), INVALID),
    (dict(kv_row0=None), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(cache_rows=-5), SHAPE), (dict(cache_rows=18), SHAPE),
    (dict(q=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(q_stride=256), SHAPE), (dict(q_stride=513), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kv_stride=127), SHAPE), (dict(out=None), INVALID),
    (dict(out_stride=500), SHAPE), (dict(cu=(1, 3, 7)), SHAPE), (dict(cu=(0, 3, 2)), SHAPE),
    (dict(lens=(2, 9)), SHAPE), (dict(row0=(-1, 10)), SHAPE), (dict(row0=(0, 12)), SHAPE),
    (dict(row0=(0, 1 << 40)), SHAPE), (dict(row0=None, lens=None, cache_rows=6), SHAPE)])
def test_prompt_attention_refuses(make_context, kw, status):
    refused(ae.ae_prompt_attention, make_context(), prompt_args(**kw), status)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(max_len=-1), SHAPE), (dict(kv_row0=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(kv_row0=FAKE + 4), INVALID), (dict(kv_len=FAKE + 2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(cache_rows=-5), SHAPE), (dict(q=None), INVALID),
    (dict(q_stride=511), SHAPE), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(kv_stride=132), INVALID),
    (dict(out=None), INVALID), (dict(out_stride=1), SHAPE)])
def test_token_attention_refuses(make_context, kw, status):
    refused(ae.ae_token_attention, make_context(), token_args(**kw), status)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(batch=65), SHAPE), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE),
    (dict(pair_axis=bytes([1] * 32)), INVALID), (dict(norm_offset=float("inf")), INVALID),
    (dict(cu_lens=None), INVALID), (dict(cu=(0, 3, 2)), SHAPE), (dict(cu=(1, 2)), SHAPE), (dict(cu=(0, 2, 5)), SHAPE),
    (dict(embeddings=None), INVALID), (dict(embeddings=FAKE + 4), INVALID), (dict(out_k=None), INVALID),
    (dict(out_v=FAKE + 2), INVALID), (dict(positions=None), INVALID), (dict(positions=FAKE + 1), INVALID)])
def test_prefill_prompts_refuses(make_context, kw, status):
    refused(ae.ae_prefill_prompts, make_context(), prefill_args(**kw), status)


@pytest.mark.parametrize("norm", [None, FAKE + 8])
def test_prefill_prompts_refuses_norm_weights(make_context, norm):
    arr = (ctypes.c_void_p * 1)(norm)
    refused(ae.ae_prefill_prompts, make_context(), prefill_args(k_norm=ctypes.addressof(arr)), INVALID)


@pytest.mark.parametrize("call,args", [(ae.ae_prefill_prompts, prefill_args), (ae.ae_qk_norm_rope, rope_args), (ae.ae_prompt_attention, prompt_args),
                                       (ae.ae_token_attention, token_args)])
def test_fp32_contexts_and_null_are_refused(make_context, call, args):
    refused(call, make_context(bf16=0), args(), UNSUPPORTED)
    lib = ae.lib()
    fn = getattr(lib, call.__name__)
    assert fn(None, ctypes.byref(args())) == INVALID
    assert fn(make_context(), None) == INVALID


def test_nothing_to_do_is_ok(make_context):
    c = make_context()
    ae.ae_qk_norm_rope(c, rope_args(tokens=0, qkv=None, q_out=None, k_cache=None, v_cache=None, positions=None))
    ae.ae_prompt_attention(c, prompt_args(cu=(0,), row0=None, lens=None, q=None, k=None, v=None, out=None))
    ae.ae_prompt_attention(c, prompt_args(cu=(0, 0, 0), row0=(0, 5), lens=(0, 3), q=None, k=None, v=None, out=None))
    ae.ae_prefill_prompts(c, prefill_args(cu=(0, 0), embeddings=None, out_k=None, out_v=None, positions=None))
    ae.ae_token_attention(c, token_args(batch=0, q=None, k=None, v=None, out=None))


@pytest.mark.parametrize("packed,fields", [(ae._ROPE_ARGS, ae.ae_qk_norm_rope_args),
                                           (ae._PROMPT_ARGS, ae.ae_prompt_attention_args),
                                           (ae._TOKEN_ARGS, ae.ae_token_attention_args)])
def test_packed_arguments_have_the_structs_layout(packed, fields):
    """Distinct values packed into bytes read back, field by field, through the ctypes structure."""
    values = list(range(1, len(fields._fields_) + 1))
    s = fields.from_buffer_copy(packed.pack(*values).ljust(ctypes.sizeof(fields), b"\0"))
    assert packed.size <= ctypes.sizeof(fields)
    for (name, kind), v in zip(fields._fields_, values):
        offset = getattr(fields, name).offset
        if kind is ctypes.c_char_p:  # a pointer this test must not follow
            got = ctypes.c_size_t.from_buffer_copy(bytes(s)[offset:offset + 8]).value
        else:
            got = getattr(s, name)
        assert got == v, name


def test_rope_token_counts_a_launch_cannot_index(make_context):
    refused(ae.ae_qk_norm_rope, make_context(), rope_args(tokens=2 ** 31 - 1, cache_rows=0x7fffff00), SHAPE)
