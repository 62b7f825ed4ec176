"""Calls that the language-model operators take, through the binding and the entry points, on launches
that only record their arguments (CPU tensors, no GPU)."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import pytest

from flow_matching_action_gb300 import ae
from flow_matching_action_gb300 import build as ae_build

HERE = os.path.dirname(os.path.abspath(__file__))
HQ, HKV, DH = 8, 2, 64
QD, KVD = HQ * DH, HKV * DH


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("hostops") / "libhostops.so")
    r = subprocess.run([ae_build._nvcc()] + ae_build.NVCC_FLAGS +
                       ["-shared", "-o", so, os.path.join(HERE, "host_lm_ops.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    h = ctypes.CDLL(so)
    h.host_context.restype = ctypes.c_void_p
    h.host_context_free.argtypes = [ctypes.c_void_p]
    for name in ("ae_qk_norm_rope", "ae_prompt_attention", "ae_token_attention", "ae_last_error"):
        fn = getattr(h, name)
        fn.restype, fn.argtypes = ae._SIGNATURES[name]
    return h


@pytest.fixture
def expert(host, monkeypatch):
    """An ActionExpert over the recording launches, for CPU tensors."""
    monkeypatch.setattr(ae, "_lib", host)
    monkeypatch.setattr(ae, "_packed", {})
    ae._load_dtypes()
    ex = object.__new__(ae.ActionExpert)
    ex.dims = type("Dims", (), dict(head_dim=DH, n_q_heads=HQ, n_kv_heads=HKV, layers=1, width=128))()
    ex._q_dim, ex._kv_dim, ex._device = QD, KVD, -1  # a CPU tensor's get_device()
    ex._axis_array = ctypes.c_uint8 * (DH // 2)
    ctx = host.host_context(HQ, HKV, DH)
    ex.ctx = ctypes.c_void_p(ctx)
    yield ex
    ex.ctx = None
    host.host_context_free(ctx)


def bf16(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("tokens", [1, 2, 5])
def test_rotation_in_place_takes_any_token_count(host, expert, tokens):
    """q_out is the projection's own columns: one row has a stride like any other."""
    import torch
    qkv = bf16(tokens, QD + 2 * KVD)
    before = host.host_launches()
    expert.qk_norm_rope(qkv, torch.zeros(tokens, dtype=torch.int32), qkv[:, :QD], bf16(8, KVD), bf16(8, KVD))
    assert host.host_launches() == before + 1
    q_stride, qkv_stride = ctypes.c_int64(), ctypes.c_int64()
    host.host_rope_rows.restype = ctypes.c_void_p
    at = host.host_rope_rows(ctypes.byref(q_stride), ctypes.byref(qkv_stride))
    assert at == qkv.data_ptr()
    assert tokens == 1 or q_stride.value == qkv_stride.value == QD + 2 * KVD


def _raw_weights(dims):
    """Weights as plain addresses (nothing reads them here)."""
    from flow_matching_action_gb300 import synth
    w = {n: 0x10000 for n, _ in synth.global_weight_shapes(dims)}
    for n, _ in synth.layer_weight_shapes(dims):
        w[n] = [0x10000] * dims.layers
    return w


@pytest.mark.parametrize("torch_there", [False, True])
def test_a_context_of_plain_addresses_needs_no_torch(host, monkeypatch, torch_there):
    """Create, bind and sample take addresses: no torch, or one without a GPU, does not matter."""
    import sys

    import torch

    from flow_matching_action_gb300 import synth
    calls = []
    if torch_there:  # a build without CUDA
        def fail():
            raise AssertionError("Torch not compiled with CUDA enabled")
        monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
        monkeypatch.setattr(torch.cuda, "current_device", fail)
    else:
        monkeypatch.setitem(sys.modules, "torch", None)  # an import of it fails
    monkeypatch.setattr(ae, "ae_create", lambda *a: ctypes.c_void_p(None))
    monkeypatch.setattr(ae, "ae_bind_prefix", lambda *a: calls.append("bind"))
    monkeypatch.setattr(ae, "ae_sample", lambda *a: calls.append("sample"))
    dims = synth.ExpertDims(layers=1, width=128, mlp=128, n_q_heads=HQ, n_kv_heads=HKV, head_dim=DH, horizon=1,
                            action_dim=8, dtype="bf16")
    ex = ae.ActionExpert(dims, _raw_weights(dims), 1, 4)
    ex.bind_prefix(0x10000, 0x10000, [0, 4])
    assert ex.sample(0x10000, 1, out=0x20000) == 0x20000 and calls == ["bind", "sample"]


def test_operators_find_the_device_when_the_constructor_could_not(host, expert, monkeypatch):
    """A context made before torch was there: its tensors' device is the current one, looked up at each call."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    expert._device = None
    before = host.host_launches()
    x = bf16(3, QD)
    k = bf16(8, KVD)
    expert.prompt_attention(x, k, k, [0, 3])
    expert.token_attention(x, k, k, torch.zeros(3, dtype=torch.int64), torch.ones(3, dtype=torch.int32), 8)
    expert.qk_norm_rope(bf16(3, QD + 2 * KVD), torch.zeros(3, dtype=torch.int32), x, k, k)
    assert host.host_launches() == before + 3
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        expert.prompt_attention(x, k, k, [0, 3])


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("stride", [QD, QD + 8, 2 * QD])
def test_attention_over_the_queries_keeps_their_stride(host, expert, rows, stride):
    """With out == q and another stride an output row would land on a query row that is still to be read."""
    import torch
    q = torch.zeros(rows * 2 * QD, dtype=torch.bfloat16)
    k = bf16(8, KVD)
    row0, lens = torch.zeros(rows, dtype=torch.int64), torch.ones(rows, dtype=torch.int32)
    wide, over = q.as_strided((rows, QD), (QD + 8, 1)), q.as_strided((rows, QD), (stride, 1))
    calls = [lambda out: expert.prompt_attention(wide, k, k, [0, rows], out=out),
             lambda out: expert.token_attention(wide, k, k, row0, lens, 8, out=out)]
    for call in calls:
        before = host.host_launches()
        if rows == 1 or stride == QD + 8:
            call(over)
            assert host.host_launches() == before + 1
        else:
            with pytest.raises(ae.AEError, match="strides differ") as e:
                call(over)
            assert e.value.status == -1 and host.host_launches() == before


TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)
FREQUENCIES = [0.0, 1.0, 0.3, 1e-3, 1e-4, 3.7e-9, 2.0 ** -60, 0.5, math.pi, 2 * math.pi, 6.283185307179587, 100.7,
               12345.678, 2.0 ** 30]


@pytest.mark.parametrize("f", FREQUENCIES + [-f for f in FREQUENCIES[1:]])
def test_frequencies_are_fractions_of_a_turn_to_64_bits(host, f):
    """radians / 2 pi modulo one turn in units of 2^-64, against 80 digits of pi.

    1 / (2 pi) is held as the sum of two doubles, off by less than 2^-110; the fraction's and the remainder's
    conversions each cut less than one unit, and the remainder (at most 2^-53 of the turns, so 2^-26 of a turn
    at 2^30 radians) is off by its own rounding of 2^-53: 2^-79 turns.  Two units in all, and 2^-110 times the
    turns (2^28 at most: 2^-82)."""
    host.host_turn_fraction.restype = ctypes.c_uint64
    host.host_turn_fraction.argtypes = [ctypes.c_double]
    want = Fraction(f) / TWO_PI % 1 * 2 ** 64
    off = (host.host_turn_fraction(f) - want) % 2 ** 64
    assert min(off, 2 ** 64 - off) <= 2, float(min(off, 2 ** 64 - off))


def test_the_gpu_s_cluster_counts_are_the_context_s_own(host, expert):
    """What the split of the keys is chosen by belongs to a context: another one's set-up, perhaps on another
    thread or GPU, does not change it."""
    host.host_set_clusters.argtypes = [ctypes.c_void_p, ctypes.c_int]
    host.host_set_clusters(expert.ctx, 152)
    other = host.host_context(HQ, HKV, DH)
    try:
        host.host_set_clusters(other, 7)
        q, k = bf16(3, QD), bf16(8, KVD)
        expert.prompt_attention(q, k, k, [0, 3])
        assert host.host_clusters() == 152
    finally:
        host.host_context_free(other)


def test_rotation_without_a_cache_row(host, expert):
    """No token's K and V are stored (all rows negative): a cache without rows, which has no address, will do."""
    import torch
    rows = torch.full((3,), -1, dtype=torch.int64)
    pos, q = torch.zeros(3, dtype=torch.int32), bf16(3, QD)
    before = host.host_launches()
    expert.qk_norm_rope(bf16(3, QD + 2 * KVD), pos, q, bf16(0, KVD), bf16(0, KVD), kv_rows=rows)
    assert host.host_launches() == before + 1
    with pytest.raises(ae.AEError):  # without kv_rows the tokens need their rows
        expert.qk_norm_rope(bf16(3, QD + 2 * KVD), pos, q, bf16(0, KVD), bf16(0, KVD))
