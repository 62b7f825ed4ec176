"""Calls that the language-model operators take, through the binding and the entry points, on launches
that only record their arguments (CPU tensors, no GPU)."""
import ctypes
import os
import subprocess

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
