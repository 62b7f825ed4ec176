"""ctypes binding of ``include/ae.h``: same names, argument marshalling only.

Every step of the denoise loop runs in the CUDA library; this module only turns
torch tensors into raw pointers and status codes into exceptions.  There is no
CPU or PyTorch fallback: if ``libae.so`` has not been built, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import sys
from typing import Dict, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libae.so")

AE_OK = 0
AE_DTYPE_BF16 = 0
AE_DTYPE_F32 = 1
AE_WEIGHTS_AS_DTYPE = 0
AE_WEIGHTS_FP8_E4M3 = 1
AE_MAX_BATCH = 64
AE_MAX_STEPS = 128
AE_MAX_AXES = 4
AE_MAX_TOKENS = 65535

STATUS_NAMES = {0: "AE_OK", -1: "AE_ERR_INVALID_ARG", -2: "AE_ERR_SHAPE", -3: "AE_ERR_NOT_BOUND",
                -4: "AE_ERR_CUDA", -5: "AE_ERR_DEVICE", -6: "AE_ERR_OOM", -7: "AE_ERR_UNSUPPORTED"}


class AEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class ae_config(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int), ("width", ctypes.c_int), ("mlp", ctypes.c_int),
                ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("action_dim", ctypes.c_int), ("horizon", ctypes.c_int),
                ("rms_eps", ctypes.c_double), ("rope_theta", ctypes.c_double),
                ("time_min_period", ctypes.c_double), ("time_max_period", ctypes.c_double),
                ("dtype", ctypes.c_int), ("ctx_dim", ctypes.c_int), ("weight_format", ctypes.c_int)]


_GLOBAL = ("w_in", "b_in", "w_t1", "b_t1", "w_t2", "b_t2", "w_mod_f", "b_mod_f", "w_out", "b_out")
_LAYER = ("wq", "wk", "wv", "wo", "wg", "wu", "wd", "w_mod1", "b_mod1", "w_mod2", "b_mod2")
_CONTEXT = ("w_ck", "w_cv")  # per layer, only with ctx_dim > 0


class ae_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _GLOBAL] + \
               [(n, ctypes.POINTER(ctypes.c_void_p)) for n in _LAYER + _CONTEXT]


class ae_info(ctypes.Structure):
    _fields_ = [("launches_last_sample", ctypes.c_int64), ("launches_last_bind", ctypes.c_int64),
                ("device_bytes", ctypes.c_int64), ("sm_count", ctypes.c_int), ("path", ctypes.c_int)]


class ae_qk_norm_rope_args(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("n_axes", ctypes.c_int), ("qkv", ctypes.c_void_p),
                ("qkv_stride", ctypes.c_int64), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("norm_offset", ctypes.c_float), ("positions", ctypes.c_void_p),
                ("pair_axis", ctypes.c_char_p), ("pair_freq", ctypes.c_void_p),
                ("kv_rows", ctypes.c_void_p), ("cache_rows", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("kv_stride", ctypes.c_int64)]


class ae_prompt_attention_args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("causal", ctypes.c_int), ("cu_q", ctypes.c_void_p),
                ("kv_row0", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("cache_rows", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("kv_stride", ctypes.c_int64), ("key_mask", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64)]


class ae_token_attention_args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("max_len", ctypes.c_int), ("kv_row0", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("cache_rows", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("kv_stride", ctypes.c_int64), ("key_mask", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64)]


class ae_prefill_prompts_args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("causal", ctypes.c_int), ("cu_lens", ctypes.c_void_p),
                ("embeddings", ctypes.c_void_p), ("token_mask", ctypes.c_void_p), ("n_axes", ctypes.c_int),
                ("positions", ctypes.c_void_p), ("pair_axis", ctypes.c_char_p), ("pair_freq", ctypes.c_void_p),
                ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("norm_offset", ctypes.c_float),
                ("out_k", ctypes.c_void_p), ("out_v", ctypes.c_void_p)]


# Every symbol include/ae.h declares, with its ctypes signature.
_SIGNATURES = {
    "ae_create": (ctypes.c_int, [ctypes.POINTER(ae_config), ctypes.POINTER(ae_weights), ctypes.c_int,
                                 ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]),
    "ae_destroy": (None, [ctypes.c_void_p]),
    "ae_set_stream": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "ae_bind_prefix": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p]),
    "ae_bind_prefix_shared": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_void_p]),
    "ae_bind_context": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p]),
    "ae_prefill": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "ae_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ae_qk_norm_rope_args)]),
    "ae_prompt_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ae_prompt_attention_args)]),
    "ae_token_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ae_token_attention_args)]),
    "ae_prefill_prompts": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ae_prefill_prompts_args)]),
    "ae_sample": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "ae_sample_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "ae_set_debug_dump": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t]),
    "ae_synchronize": (ctypes.c_int, [ctypes.c_void_p]),
    "ae_last_error": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_size_t]),
    "ae_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ae_get_info": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ae_info)]),
    "ae_get_fp8_weight": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.POINTER(ctypes.c_float)]),
    "ae_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m flow_matching_action_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _msg(ctx) -> str:
    buf = ctypes.create_string_buffer(512)
    lib().ae_last_error(ctx, buf, 512)
    return buf.value.decode(errors="replace")


def _check(status: int, ctx=None):
    if status != AE_OK:
        raise AEError(status, _msg(ctx))


def ae_status_string(status: int) -> str:
    return lib().ae_status_string(status).decode()


def make_config(dims, dtype: Optional[str] = None, fp8_weights: bool = False) -> ae_config:
    """An ae_config from any object with the expert-dimension attributes."""
    dt = dtype or dims.dtype
    return ae_config(dims.layers, dims.width, dims.mlp, dims.n_q_heads, dims.n_kv_heads, dims.head_dim,
                     dims.action_dim, dims.horizon, dims.rms_eps, dims.rope_theta,
                     dims.time_min_period, dims.time_max_period,
                     AE_DTYPE_BF16 if dt == "bf16" else AE_DTYPE_F32, getattr(dims, "ctx_dim", 0),
                     AE_WEIGHTS_FP8_E4M3 if fp8_weights else AE_WEIGHTS_AS_DTYPE)


def make_weights(w: Dict) -> ae_weights:
    """An ae_weights from a dict of tensors (global names -> tensor, layer names -> list).

    The returned struct keeps the per-layer pointer arrays alive as attributes.
    """
    s = ae_weights()
    keep = []
    for n in _GLOBAL:
        setattr(s, n, _ptr(w[n]))
    for n in _LAYER + _CONTEXT:
        if n not in w:  # context projections are optional
            continue
        arr = (ctypes.c_void_p * len(w[n]))(*[_ptr(t) for t in w[n]])
        keep.append(arr)
        setattr(s, n, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)))
    s._keep = keep
    return s


def ae_create(config: ae_config, weights: ae_weights, max_batch: int, max_prefix_rows: int,
              stream=None) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    st = lib().ae_create(ctypes.byref(config), ctypes.byref(weights), max_batch, max_prefix_rows,
                         stream, ctypes.byref(out))
    _check(st, None)
    return out


def ae_destroy(ctx) -> None:
    lib().ae_destroy(ctx)


def ae_set_stream(ctx, stream) -> None:
    _check(lib().ae_set_stream(ctx, stream), ctx)


def ae_bind_prefix(ctx, batch: int, prefix_k, prefix_v, cu_lens: Sequence[int], prefix_mask=None) -> None:
    cu = (ctypes.c_int32 * (len(cu_lens)))(*[int(v) for v in cu_lens]) if cu_lens is not None else None
    _check(lib().ae_bind_prefix(ctx, batch, _ptr(prefix_k), _ptr(prefix_v), cu, _ptr(prefix_mask)), ctx)


def ae_bind_prefix_shared(ctx, n_samples: int, prefix_k, prefix_v, n_rows: int, prefix_mask=None) -> None:
    _check(lib().ae_bind_prefix_shared(ctx, n_samples, _ptr(prefix_k), _ptr(prefix_v), int(n_rows),
                                       _ptr(prefix_mask)), ctx)


def ae_bind_context(ctx, batch: int, hidden, cu_lens: Sequence[int], prefix_mask=None) -> None:
    cu = (ctypes.c_int32 * (len(cu_lens)))(*[int(v) for v in cu_lens]) if cu_lens is not None else None
    _check(lib().ae_bind_context(ctx, batch, _ptr(hidden), cu, _ptr(prefix_mask)), ctx)


def ae_prefill(ctx, batch: int, embeddings, out_k, out_v) -> None:
    _check(lib().ae_prefill(ctx, batch, _ptr(embeddings), _ptr(out_k), _ptr(out_v)), ctx)


def ae_qk_norm_rope(ctx, args: ae_qk_norm_rope_args) -> None:
    _check(lib().ae_qk_norm_rope(ctx, ctypes.byref(args)), ctx)


def ae_prompt_attention(ctx, args: ae_prompt_attention_args) -> None:
    _check(lib().ae_prompt_attention(ctx, ctypes.byref(args)), ctx)


def ae_token_attention(ctx, args: ae_token_attention_args) -> None:
    _check(lib().ae_token_attention(ctx, ctypes.byref(args)), ctx)


def ae_prefill_prompts(ctx, args: ae_prefill_prompts_args) -> None:
    _check(lib().ae_prefill_prompts(ctx, ctypes.byref(args)), ctx)


_BF16 = _I32 = _I64 = _U8 = None  # torch dtypes: this module imports torch only for the operators' tensors


def _load_dtypes():
    global _BF16, _I32, _I64, _U8
    import torch
    _BF16, _I32, _I64, _U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8


def _torch_device() -> Optional[int]:
    """The current device where this process uses torch with a GPU, else None."""
    torch = sys.modules.get("torch")
    return torch.cuda.current_device() if torch is not None and torch.cuda.is_available() else None


def _rows(name: str, t, width: int, device: int, rows: int = -1):
    """(pointer, row stride, rows) of a bf16 tensor [rows, width] on the device whose rows are contiguous."""
    shape, step = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width or (rows >= 0 and shape[0] != rows):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{'rows' if rows < 0 else rows}, {width}]")
    if t.dtype is not _BF16 or t.get_device() != device:
        raise ValueError(f"{name}: expected a bf16 tensor on cuda:{device}, got {t.dtype} on {t.device}")
    if step[1] != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    n = shape[0]
    return t.data_ptr(), step[0] if n > 1 else width, n  # one row has no stride


def _vec(name: str, t, dtype, device: int, n: int) -> int:
    """Pointer of a contiguous tensor of n elements on the device, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name}: expected {n} contiguous {dtype} elements on cuda:{device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    return t.data_ptr()


def _host_array(ctype, x):
    """A host array of a sequence (kept as it is when it already is one of that type), or None."""
    if x is None or (isinstance(x, ctypes.Array) and x._type_ is ctype):
        return x
    return (ctype * len(x))(*x)


def _addr(arr) -> int:
    return 0 if arr is None else ctypes.addressof(arr)


# The argument structs of the operators as packed bytes, in C's own layout ("@"):
# a third of the time of filling a ctypes structure, which shows in a call that
# takes the GPU a few microseconds.
_ROPE_ARGS = struct.Struct("@iiPqPPfPPPPqPqPPq")
_PROMPT_ARGS = struct.Struct("@iiPPPqPqPPqPfPq")
_TOKEN_ARGS = struct.Struct("@iiPPqPqPPqPfPq")
_packed = {}


def _call_packed(name: str, ctx, args: bytes) -> None:
    fn = _packed.get(name)
    if fn is None:
        fn = _packed[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_char_p)((name, lib()))
    status = fn(ctx, args)
    if status != AE_OK:
        raise AEError(status, _msg(ctx))


def _pairs(pair_axis, pair_freq, half: int):
    """(bytes of the axes, array of the frequencies) of dh / 2 rotation pairs, None as given."""
    if pair_axis is not None:
        if len(pair_axis) != half:
            raise ValueError(f"pair_axis: {len(pair_axis)} entries, expected {half}")
        pair_axis = pair_axis if isinstance(pair_axis, bytes) else bytes(pair_axis)
    freq = _host_array(ctypes.c_double, pair_freq)
    if freq is not None and len(freq) != half:
        raise ValueError(f"pair_freq: {len(freq)} entries, expected {half}")
    return pair_axis, freq


def ae_sample(ctx, noise, n_steps: int, out_actions) -> None:
    _check(lib().ae_sample(ctx, _ptr(noise), n_steps, _ptr(out_actions)), ctx)


def ae_sample_noalloc(ctx, noise, n_steps: int, out_actions) -> None:
    """ae_sample without device-memory allocation (see include/ae.h): for callers
    that sample inside a stream capture or under a fixed HBM budget."""
    _check(lib().ae_sample_noalloc(ctx, _ptr(noise), n_steps, _ptr(out_actions)), ctx)


def ae_selftest_wait_timeout(ctx, budget_cycles: int) -> None:
    """Run one bounded device wait that nothing completes (see include/ae.h):
    the context's sticky status becomes AE_ERR_DEVICE."""
    _check(lib().ae_selftest_wait_timeout(ctx, int(budget_cycles)), ctx)


def ae_set_debug_dump(ctx, hidden, capacity: int) -> None:
    _check(lib().ae_set_debug_dump(ctx, _ptr(hidden), capacity), ctx)


def ae_synchronize(ctx) -> None:
    _check(lib().ae_synchronize(ctx), ctx)


def ae_last_error(ctx) -> str:
    return _msg(ctx)


FP8_LINEARS = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")  # the `which` of ae_get_fp8_weight


def ae_get_fp8_weight(ctx, layer: int, which: int, codes=None) -> float:
    """Copy one quantized block Linear's e4m3 codes into `codes` (a writable
    uint8 numpy array of the tensor's shape, or None) and return its factor r."""
    r = ctypes.c_float(0.0)
    ptr = None if codes is None else codes.ctypes.data_as(ctypes.c_void_p)
    _check(lib().ae_get_fp8_weight(ctx, layer, which, ptr, ctypes.byref(r)), ctx)
    return r.value


def ae_get_info(ctx) -> dict:
    info = ae_info()
    _check(lib().ae_get_info(ctx, ctypes.byref(info)), ctx)
    return {f: getattr(info, f) for f, _ in ae_info._fields_}


class ActionExpert:
    """Convenience owner of one context: create / bind / sample / destroy.

    Holds references to the borrowed prefix tensors so they outlive the binding.
    Calls enqueue on the context's stream: tensors (returned ones too) have to be
    ready and used there, or ordered with it, and stay allocated until it is done.
    """

    def __init__(self, dims, weights: Dict, max_batch: int, max_prefix_rows: int, stream=None,
                 dtype: Optional[str] = None, fp8_weights: bool = False):
        self.dims = dims
        self.config = make_config(dims, dtype, fp8_weights)
        self._wstruct = make_weights(weights)
        self._q_dim, self._kv_dim = dims.n_q_heads * dims.head_dim, dims.n_kv_heads * dims.head_dim
        self.ctx = ae_create(self.config, self._wstruct, max_batch, max_prefix_rows, stream)
        self._device = _torch_device()  # the context's, as ae_create takes it; None: not known
        self._axis_array = ctypes.c_uint8 * (dims.head_dim // 2)
        self._bound = None

    def _tensor_device(self) -> int:
        """The device an operator's tensors have to be on (the library checks that the context's is current)."""
        if _BF16 is None:
            _load_dtypes()
        if self._device is not None:
            return self._device
        import torch
        return torch.cuda.current_device()

    def bind_prefix(self, prefix_k, prefix_v, cu_lens, prefix_mask=None):
        batch = len(cu_lens) - 1
        ae_bind_prefix(self.ctx, batch, prefix_k, prefix_v, cu_lens, prefix_mask)
        self._bound = (prefix_k, prefix_v, prefix_mask)

    def bind_context(self, hidden, cu_lens, prefix_mask=None):
        """Per-layer VLM hidden states projected into K/V once, then bound."""
        ae_bind_context(self.ctx, len(cu_lens) - 1, hidden, cu_lens, prefix_mask)
        self._bound = (None, None, prefix_mask)

    def bind_prefix_shared(self, n_samples: int, prefix_k, prefix_v, n_rows: int, prefix_mask=None):
        """One request's prefix bound for n_samples samples of the same observation."""
        ae_bind_prefix_shared(self.ctx, n_samples, prefix_k, prefix_v, n_rows, prefix_mask)
        self._bound = (prefix_k, prefix_v, prefix_mask)

    def qk_norm_rope(self, qkv, positions, q_out, k_cache, v_cache, q_norm=None, k_norm=None,
                     norm_offset: float = 0.0, pair_axis=None, pair_freq=None, kv_rows=None):
        """Per-head norm, rotation and cache write of merged q|k|v rows (see include/ae.h).

        qkv [tokens, (Hq + 2 Hkv) dh], q_out [tokens, Hq dh], k_cache / v_cache [rows, Hkv dh]: bf16.
        positions int32 [tokens] or [axes, tokens]; kv_rows int64 [tokens] or None; pair_axis bytes or a
        sequence of dh / 2 axes; pair_freq a sequence of dh / 2 frequencies.
        """
        qd, kvd, dh, dev = self._q_dim, self._kv_dim, self.dims.head_dim, self._tensor_device()
        axes = positions.shape[0] if positions.dim() == 2 else 1
        pair_axis, freq = _pairs(pair_axis, pair_freq, dh // 2)
        x, x_stride, n = _rows("qkv", qkv, qd + 2 * kvd, dev)
        q, q_stride, _ = _rows("q_out", q_out, qd, dev, n)
        k, k_stride, cache_rows = _rows("k_cache", k_cache, kvd, dev)
        v, v_stride, _ = _rows("v_cache", v_cache, kvd, dev, cache_rows)
        if v_stride != k_stride:
            raise ValueError("k_cache and v_cache have different row strides")
        axis = None if pair_axis is None else self._axis_array.from_buffer_copy(pair_axis)
        _call_packed("ae_qk_norm_rope", self.ctx, _ROPE_ARGS.pack(
            n, axes, x, x_stride, _vec("q_norm", q_norm, _BF16, dev, dh), _vec("k_norm", k_norm, _BF16, dev, dh),
            norm_offset, _vec("positions", positions, _I32, dev, axes * n), _addr(axis), _addr(freq),
            _vec("kv_rows", kv_rows, _I64, dev, n), cache_rows, q, q_stride, k, v, k_stride))

    def prompt_attention(self, q, k, v, cu_q, kv_row0=None, kv_len=None, key_mask=None, causal: bool = True,
                         scale: float = 0.0, out=None):
        """Attention of packed prompts (see include/ae.h); returns out [rows, Hq dh].

        q [rows, Hq dh], k / v [cache rows, Hkv dh]: bf16.  cu_q, kv_row0, kv_len are host sequences;
        key_mask uint8 [cache rows] on the GPU.  Rows of out behind the last sequence are not written.
        """
        if out is None:
            out = q.new_empty(q.shape)
        cu = _host_array(ctypes.c_int32, cu_q)
        row0, lens = _host_array(ctypes.c_int64, kv_row0), _host_array(ctypes.c_int32, kv_len)
        batch = len(cu) - 1
        for name, x in (("kv_row0", row0), ("kv_len", lens)):
            if x is not None and len(x) != batch:
                raise ValueError(f"{name}: {len(x)} entries for {batch} sequences")
        dev = self._tensor_device()
        qp, q_stride, rows = _rows("q", q, self._q_dim, dev)
        if rows < cu[batch]:
            raise ValueError(f"q: {rows} rows, cu_q ends at {cu[batch]}")
        kp, k_stride, cache_rows = _rows("k", k, self._kv_dim, dev)
        vp, v_stride, _ = _rows("v", v, self._kv_dim, dev, cache_rows)
        if v_stride != k_stride:
            raise ValueError("k and v have different row strides")
        op, o_stride, _ = _rows("out", out, self._q_dim, dev, rows)
        _call_packed("ae_prompt_attention", self.ctx, _PROMPT_ARGS.pack(
            batch, 1 if causal else 0, _addr(cu), _addr(row0), _addr(lens), cache_rows, qp, q_stride, kp, vp, k_stride,
            _vec("key_mask", key_mask, _U8, dev, cache_rows), scale, op, o_stride))
        return out

    def token_attention(self, q, k, v, kv_row0, kv_len, max_len: int, key_mask=None, scale: float = 0.0, out=None):
        """Attention of one new token per request over its cached rows (see include/ae.h); returns out.

        q [requests, Hq dh], k / v [cache rows, Hkv dh]: bf16; kv_row0 int64, kv_len int32 [requests] and
        key_mask uint8 [cache rows] on the GPU.
        """
        if out is None:
            out = q.new_empty(q.shape)
        dev = self._tensor_device()
        qp, q_stride, n = _rows("q", q, self._q_dim, dev)
        kp, k_stride, cache_rows = _rows("k", k, self._kv_dim, dev)
        vp, v_stride, _ = _rows("v", v, self._kv_dim, dev, cache_rows)
        if v_stride != k_stride:
            raise ValueError("k and v have different row strides")
        op, o_stride, _ = _rows("out", out, self._q_dim, dev, n)
        _call_packed("ae_token_attention", self.ctx, _TOKEN_ARGS.pack(
            n, max_len, _vec("kv_row0", kv_row0, _I64, dev, n), _vec("kv_len", kv_len, _I32, dev, n), cache_rows, qp,
            q_stride, kp, vp, k_stride, _vec("key_mask", key_mask, _U8, dev, cache_rows), scale, op, o_stride))
        return out

    def prefill_prompts(self, embeddings, cu_lens, positions, out_k, out_v, causal: bool = True, token_mask=None,
                        q_norm=None, k_norm=None, norm_offset: float = 0.0, pair_axis=None, pair_freq=None):
        """VLM prefill of packed prompts (see include/ae.h): K and V of every layer into out_k / out_v.

        embeddings [total, width] bf16; positions int32 [total] or [axes, total]; out_k / out_v
        [layers, total, Hkv dh] bf16; q_norm / k_norm one bf16 [dh] tensor a layer.
        """
        d, dev = self.dims, self._tensor_device()
        cu = _host_array(ctypes.c_int32, cu_lens)
        n = embeddings.shape[0]
        if cu[len(cu) - 1] != n:
            raise ValueError(f"embeddings: {n} rows, cu_lens ends at {cu[len(cu) - 1]}")
        a = ae_prefill_prompts_args()
        a.batch, a.causal, a.cu_lens = len(cu) - 1, 1 if causal else 0, _addr(cu)
        a.embeddings = _vec("embeddings", embeddings, _BF16, dev, n * d.width)
        a.token_mask = _vec("token_mask", token_mask, _U8, dev, n)
        a.n_axes = positions.shape[0] if positions.dim() == 2 else 1
        a.positions = _vec("positions", positions, _I32, dev, a.n_axes * n)
        a.pair_axis, freq = _pairs(pair_axis, pair_freq, d.head_dim // 2)
        a.pair_freq = _addr(freq)
        norms = []
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None and len(w) != d.layers:
                raise ValueError(f"{name}: {len(w)} tensors for {d.layers} layers")
            norms.append(None if w is None else (ctypes.c_void_p * d.layers)(
                *[_vec(name, x, _BF16, dev, d.head_dim) for x in w]))
        a.q_norm, a.k_norm = _addr(norms[0]), _addr(norms[1])
        a.norm_offset = norm_offset
        a.out_k = _vec("out_k", out_k, _BF16, dev, d.layers * n * d.kv_dim)
        a.out_v = _vec("out_v", out_v, _BF16, dev, d.layers * n * d.kv_dim)
        ae_prefill_prompts(self.ctx, a)

    def sample(self, noise, n_steps: int, out=None):
        if out is None:
            out = noise.new_empty(noise.shape)
        ae_sample(self.ctx, noise, n_steps, out)
        return out

    def set_debug_dump(self, hidden):
        ae_set_debug_dump(self.ctx, hidden, 0 if hidden is None else hidden.numel())
        self._dump = hidden

    def synchronize(self):
        ae_synchronize(self.ctx)

    def info(self) -> dict:
        return ae_get_info(self.ctx)

    def close(self):
        if self.ctx is not None and self.ctx.value:
            ae_destroy(self.ctx)
        self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
