"""GB300 (sm_103a) SP-TP FFN boundary and Delayed-TP stack.

Thin ctypes binding over libsptp.so: every function here marshals torch
tensors (device memory) and the current CUDA stream into the C ABI declared
in include/sptp.h and raises on a non-zero status.  All computation runs in
the library's CUDA kernels; there is no fallback.  The calls of a decoding
step, a few microseconds each on the device, have a second way in, the
extension module _decode_binding (csrc/decode_binding.cpp): it makes the same
library call where nothing is wrong with the arguments, and leaves every other
call to the functions here.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import struct
import warnings

import torch

__all__ = [
    "SPTP_BF16", "SPTP_FP32", "SPTP_WS_HEADER_BYTES", "SptpError", "lib", "load_library",
    "sptp_ffn_workspace_size", "sptp_ffn_forward", "dtp_ffn_stack_workspace_size",
    "dtp_ffn_stack_forward", "sptp_prologue", "sptp_gateup_swiglu", "sptp_down_proj",
    "sptp_read_device_status", "sptp_wait_selftest", "sptp_status_string", "EXPORTED_SYMBOLS",
    "sptp_ffn_forward_noalloc", "SPTP_NOALLOC_SCRATCH_BYTES", "sptp_permute_ffn_neurons",
    "sptp_attn_qkv_workspace_size", "sptp_attn_qkv_forward", "sptp_quantize_rows_e4m3",
    "quantize_ffn_weights_e4m3", "sptp_ffn_fp8_workspace_size", "sptp_ffn_forward_fp8",
    "sptp_gateup_swiglu_e4m3", "sptp_down_proj_e4m3", "sptp_prologue_e4m3", "VARIANTS", "STATUS",
    "sptp_noalloc_read_device_status", "sptp_noalloc_wait_selftest", "CHECKED_LIB_PATH", "set_library",
    "sptp_rope_turns", "sptp_rope", "sptp_rope_append_kv", "sptp_paged_attn_workspace_size",
    "sptp_paged_attn_decode", "paged_kv_cache", "ROPE_SCALINGS", "sptp_paged_attn_wait_selftest",
    "sptp_paged_attn_prompt_workspace_size", "sptp_paged_attn_prompt", "sptp_lora_workspace_size", "sptp_lora",
    "sptp_paged_attn_prompt_wait_selftest",
]

SPTP_BF16 = 0
SPTP_FP32 = 1
SPTP_WS_HEADER_BYTES = 4096
SPTP_NOALLOC_SCRATCH_BYTES = 64 << 20
# sptp_variant: how a boundary call is split into launches (include/sptp.h)
VARIANTS = {"auto": 0, "pair": 1, "chain": 2, "fused": 3, "layers": 4}
# sptp_status codes
STATUS = {"ok": 0, "null": -1, "shape": -2, "dtype": -3, "workspace": -4, "cuda": -5, "timeout": -6,
          "unimplemented": -7, "alias": -8, "too_large": -9, "device": -10, "bounds": -11}
# sptp_rope_scaling: how the rotary frequencies change for longer contexts
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}
# sptp_kv_type
SPTP_KV_SAME = 0
SPTP_KV_E4M3 = 1
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsptp.so")
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_decode_binding.so")

EXPORTED_SYMBOLS = (
    "sptp_ffn_workspace_size", "sptp_ffn_forward", "dtp_ffn_stack_workspace_size",
    "dtp_ffn_stack_forward", "sptp_prologue", "sptp_gateup_swiglu", "sptp_down_proj",
    "sptp_read_device_status", "sptp_wait_selftest", "sptp_status_string", "sptp_ffn_forward_noalloc",
    "sptp_permute_ffn_neurons", "sptp_attn_qkv_workspace_size", "sptp_attn_qkv_forward",
    "sptp_quantize_rows_e4m3", "sptp_ffn_fp8_workspace_size", "sptp_ffn_forward_fp8", "sptp_gateup_swiglu_e4m3",
    "sptp_down_proj_e4m3", "sptp_prologue_e4m3", "sptp_ffn_forward_ex", "dtp_ffn_stack_forward_ex",
    "sptp_attn_qkv_forward_ex", "sptp_noalloc_read_device_status", "sptp_noalloc_wait_selftest",
    "sptp_rope_turns", "sptp_rope", "sptp_rope_append_kv", "sptp_paged_attn_workspace_size",
    "sptp_paged_attn_decode", "sptp_rope_packed", "sptp_rope_append_kv_packed", "sptp_paged_attn_decode_packed",
    "sptp_paged_attn_wait_selftest", "sptp_paged_attn_prompt_workspace_size", "sptp_paged_attn_prompt",
    "sptp_paged_attn_decode_ex", "sptp_lora_workspace_size", "sptp_lora", "sptp_lora_ex",
    "sptp_paged_attn_prompt_wait_selftest",
)

_lib = None
_fast = None  # the extension module, once it calls _lib

_P, _I, _F, _Z, _U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_ulonglong
_LL, _D = ctypes.c_longlong, ctypes.c_double
_SIGS = {
    "sptp_ffn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "sptp_ffn_forward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _Z, _P]),
    "dtp_ffn_stack_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "dtp_ffn_stack_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _Z, _P]),
    "sptp_prologue": (_I, [_P, _P, _P, _I, _I, _I, _F, _I, _P, _P, _P]),
    "sptp_gateup_swiglu": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "sptp_down_proj": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "sptp_read_device_status": (_I, [_P, _P]),
    "sptp_wait_selftest": (_I, [_P, _Z, _U64, _I, _P]),
    "sptp_status_string": (ctypes.c_char_p, [_I]),
    "sptp_ffn_forward_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P]),
    "sptp_permute_ffn_neurons": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "sptp_attn_qkv_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "sptp_attn_qkv_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _Z, _P]),
    "sptp_quantize_rows_e4m3": (_I, [_P, _LL, _I, _P, _P, _P]),
    "sptp_ffn_fp8_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sptp_ffn_forward_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z,
                                  _P]),
    "sptp_gateup_swiglu_e4m3": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "sptp_down_proj_e4m3": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "sptp_prologue_e4m3": (_I, [_P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "sptp_ffn_forward_ex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _Z, _P, _I]),
    "dtp_ffn_stack_forward_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _Z, _P, _I]),
    "sptp_attn_qkv_forward_ex": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _Z, _P, _I]),
    "sptp_noalloc_read_device_status": (_I, [_P]),
    "sptp_noalloc_wait_selftest": (_I, [_U64, _I, _P]),
    "sptp_rope_turns": (_I, [_I, _D, _I, _D, _D, _D, _D, _P]),
    "sptp_rope": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P]),
    "sptp_rope_append_kv": (_I, [_P] * 5 + [_I] * 7 + [_F] + [_I] * 6 + [_P] * 6 + [_Z, _P]),
    "sptp_rope_packed": (_I, [ctypes.c_char_p]),
    "sptp_rope_append_kv_packed": (_I, [ctypes.c_char_p]),
    "sptp_paged_attn_decode_packed": (_I, [ctypes.c_char_p]),
    "sptp_paged_attn_wait_selftest": (_I, [ctypes.c_char_p, _I, _I, _U64]),
    "sptp_paged_attn_decode_ex": (_I, [ctypes.c_char_p, _F, _P]),
    "sptp_lora_workspace_size": (_Z, [_I] * 6),
    "sptp_lora": (_I, [_P] * 5 + [_I] * 8 + [_P] * 3 + [_Z, _P]),
    "sptp_lora_ex": (_I, [_P] * 5 + [_I] * 8 + [_P] * 3 + [_Z, _P, _P, _I]),
    "sptp_paged_attn_prompt_workspace_size": (_Z, [_I] * 6),
    "sptp_paged_attn_prompt": (_I, [ctypes.c_char_p]),
    "sptp_paged_attn_prompt_wait_selftest": (_I, [ctypes.c_char_p, _I, _U64]),
    "sptp_paged_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sptp_paged_attn_decode": (_I, [_P] * 7 + [_I] * 9 + [_F, _I, _I, _P, _P, _P, _Z, _P]),
}


class SptpError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({sptp_status_string(code)})")
        self.code = code


CHECKED_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsptp_check.so")


def load_library(path: str = LIB_PATH, replace: bool = False):
    """Loads libsptp.so (built by sequence_tensor_transformer_gb300.build) on
    first use.  replace=True makes `path` the library every later call uses:
    for example CHECKED_LIB_PATH, the bounds-checked build (build(checked=True))."""
    global _lib
    if _lib is None or replace:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib_ = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            f = getattr(lib_, name)
            f.restype = res
            f.argtypes = args
        set_library(lib_)
    return _lib


def set_library(handle):
    """Makes a handle returned by load_library the one every call uses.  Where
    the extension module cannot be loaded (built for another torch or Python),
    the functions here make every call, and a warning says so."""
    global _lib, _fast
    _lib, _fast = handle, None
    if handle is None or not os.path.exists(BINDING_PATH):
        return
    importlib.invalidate_caches()  # it may have been built by this process
    try:
        _decode_binding = importlib.import_module("._decode_binding", __package__)
    except ImportError as e:
        warnings.warn(f"{BINDING_PATH} cannot be loaded ({e}): build it anew (build.build()); until then a decoding "
                      "step's calls cost some microseconds more", RuntimeWarning, stacklevel=2)
        return
    for use, names in ((_decode_binding.use, ("sptp_rope_packed", "sptp_rope_append_kv_packed", "sptp_paged_attn_decode_packed")),
                       (_decode_binding.use_batch, ("sptp_paged_attn_decode_ex", "sptp_paged_attn_prompt", "sptp_lora_ex"))):
        use(*(ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in names))
    _fast = _decode_binding


def lib():
    return load_library()


def sptp_status_string(code: int) -> str:
    return lib().sptp_status_string(int(code)).decode()


# ------------------------------------------------------------------ helpers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPTP_BF16
    if t.dtype == torch.float32:
        return SPTP_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensors only")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _expect(name, t, shape, dtype, optional=False):
    """Shape and dtype of a tensor argument, checked before any pointer is
    passed: the C ABI takes pointers and sizes only, so a tensor of the wrong
    shape would otherwise be read or written past its end."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _same_device(*ts):
    """Every tensor argument on one CUDA device, the current one: the library
    launches on the current device and takes its stream, scratch and device
    properties from it, so a tensor elsewhere would be handed to kernels of
    another device.  Checked before any pointer reaches the C ABI."""
    ts = [t for t in ts if t is not None]
    if not ts:
        return
    device = ts[0].device
    for t in ts:
        if t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}: one device expected")
    if device.type != "cuda":
        raise ValueError("device tensors only")
    cur = torch.cuda.current_device()
    if device.index != cur:
        raise ValueError(f"tensors on {device} but the current device is cuda:{cur}: "
                         f"call torch.cuda.set_device({device.index}) first")


def _variant(v) -> int:
    if isinstance(v, str):
        if v not in VARIANTS:
            raise ValueError(f"unknown variant {v!r}; one of {sorted(VARIANTS)}")
        return VARIANTS[v]
    return int(v)


def _nbytes(t) -> int:
    return t.nbytes


def _stream(stream):
    if stream is None:
        # the handle alone: building torch's stream object takes 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream on {stream.device} but the current device is cuda:{torch.cuda.current_device()}")
    return stream.cuda_stream


def _check(fn: str, code: int):
    if code != 0:
        raise SptpError(fn, code)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, SPTP_WS_HEADER_BYTES), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ entry points

def sptp_ffn_workspace_size(M, d, F, P, chunks, dtype=SPTP_BF16) -> int:
    return int(lib().sptp_ffn_workspace_size(M, d, F, P, chunks, dtype))


def dtp_ffn_stack_workspace_size(M, d, F, P, L, delta, dtype=SPTP_BF16) -> int:
    return int(lib().dtp_ffn_stack_workspace_size(M, d, F, P, L, delta, dtype))


def _check_ffn_args(x, partials, gamma, W1g, W1u, W2, P, out, resid_out, dtype=None):
    M, d = x.shape
    F = W1g.shape[0]
    dt = x.dtype if dtype is None else dtype
    _expect("partials", partials, (P, M, d), dt)
    _expect("gamma", gamma, (d,), dt)
    _expect("W1g", W1g, (F, d), dt)
    _expect("W1u", W1u, (F, d), dt)
    _expect("W2", W2, (d, F), dt)
    _expect("out", out, (P, M, d), dt, optional=True)
    _expect("resid_out", resid_out, (M, d), dt, optional=True)
    _same_device(x, partials, gamma, W1g, W1u, W2, out, resid_out)


def sptp_ffn_forward(x, partials, gamma, W1g, W1u, W2, P, chunks, eps, out=None, resid_out=None,
                     workspace=None, stream=None, write_resid=True, variant="auto"):
    """SP-TP FFN boundary.  Returns (out [P,M,d], resid_out [M,d] or None).
    variant: "auto" (the library's default), "pair", "chain" or "fused"."""
    M, d = x.shape
    F = W1g.shape[0]
    dt = _dtype_code(x)
    _check_ffn_args(x, partials, gamma, W1g, W1u, W2, P, out, resid_out)
    if out is None:
        out = torch.empty((P, M, d), dtype=x.dtype, device=x.device)
    if resid_out is None and write_resid:
        resid_out = torch.empty_like(x)
    if workspace is None:
        workspace = _workspace(sptp_ffn_workspace_size(M, d, F, P, chunks, dt), x.device)
    _same_device(x, workspace)
    code = lib().sptp_ffn_forward_ex(
        _ptr(x), _ptr(partials), _ptr(gamma), _ptr(W1g), _ptr(W1u), _ptr(W2), M, d, F, P, chunks,
        float(eps), dt, _ptr(out), _ptr(resid_out), _ptr(workspace), _nbytes(workspace), _stream(stream),
        _variant(variant))
    _check("sptp_ffn_forward", code)
    return out, resid_out


def dtp_ffn_stack_forward(x_shards, gamma, W1g, W1u, W2, P, L, delta, flush, eps, workspace=None,
                          stream=None, variant="auto"):
    """Delayed-TP stack; updates x_shards [P,M,d] in place and returns it.
    variant: "auto" (the library's default), "fused" or "layers"."""
    _, M, d = x_shards.shape
    F = W1g.shape[1]
    dt = _dtype_code(x_shards)
    _expect("x_shards", x_shards, (P, M, d), x_shards.dtype)
    _expect("gamma", gamma, (L, d), x_shards.dtype)
    _expect("W1g", W1g, (L, F, d), x_shards.dtype)
    _expect("W1u", W1u, (L, F, d), x_shards.dtype)
    _expect("W2", W2, (L, d, F), x_shards.dtype)
    if workspace is None:
        workspace = _workspace(dtp_ffn_stack_workspace_size(M, d, F, P, L, delta, dt), x_shards.device)
    _same_device(x_shards, gamma, W1g, W1u, W2, workspace)
    code = lib().dtp_ffn_stack_forward_ex(
        _ptr(x_shards), _ptr(gamma), _ptr(W1g), _ptr(W1u), _ptr(W2), M, d, F, P, L, delta, int(flush),
        float(eps), dt, _ptr(workspace), _nbytes(workspace), _stream(stream), _variant(variant))
    _check("dtp_ffn_stack_forward", code)
    return x_shards


def sptp_prologue(x, partials, gamma, eps, h_out=None, y_out=None, stream=None, write_h=True):
    M, d = x.shape
    P = partials.shape[0]
    _expect("partials", partials, (P, M, d), x.dtype)
    _expect("gamma", gamma, (d,), x.dtype)
    _expect("h_out", h_out, (M, d), x.dtype, optional=True)
    _expect("y_out", y_out, (M, d), x.dtype, optional=True)
    _same_device(x, partials, gamma, h_out, y_out)
    if y_out is None:
        y_out = torch.empty_like(x)
    if h_out is None and write_h:
        h_out = torch.empty_like(x)
    code = lib().sptp_prologue(_ptr(x), _ptr(partials), _ptr(gamma), M, d, P, float(eps), _dtype_code(x),
                               _ptr(h_out), _ptr(y_out), _stream(stream))
    _check("sptp_prologue", code)
    return h_out, y_out


def sptp_gateup_swiglu(y, W1g, W1u, P, s_out=None, workspace=None, stream=None):
    M, d = y.shape
    F = W1g.shape[0]
    _expect("W1g", W1g, (F, d), y.dtype)
    _expect("W1u", W1u, (F, d), y.dtype)
    _expect("s_out", s_out, (P, M, F // P), y.dtype, optional=True)
    if s_out is None:
        s_out = torch.empty((P, M, F // P), dtype=y.dtype, device=y.device)
    if workspace is None:
        workspace = _workspace(SPTP_WS_HEADER_BYTES, y.device)
    _same_device(y, W1g, W1u, s_out, workspace)
    code = lib().sptp_gateup_swiglu(_ptr(y), _ptr(W1g), _ptr(W1u), M, d, F, P, _dtype_code(y), _ptr(s_out),
                                    _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check("sptp_gateup_swiglu", code)
    return s_out


def sptp_down_proj(s, W2, P, out=None, workspace=None, stream=None, adapters=None, adapter_workspace=None):
    """Row-parallel projection of every shard: out [P,M,d] from s [P,M,F/P].  adapters:
    (A, B, ids, gains) as in sptp_lora, added to out in place.  adapter_workspace: that
    call's, with its status; left out, an id outside its range is recorded in workspace."""
    _, M, f = s.shape
    d, F = W2.shape
    _expect("s", s, (P, M, F // P), s.dtype)
    _expect("out", out, (P, M, d), s.dtype, optional=True)
    _expect("W2", W2, (d, F), s.dtype)
    if out is None:
        out = torch.empty((P, M, d), dtype=s.dtype, device=s.device)
    if workspace is None:
        workspace = _workspace(SPTP_WS_HEADER_BYTES, s.device)
    _same_device(s, W2, out, workspace)
    beside = None if adapters is None else _adapters_beside(s, adapters, out, workspace, adapter_workspace, stream)
    code = lib().sptp_down_proj(_ptr(s), _ptr(W2), M, d, F, P, _dtype_code(s), _ptr(out), _ptr(workspace),
                                _nbytes(workspace), _stream(stream))
    _check("sptp_down_proj", code)
    if beside is not None:
        _lora_beside(beside, stream)
    return out


def sptp_ffn_forward_noalloc(x, partials, gamma, W1g, W1u, W2, P, chunks, eps, out, resid_out=None,
                             stream=None):
    """SP-TP FFN boundary on the library's static scratch (no workspace and no
    device allocation inside the call; the caller passes out/resid_out)."""
    M, d = x.shape
    F = W1g.shape[0]
    _expect("out", out, (P, M, d), x.dtype)
    _check_ffn_args(x, partials, gamma, W1g, W1u, W2, P, out, resid_out)
    code = lib().sptp_ffn_forward_noalloc(
        _ptr(x), _ptr(partials), _ptr(gamma), _ptr(W1g), _ptr(W1u), _ptr(W2), M, d, F, P, chunks, float(eps),
        _dtype_code(x), _ptr(out), _ptr(resid_out), _stream(stream))
    _check("sptp_ffn_forward_noalloc", code)
    return out, resid_out


def sptp_noalloc_read_device_status(stream=None) -> int:
    """Status words of the last no-allocation forward on the current device."""
    return int(lib().sptp_noalloc_read_device_status(_stream(stream)))


def sptp_noalloc_wait_selftest(limit_ns: int, preset_flag: bool, stream=None) -> int:
    return int(lib().sptp_noalloc_wait_selftest(int(limit_ns), int(preset_flag), _stream(stream)))


def sptp_attn_qkv_workspace_size(M, d, N, P, chunks, dtype=SPTP_BF16) -> int:
    return int(lib().sptp_attn_qkv_workspace_size(M, d, N, P, chunks, dtype))


def sptp_attn_qkv_forward(x, partials, gamma, Wqkv, P, chunks, eps, qkv_out=None, resid_out=None,
                          workspace=None, stream=None, write_resid=True, variant="auto", adapters=None,
                          adapter_workspace=None):
    """Boundary in front of attention: returns (qkv [P,M,N/P], resid_out).
    variant: "auto" (the library's default), "pair" or "fused".  adapters: (A, B,
    ids, gains) as in sptp_lora, added to qkv in place (sptp_lora on the normed rows
    in the workspace).  adapter_workspace: that call's, with its status; left out, an
    id outside its range is recorded in workspace."""
    M, d = x.shape
    N = Wqkv.shape[0]
    dt = _dtype_code(x)
    _expect("partials", partials, (P, M, d), x.dtype)
    _expect("gamma", gamma, (d,), x.dtype)
    _expect("Wqkv", Wqkv, (N, d), x.dtype)
    _expect("qkv_out", qkv_out, (P, M, N // P), x.dtype, optional=True)
    _expect("resid_out", resid_out, (M, d), x.dtype, optional=True)
    _same_device(x, partials, gamma, Wqkv, qkv_out, resid_out, workspace)
    if qkv_out is None:
        qkv_out = torch.empty((P, M, N // P), dtype=x.dtype, device=x.device)
    if resid_out is None and write_resid:
        resid_out = torch.empty_like(x)
    if workspace is None:
        workspace = _workspace(sptp_attn_qkv_workspace_size(M, d, N, P, chunks, dt), x.device)
    beside = None
    if adapters is not None:
        # the normed rows, behind the workspace's header
        _ptr(workspace)  # (dense)
        rows = workspace.view(-1).view(torch.uint8)[SPTP_WS_HEADER_BYTES:SPTP_WS_HEADER_BYTES + x.nbytes]
        if rows.nbytes < x.nbytes:
            raise SptpError("sptp_attn_qkv_forward", STATUS["workspace"])
        beside = _adapters_beside(rows.view(x.dtype).view(M, d), adapters, qkv_out, workspace, adapter_workspace, stream)
    code = lib().sptp_attn_qkv_forward_ex(_ptr(x), _ptr(partials), _ptr(gamma), _ptr(Wqkv), M, d, N, P, chunks,
                                          float(eps), dt, _ptr(qkv_out), _ptr(resid_out), _ptr(workspace),
                                          _nbytes(workspace), _stream(stream), _variant(variant))
    _check("sptp_attn_qkv_forward", code)
    if beside is not None:
        _lora_beside(beside, stream)
    return qkv_out, resid_out


def sptp_permute_ffn_neurons(W1g, W1u, W2, perm, workspace=None, stream=None):
    """Renumbers every module's neurons (W1g/W1u [L,F,d] rows, W2 [L,d,F]
    columns) by perm [L,F] (int32, device); returns the permuted copies."""
    L, F, d = W1g.shape
    _expect("W1u", W1u, (L, F, d), W1g.dtype)
    _expect("W2", W2, (L, d, F), W1g.dtype)
    _expect("perm", perm, (L, F), torch.int32)
    if workspace is None:
        workspace = _workspace(SPTP_WS_HEADER_BYTES, W1g.device)
    _same_device(W1g, W1u, W2, perm, workspace)
    outs = [torch.empty_like(W1g), torch.empty_like(W1u), torch.empty_like(W2)]
    code = lib().sptp_permute_ffn_neurons(_ptr(W1g), _ptr(W1u), _ptr(W2), _ptr(perm), L, d, F, _dtype_code(W1g),
                                          _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(workspace),
                                          _nbytes(workspace), _stream(stream))
    _check("sptp_permute_ffn_neurons", code)
    return tuple(outs)


def sptp_read_device_status(workspace, stream=None) -> int:
    _same_device(workspace)
    return int(lib().sptp_read_device_status(_ptr(workspace), _stream(stream)))


def sptp_wait_selftest(workspace, limit_ns: int, preset_flag: bool, stream=None) -> int:
    _same_device(workspace)
    return int(lib().sptp_wait_selftest(_ptr(workspace), _nbytes(workspace), int(limit_ns), int(preset_flag),
                                        _stream(stream)))


# ------------------------------------------------------------------ fp8 (E4M3)

def sptp_quantize_rows_e4m3(a, q=None, scale=None, stream=None):
    """Row-wise E4M3 quantisation of a bf16 tensor viewed as [R][K] (K = the
    last dimension).  Returns (q uint8 [..., K], scale float32 [...]):
    a ~= q * scale[..., None] with scale a power of two per row."""
    if a.dtype != torch.bfloat16:
        raise TypeError("bf16 input expected")
    K = a.shape[-1]
    R = a.numel() // K if K else 0
    _expect("q", q, tuple(a.shape), torch.uint8, optional=True)
    _expect("scale", scale, tuple(a.shape[:-1]), torch.float32, optional=True)
    _same_device(a, q, scale)
    if q is None:
        q = torch.empty(a.shape, dtype=torch.uint8, device=a.device)
    if scale is None:
        scale = torch.empty(a.shape[:-1], dtype=torch.float32, device=a.device)
    code = lib().sptp_quantize_rows_e4m3(_ptr(a), R, K, _ptr(q), _ptr(scale), _stream(stream))
    _check("sptp_quantize_rows_e4m3", code)
    return q, scale


def quantize_ffn_weights_e4m3(W1g, W1u, W2, P, stream=None):
    """The fp8 weights of one FFN in the layout sptp_ffn_forward_fp8 takes:
    (qW1g, sW1g [F], qW1u, sW1u [F], qW2 [d,F], sW2 [d,P]); W2 is quantised as
    [d*P][F/P] rows, one scale per output feature and shard."""
    d, F = W2.shape
    _expect("W1g", W1g, (F, d), torch.bfloat16)
    _expect("W1u", W1u, (F, d), torch.bfloat16)
    if F % P != 0:
        raise ValueError(f"F = {F} is not a multiple of P = {P}")
    qg, sg = sptp_quantize_rows_e4m3(W1g, stream=stream)
    qu, su = sptp_quantize_rows_e4m3(W1u, stream=stream)
    q2, s2 = sptp_quantize_rows_e4m3(W2.view(d, P, F // P), stream=stream)
    return qg, sg, qu, su, q2.view(d, F), s2


def sptp_ffn_fp8_workspace_size(M, d, F, P, chunks) -> int:
    return int(lib().sptp_ffn_fp8_workspace_size(M, d, F, P, chunks))


def sptp_ffn_forward_fp8(x, partials, gamma, qweights, P, chunks, eps, out=None, resid_out=None, workspace=None,
                         stream=None, write_resid=True):
    """SP-TP FFN boundary with E4M3 linear layers; qweights as returned by
    quantize_ffn_weights_e4m3.  Returns (out [P,M,d], resid_out [M,d] or None)."""
    qg, sg, qu, su, q2, s2 = qweights
    M, d = x.shape
    F = qg.shape[0]
    bf = torch.bfloat16
    _expect("x", x, (M, d), bf)
    _expect("partials", partials, (P, M, d), bf)
    _expect("gamma", gamma, (d,), bf)
    for name, t, shape, dt in (("qW1g", qg, (F, d), torch.uint8), ("sW1g", sg, (F,), torch.float32),
                               ("qW1u", qu, (F, d), torch.uint8), ("sW1u", su, (F,), torch.float32),
                               ("qW2", q2, (d, F), torch.uint8), ("sW2", s2, (d, P), torch.float32)):
        _expect(name, t, shape, dt)
    _expect("out", out, (P, M, d), bf, optional=True)
    _expect("resid_out", resid_out, (M, d), bf, optional=True)
    _same_device(x, partials, gamma, qg, sg, qu, su, q2, s2, out, resid_out, workspace)
    if out is None:
        out = torch.empty((P, M, d), dtype=x.dtype, device=x.device)
    if resid_out is None and write_resid:
        resid_out = torch.empty_like(x)
    if workspace is None:
        workspace = _workspace(sptp_ffn_fp8_workspace_size(M, d, F, P, chunks), x.device)
    code = lib().sptp_ffn_forward_fp8(
        _ptr(x), _ptr(partials), _ptr(gamma), _ptr(qg), _ptr(sg), _ptr(qu), _ptr(su), _ptr(q2), _ptr(s2), M, d, F,
        P, chunks, float(eps), _ptr(out), _ptr(resid_out), _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check("sptp_ffn_forward_fp8", code)
    return out, resid_out


def sptp_prologue_e4m3(x, partials, gamma, eps, h_out=None, y_work=None, q_out=None, scale_out=None, stream=None,
                       write_h=True):
    """Partial sum + residual + RMSNorm with y quantised to E4M3 in the same
    launch.  Returns (h or None, q uint8 [M,d], scale float32 [M])."""
    M, d = x.shape
    P = partials.shape[0]
    bf = torch.bfloat16
    _expect("x", x, (M, d), bf)
    _expect("partials", partials, (P, M, d), bf)
    _expect("gamma", gamma, (d,), bf)
    _expect("h_out", h_out, (M, d), bf, optional=True)
    _expect("y_work", y_work, (M, d), bf, optional=True)
    _expect("q_out", q_out, (M, d), torch.uint8, optional=True)
    _expect("scale_out", scale_out, (M,), torch.float32, optional=True)
    _same_device(x, partials, gamma, h_out, y_work, q_out, scale_out)
    if h_out is None and write_h:
        h_out = torch.empty_like(x)
    if y_work is None:
        y_work = torch.empty_like(x)
    if q_out is None:
        q_out = torch.empty((M, d), dtype=torch.uint8, device=x.device)
    if scale_out is None:
        scale_out = torch.empty((M,), dtype=torch.float32, device=x.device)
    code = lib().sptp_prologue_e4m3(_ptr(x), _ptr(partials), _ptr(gamma), M, d, P, float(eps), _ptr(h_out),
                                    _ptr(y_work), _ptr(q_out), _ptr(scale_out), _stream(stream))
    _check("sptp_prologue_e4m3", code)
    return h_out, q_out, scale_out


def sptp_gateup_swiglu_e4m3(qy, sy, qW1g, sW1g, qW1u, sW1u, P, s_out=None, workspace=None, stream=None):
    M, d = qy.shape
    F = qW1g.shape[0]
    for name, t, shape, dt in (("qy", qy, (M, d), torch.uint8), ("sy", sy, (M,), torch.float32),
                               ("qW1g", qW1g, (F, d), torch.uint8), ("sW1g", sW1g, (F,), torch.float32),
                               ("qW1u", qW1u, (F, d), torch.uint8), ("sW1u", sW1u, (F,), torch.float32)):
        _expect(name, t, shape, dt)
    _expect("s_out", s_out, (P, M, F // P), torch.bfloat16, optional=True)
    _same_device(qy, sy, qW1g, sW1g, qW1u, sW1u, s_out, workspace)
    if s_out is None:
        s_out = torch.empty((P, M, F // P), dtype=torch.bfloat16, device=qy.device)
    if workspace is None:
        workspace = _workspace(SPTP_WS_HEADER_BYTES, qy.device)
    code = lib().sptp_gateup_swiglu_e4m3(_ptr(qy), _ptr(sy), _ptr(qW1g), _ptr(sW1g), _ptr(qW1u), _ptr(sW1u), M, d,
                                         F, P, _ptr(s_out), _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check("sptp_gateup_swiglu_e4m3", code)
    return s_out


def sptp_down_proj_e4m3(qs, ss, qW2, sW2, P, out=None, workspace=None, stream=None):
    _, M, f = qs.shape
    d, F = qW2.shape
    for name, t, shape, dt in (("qs", qs, (P, M, F // P), torch.uint8), ("ss", ss, (P, M), torch.float32),
                               ("qW2", qW2, (d, F), torch.uint8), ("sW2", sW2, (d, P), torch.float32)):
        _expect(name, t, shape, dt)
    _expect("out", out, (P, M, d), torch.bfloat16, optional=True)
    _same_device(qs, ss, qW2, sW2, out, workspace)
    if out is None:
        out = torch.empty((P, M, d), dtype=torch.bfloat16, device=qs.device)
    if workspace is None:
        workspace = _workspace(SPTP_WS_HEADER_BYTES, qs.device)
    code = lib().sptp_down_proj_e4m3(_ptr(qs), _ptr(ss), _ptr(qW2), _ptr(sW2), M, d, F, P, _ptr(out),
                                     _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check("sptp_down_proj_e4m3", code)
    return out


# ------------------------------------------------------------------ rotary positions, paged key-value cache

def sptp_rope_turns(rot, theta=10000.0, scaling="none", factor=1.0, orig_len=0, alpha=1.0, beta=32.0, device=None):
    """The rotation's frequency table, made once per model: int64 [rot/2] on
    `device` (the current CUDA device if None), turns per position as 64-bit
    binary fractions.  scaling: "none", "linear", "ntk" or "parts"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}; one of {sorted(ROPE_SCALINGS)}")
    turns = torch.empty(max(int(rot) // 2, 0), dtype=torch.int64)
    code = lib().sptp_rope_turns(int(rot), float(theta), ROPE_SCALINGS[scaling], float(factor), float(orig_len),
                                 float(alpha), float(beta), turns.data_ptr())
    _check("sptp_rope_turns", code)
    return turns.to(torch.device("cuda", torch.cuda.current_device()) if device is None else device)


def sptp_rope(x, positions, turns, Hr=None, interleaved=False, transpose=False, gain=1.0, out=None, stream=None):
    """Rotary positions of the first Hr (default: all) heads of x [P,M,H,D];
    positions int32 [M]; turns from sptp_rope_turns.  transpose: the gradient.
    out may be x (in place).  Returns out."""
    if _fast is not None and stream is None:
        done = _fast.rope(x, positions, turns, Hr, interleaved, transpose, gain, out)
        if done is not NotImplemented:
            return done
    P, M, H, D = x.shape
    pairs, dtype = turns.shape[0], x.dtype
    dt = _dtype_code(x)
    if not (positions.shape == (M,) and positions.dtype is torch.int32 and turns.dtype is torch.int64 and turns.dim() == 1
            and (out is None or (out.shape == (P, M, H, D) and out.dtype is dtype))):
        _expect("positions", positions, (M,), torch.int32)
        _expect("turns", turns, (pairs,), torch.int64)
        _expect("out", out, (P, M, H, D), dtype, optional=True)
    cur = _ready(x, positions, turns, out)
    if out is None:
        out = _new((P, M, H, D), dtype, x.device, stream)
    code = lib().sptp_rope_packed(_ROPE_ARGS.pack(
        x.data_ptr(), positions.data_ptr(), turns.data_ptr(), out.data_ptr(), _raw_stream(stream, cur), P, M, H,
        H if Hr is None else Hr, D, 2 * pairs, interleaved, transpose, dt, gain))
    _check("sptp_rope", code)
    return out


def paged_kv_cache(P, num_pages, Hkv, page_size, D, dtype=torch.bfloat16, e4m3=False, device="cuda"):
    """An empty paged key-value cache (k, v, k_scale, v_scale): k and v
    [P,num_pages,Hkv,page_size,D] of `dtype`, or with e4m3 uint8 codes with
    fp32 scales [P,num_pages,Hkv,page_size] (None otherwise)."""
    shape = (P, num_pages, Hkv, page_size, D)
    k, v = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else dtype, device=device) for _ in range(2))
    if not e4m3:
        return k, v, None, None
    return k, v, torch.zeros(shape[:-1], device=device), torch.zeros(shape[:-1], device=device)


# The calls of a decoding step last a few microseconds on the device.  With a
# workspace (or none needed) and stream left out they go through the extension
# module; what it does not take comes here, to the same checks, which are written
# to cost little: one condition over all tensors on the way in, those with
# messages (_expect, _same_device) only if it fails.

# The arguments of a call as one block (the *_args structs of include/sptp.h):
# pointers, sizes, ints and the float in the structs' order and native layout.
_ROPE_ARGS = struct.Struct("@5P9if")
_APPEND_ARGS = struct.Struct("@12PN13if")
_DECODE_ARGS = struct.Struct("@11PN11if")
_PROMPT_ARGS = struct.Struct("@14PN12i2f")


def _ready(*ts):
    """Every tensor given is dense and on the current CUDA device, whose index
    is returned."""
    cur = torch._C._cuda_getDevice() if ts[0].is_cuda else -1
    for t in ts:
        if t is not None and (cur < 0 or t.get_device() != cur or not t.is_contiguous()):
            _same_device(*ts)
            raise ValueError("tensors must be contiguous")
    return cur


def _raw_stream(stream, device_index):
    return torch._C._cuda_getCurrentRawStream(device_index) if stream is None else _stream(stream)


def _new(shape, dtype, device, stream):
    """An output or a workspace that the caller left out.  Memory from the
    allocator is ordered by the stream it is asked for on: the call's own."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check_cache(cache, P, D, dtype):
    """Sizes (num_pages, Hkv, page_size, kv_type) of a cache of activations of `dtype`."""
    k, v, ks, vs = cache
    shape, kvt = k.shape, k.dtype
    if len(shape) != 5:
        raise ValueError(f"cache: {len(shape)} dimensions, expected [P,num_pages,Hkv,page_size,D]")
    if v.shape == shape and v.dtype is kvt and shape[0] == P and shape[4] == D:
        if ks is None and vs is None and kvt is dtype:
            return shape[1], shape[2], shape[3], SPTP_KV_SAME
        if (kvt is torch.uint8 and dtype is torch.bfloat16 and ks is not None and vs is not None
                and ks.shape == vs.shape == shape[:4] and ks.dtype is vs.dtype is torch.float32):
            return shape[1], shape[2], shape[3], SPTP_KV_E4M3
    if kvt != dtype:
        if kvt != torch.uint8:
            raise TypeError(f"cache: dtype {kvt}, expected {dtype} or uint8 codes")
        if dtype != torch.bfloat16:
            raise TypeError("an E4M3 cache takes bf16 activations")
    want = (P, *shape[1:4], D)
    _expect("k_cache", k, want, kvt)
    _expect("v_cache", v, want, kvt)
    if kvt == dtype:
        raise ValueError("scales belong to an E4M3 cache")
    _expect("k_scale", ks, want[:-1], torch.float32)
    _expect("v_scale", vs, want[:-1], torch.float32)
    return shape[1], shape[2], shape[3], SPTP_KV_E4M3


def sptp_rope_append_kv(qkv, positions, seq_ids, page_table, turns, cache, Hq, interleaved=False, gain=1.0, q_out=None,
                        workspace=None, stream=None):
    """Rotates the q and k heads of qkv [P,M,(Hq+2Hkv)D] and stores k and v in
    `cache` (see paged_kv_cache).  positions, seq_ids int32 [M] (seq_ids < 0:
    padding, whose rows of q_out are left as they are: undefined in one that is
    left out); page_table int32 [B,max_pages]; turns None: no rotation.  Returns
    q_out [P,M,Hq,D].  Costs the host less with a workspace given and stream left
    out."""
    if _fast is not None and stream is None:
        done = _fast.append(qkv, positions, seq_ids, page_table, turns, cache, Hq, interleaved, gain, q_out, workspace)
        if done is not NotImplemented:
            return done
    P, M, N = qkv.shape
    k, v, ks, vs = cache
    D, dtype, i32 = k.shape[-1], qkv.dtype, torch.int32
    dt = _dtype_code(qkv)
    num_pages, Hkv, page_size, kv_type = _check_cache(cache, P, D, dtype)
    B, max_pages = page_table.shape
    pairs = 0 if turns is None else turns.shape[0]
    if not (N == (Hq + 2 * Hkv) * D and positions.shape == (M,) and positions.dtype is i32 and seq_ids.shape == (M,)
            and seq_ids.dtype is i32 and page_table.dtype is i32
            and (turns is None or (turns.dtype is torch.int64 and turns.dim() == 1))
            and (q_out is None or (q_out.shape == (P, M, Hq, D) and q_out.dtype is dtype))):
        _expect("qkv", qkv, (P, M, (Hq + 2 * Hkv) * D), dtype)
        _expect("positions", positions, (M,), i32)
        _expect("seq_ids", seq_ids, (M,), i32)
        _expect("page_table", page_table, (B, max_pages), i32)
        _expect("turns", turns, (pairs,), torch.int64, optional=True)
        _expect("q_out", q_out, (P, M, Hq, D), dtype, optional=True)
    cur = _ready(qkv, positions, seq_ids, page_table, turns, k, v, ks, vs, q_out, workspace)
    if q_out is None:
        q_out = _new((P, M, Hq, D), dtype, qkv.device, stream)
    if workspace is None:
        workspace = _new((SPTP_WS_HEADER_BYTES,), torch.uint8, qkv.device, stream)
    code = lib().sptp_rope_append_kv_packed(_APPEND_ARGS.pack(
        qkv.data_ptr(), positions.data_ptr(), seq_ids.data_ptr(), page_table.data_ptr(),
        0 if turns is None else turns.data_ptr(), q_out.data_ptr(), k.data_ptr(), v.data_ptr(),
        0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(), workspace.data_ptr(),
        _raw_stream(stream, cur), workspace.nbytes, P, M, Hq, Hkv, D, 2 * pairs, interleaved, B, max_pages, num_pages,
        page_size, dt, kv_type, gain))
    _check("sptp_rope_append_kv", code)
    return q_out


def sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D) -> int:
    return int(lib().sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D))


def sptp_paged_attn_decode(q, cache, page_table, seq_lens, scale=None, window=0, out=None, lse=None, workspace=None,
                           stream=None, write_lse=True, cap=0.0, slopes=None):
    """Attention of one token per sequence over a paged cache: q [P,B,Hq,D],
    page_table int32 [B,max_pages], seq_lens int32 [B] (0: an empty row);
    scale defaults to D^-1/2; window 0: the whole sequence.  cap and slopes:
    scores as in sptp_paged_attn_prompt.  Returns (out [P,B,Hq*D], lse fp32
    [P,B,Hq] or None).  Costs the host less with a workspace given and stream
    left out."""
    if _fast is not None and stream is None:
        if slopes is None and isinstance(cap, (int, float)) and cap == 0:
            done = _fast.decode(q, cache, page_table, seq_lens, scale, window, out, lse, workspace, write_lse)
        else:
            done = _fast.decode_ex(q, cache, page_table, seq_lens, scale, window, out, lse, workspace, write_lse, cap, slopes)
        if done is not NotImplemented:
            return done
    _check_cap("sptp_paged_attn_decode", cap)
    P, B, Hq, D = q.shape
    k, v, ks, vs = cache
    dtype, i32 = q.dtype, torch.int32
    dt = _dtype_code(q)
    num_pages, Hkv, page_size, kv_type = _check_cache(cache, P, D, dtype)
    max_pages = page_table.shape[-1]
    if not (page_table.shape == (B, max_pages) and page_table.dtype is i32 and seq_lens.shape == (B,)
            and seq_lens.dtype is i32 and (out is None or (out.shape == (P, B, Hq * D) and out.dtype is dtype))
            and (lse is None or (lse.shape == (P, B, Hq) and lse.dtype is torch.float32))):
        _expect("page_table", page_table, (B, max_pages), i32)
        _expect("seq_lens", seq_lens, (B,), i32)
        _expect("out", out, (P, B, Hq * D), dtype, optional=True)
        _expect("lse", lse, (P, B, Hq), torch.float32, optional=True)
    _expect("slopes", slopes, (P, Hq), torch.float32, optional=True)
    cur = _ready(q, k, v, ks, vs, page_table, seq_lens, slopes, out, lse, workspace)
    if out is None:
        out = _new((P, B, Hq * D), dtype, q.device, stream)
    if lse is None and write_lse:
        lse = _new((P, B, Hq), torch.float32, q.device, stream)
    if workspace is None:
        n = max(sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D), SPTP_WS_HEADER_BYTES)
        workspace = _new((n,), torch.uint8, q.device, stream)
    code = lib().sptp_paged_attn_decode_ex(_DECODE_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(),
        page_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        workspace.data_ptr(), _raw_stream(stream, cur), workspace.nbytes, P, B, Hq, Hkv, D, max_pages, num_pages,
        page_size, window, dt, kv_type, D ** -0.5 if scale is None else scale), cap, None if slopes is None else slopes.data_ptr())
    _check("sptp_paged_attn_decode", code)
    return out, lse


def _check_cap(fn, cap):
    """A cap too small for fp32 is refused like any below 1e-30 (it would be passed as 0: none)."""
    if cap != 0 and abs(cap) < 1e-30:
        raise SptpError(fn, STATUS["shape"])


def sptp_paged_attn_prompt_workspace_size(P, M, B, Hq, Hkv, D) -> int:
    return int(lib().sptp_paged_attn_prompt_workspace_size(P, M, B, Hq, Hkv, D))


def sptp_paged_attn_prompt(q, cache, page_table, seq_lens, row_starts, scale=None, window=0, cap=0.0, slopes=None,
                           prefix_lens=None, out=None, lse=None, workspace=None, stream=None, write_lse=True):
    """Attention of many new rows per sequence over a paged cache: q [P,M,Hq,D],
    the rows of B sequences packed, sequence b's from row_starts[b] to
    row_starts[b+1] (int32 [B+1]); page_table int32 [B,max_pages]; seq_lens int32
    [B], the new rows' keys included.  A row at position pos sees its sequence's
    keys up to pos, or up to prefix_lens[b] (int32 [B]) where that is more, from
    pos + 1 - window on if window is not 0.  Scores: cap tanh(scale q.k / cap) (cap 0:
    none) - slopes[head] |pos - key| (slopes fp32 [P,Hq]); scale defaults to
    D^-1/2.  Rows of no sequence are left as they are (undefined in an output
    that is left out).  Returns (out [P,M,Hq*D], lse fp32 [P,M,Hq] or None).
    Costs the host less with a workspace given and stream left out."""
    if _fast is not None and stream is None:
        done = _fast.prompt(q, cache, page_table, seq_lens, row_starts, scale, window, cap, slopes, prefix_lens, out, lse,
                            workspace, write_lse)
        if done is not NotImplemented:
            return done
    args, out, lse, workspace = _prompt_call(q, cache, page_table, seq_lens, row_starts, scale, window, cap, slopes, prefix_lens,
                                             out, lse, workspace, stream, write_lse)
    _check("sptp_paged_attn_prompt", lib().sptp_paged_attn_prompt(args))
    return out, lse


def sptp_paged_attn_prompt_wait_selftest(q, cache, page_table, seq_lens, row_starts, out, workspace, withhold_full,
                                         limit_ns=20_000_000):
    """sptp_paged_attn_prompt on two CTAs, the first of which never loads a tile of its
    share, so that its bounded waits run out (SPTP_ERR_TIMEOUT in the workspace's
    status words)."""
    args = _prompt_call(q, cache, page_table, seq_lens, row_starts, None, 0, 0.0, None, None, out, None, workspace, None,
                        False)[0]
    _check("sptp_paged_attn_prompt_wait_selftest",
           lib().sptp_paged_attn_prompt_wait_selftest(args, int(withhold_full), int(limit_ns)))


def _prompt_call(q, cache, page_table, seq_lens, row_starts, scale, window, cap, slopes, prefix_lens, out, lse, workspace,
                 stream, write_lse):
    """The checked arguments of a call as one block, its out and its lse, and the
    workspace (to be kept until the call is made)."""
    _check_cap("sptp_paged_attn_prompt", cap)
    P, M, Hq, D = q.shape
    k, v, ks, vs = cache
    dtype, i32 = q.dtype, torch.int32
    dt = _dtype_code(q)
    num_pages, Hkv, page_size, kv_type = _check_cache(cache, P, D, dtype)
    B, max_pages = page_table.shape
    if not (page_table.dtype is i32 and seq_lens.shape == (B,) and seq_lens.dtype is i32 and row_starts.shape == (B + 1,)
            and row_starts.dtype is i32 and (out is None or (out.shape == (P, M, Hq * D) and out.dtype is dtype))
            and (lse is None or (lse.shape == (P, M, Hq) and lse.dtype is torch.float32))):
        _expect("page_table", page_table, (B, max_pages), i32)
        _expect("seq_lens", seq_lens, (B,), i32)
        _expect("row_starts", row_starts, (B + 1,), i32)
        _expect("out", out, (P, M, Hq * D), dtype, optional=True)
        _expect("lse", lse, (P, M, Hq), torch.float32, optional=True)
    _expect("slopes", slopes, (P, Hq), torch.float32, optional=True)
    _expect("prefix_lens", prefix_lens, (B,), i32, optional=True)
    cur = _ready(q, k, v, ks, vs, page_table, seq_lens, row_starts, prefix_lens, slopes, out, lse, workspace)
    if out is None:
        out = _new((P, M, Hq * D), dtype, q.device, stream)
    if lse is None and write_lse:
        lse = _new((P, M, Hq), torch.float32, q.device, stream)
    if workspace is None:
        n = max(sptp_paged_attn_prompt_workspace_size(P, M, B, Hq, Hkv, D), SPTP_WS_HEADER_BYTES)
        workspace = _new((n,), torch.uint8, q.device, stream)
    args = _PROMPT_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(),
        page_table.data_ptr(), seq_lens.data_ptr(), row_starts.data_ptr(), 0 if prefix_lens is None else prefix_lens.data_ptr(),
        0 if slopes is None else slopes.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        workspace.data_ptr(), _raw_stream(stream, cur), workspace.nbytes, P, M, B, Hq, Hkv, D, max_pages, num_pages,
        page_size, window, dt, kv_type, D ** -0.5 if scale is None else scale, cap)
    return args, out, lse, workspace


def sptp_paged_attn_wait_selftest(q, cache, page_table, seq_lens, out, workspace, withhold_full=-1, withhold_empty=-1,
                                  limit_ns=20_000_000):
    """The attention (scale 1) on two CTAs with an arrival withheld in the first,
    so that its bounded waits run out (SPTP_ERR_TIMEOUT in the workspace's
    status words)."""
    P, B, Hq, D = q.shape
    k, v, ks, vs = cache
    dt = _dtype_code(q)
    num_pages, Hkv, page_size, kv_type = _check_cache(cache, P, D, q.dtype)
    max_pages = page_table.shape[-1]
    _expect("page_table", page_table, (B, max_pages), torch.int32)
    _expect("seq_lens", seq_lens, (B,), torch.int32)
    _expect("out", out, (P, B, Hq * D), q.dtype)
    cur = _ready(q, k, v, ks, vs, page_table, seq_lens, out, workspace)
    code = lib().sptp_paged_attn_wait_selftest(_DECODE_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(),
        page_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), 0, workspace.data_ptr(), _raw_stream(None, cur),
        workspace.nbytes, P, B, Hq, Hkv, D, max_pages, num_pages, page_size, 0, dt, kv_type, 1.0), int(withhold_full),
        int(withhold_empty), int(limit_ns))
    _check("sptp_paged_attn_wait_selftest", code)


# ------------------------------------------------------------------ low-rank adapters

def sptp_lora_workspace_size(P, M, K, N, R, rowwise=False) -> int:
    return int(lib().sptp_lora_workspace_size(P, M, K, N, R, int(rowwise)))


def sptp_lora(x, A, B, ids, base, gains=None, out=None, workspace=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection:
    out[p][m] = base[p][m] + gains[a] B[a] (A[a] x_m), a = ids[m] (int32 [M], < 0:
    none).  A [adapters,R,K], B [adapters,N,R], gains fp32 [adapters] or None.
    x [M,K] with base [P,M,N/P]: beside a column-parallel projection; x [P,M,K/P]
    with base [P,M,N]: beside a row-parallel one.  out may be base (in place).
    Returns out.  Costs the host less with a workspace given and stream left out."""
    if _fast is not None and stream is None:
        done = _fast.lora(x, A, B, ids, base, gains, out, workspace, None, False)
        if done is not NotImplemented:
            return done
    args, out, workspace = _lora_call(x, A, B, ids, base, gains, out, workspace, stream)
    _check("sptp_lora", lib().sptp_lora(*args))
    return out


def _adapters_beside(x, adapters, out, workspace, adapter_workspace, stream):
    """The adapters of a projection that is about to be enqueued into `out`: their call, to be
    made by _lora_beside behind it.  What is wrong with it is raised here, before anything is
    enqueued."""
    A, B, ids, gains = adapters
    status = None if adapter_workspace is not None else workspace
    if adapter_workspace is None and A.dim() == 3 and B.dim() == 3:
        n = sptp_lora_workspace_size(out.shape[0], x.shape[-2], A.shape[2], B.shape[1], A.shape[1], x.dim() == 3)
        adapter_workspace = _new((max(n, SPTP_WS_HEADER_BYTES),), torch.uint8, x.device, stream)
    call = (x, A, B, ids, out, gains, out, adapter_workspace, status)
    _lora_beside(call, stream, check_only=True)
    return call


def _lora_beside(call, stream, check_only=False):
    if _fast is not None and stream is None and _fast.lora(*call, check_only) is not NotImplemented:
        return
    *arguments, status = call
    args = _lora_call(*arguments, stream)[0]
    _check("sptp_lora", lib().sptp_lora_ex(*args, None if status is None else status.data_ptr(), int(check_only)))


def _lora_call(x, A, B, ids, base, gains, out, workspace, stream):
    """The checked arguments of a call, its out, and the workspace (to be kept until the
    call is made)."""
    n, R, K = A.shape
    N, dtype = B.shape[1], x.dtype
    dt = _dtype_code(x)
    rowwise = x.dim() == 3
    P, M = base.shape[0], x.shape[-2]
    if P < 1 or (K if rowwise else N) % P != 0:
        raise ValueError(f"{'K' if rowwise else 'N'} = {K if rowwise else N} is not a multiple of P = {P}")
    shape = (P, M, N if rowwise else N // P)
    _expect("x", x, (P, M, K // P) if rowwise else (M, K), dtype)
    _expect("A", A, (n, R, K), dtype)
    _expect("B", B, (n, N, R), dtype)
    _expect("ids", ids, (M,), torch.int32)
    _expect("base", base, shape, dtype)
    _expect("gains", gains, (n,), torch.float32, optional=True)
    _expect("out", out, shape, dtype, optional=True)
    cur = _ready(x, A, B, ids, base, gains, out, workspace)
    if out is None:
        out = _new(shape, dtype, x.device, stream)
    if workspace is None:
        workspace = _new((max(sptp_lora_workspace_size(P, M, K, N, R, rowwise), SPTP_WS_HEADER_BYTES),), torch.uint8, x.device,
                         stream)
    args = (x.data_ptr(), A.data_ptr(), B.data_ptr(), ids.data_ptr(), None if gains is None else gains.data_ptr(), P, M, K, N, R, n,
            int(rowwise), dt, base.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, cur))
    return args, out, workspace
