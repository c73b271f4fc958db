"""Python binding of libgdn.so, the Gated DeltaNet token mixer for B200.

Argument marshalling only: every function here hands device pointers of
torch tensors, sizes and the current CUDA stream to one C entry point of
``libgdn.so`` (declared in ``include/gdn.h``) and raises ``GdnError`` on a
non-zero status.  There is no fallback: if the library is missing or was not
built, the first call raises.  Build it with
``python -m linear_attention_recurrence_deltanet_b200.build``.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

__all__ = [
    "GdnError", "Config", "Params", "lib", "make_config", "conv_prefill", "conv_step", "prefill_workspace_size",
    "prefill", "prefill_noalloc", "decode_step", "decode_multi", "decode_step_indexed", "decode_multi_indexed",
    "prefill_indexed_workspace_size", "prefill_indexed", "gemm_bf16", "project_in", "project_out", "prefill_seqpar_workspace_size", "prefill_seqpar", "state_blob_size", "state_save", "state_restore", "device_status", "debug_wait_expiry", "last_error",
    "abi_version", "launch_count", "launch_count_reset", "profiler_enable", "profiler_reset", "profiler_read",
    "kernel_name", "AttnConfig", "RopePlan", "Q4Weight", "make_attn_config", "rope_plan", "rope", "kv_page_bytes",
    "kv_append", "kv_read", "attention_workspace_size", "attention", "q4_pack", "linear_q4_workspace_size", "linear_q4",
    "EXPORTS", "ZERO_INIT_STATE", "ZERO_INIT_CONV", "PREFILL_RECURRENT", "PREFILL_FUSED", "PREFILL_FACTORED", "PREFILL_AFFINE", "K", "MAX_DRAFT_TOKENS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdn.so")

ZERO_INIT_STATE = 0x1
ZERO_INIT_CONV = 0x2
PREFILL_RECURRENT = 0x4
PREFILL_FUSED = 0x8
PREFILL_FACTORED = 0x10
PREFILL_AFFINE = 0x20
MAX_DRAFT_TOKENS = 4

F32, BF16 = 0, 1

STATUS = {0: "GDN_OK", -1: "GDN_E_INVAL", -2: "GDN_E_UNSUPPORTED", -3: "GDN_E_WORKSPACE", -4: "GDN_E_CUDA",
          -5: "GDN_E_BLOB_FORMAT", -6: "GDN_E_BLOB_VERSION", -7: "GDN_E_BLOB_GEOMETRY", -8: "GDN_E_BLOB_CHECKSUM",
          -9: "GDN_E_DEVICE"}


class K:
    """Kernel ids of the profiler (gdn_kernel_id)."""
    (CONV_PREFILL, CONV_STEP, CONV_HISTORY, SCHEDULE, PREFILL_RECURRENT, PREFILL_CHUNKED, DECODE, STATE_CHECKSUM,
     SPLIT_CONV, SPLIT_PREP, SPLIT_CHAIN, SLOT_COPY, GEMM, SEQPAR, DIAG, WY_CONV, WY_PREP, WY_CHAIN, ROPE, KV_APPEND,
     KV_READ, ATTENTION, ATTN_COMBINE, Q4_PACK, LINEAR_Q4, X_HALF) = range(26)
    COUNT = 26


# Every symbol include/gdn.h declares.
EXPORTS = [
    "gdn_conv_prefill", "gdn_conv_step", "gdn_prefill_workspace_size", "gdn_prefill", "gdn_decode_step",
    "gdn_state_blob_size", "gdn_state_save", "gdn_state_restore", "gdn_get_device_status", "gdn_last_error",
    "gdn_abi_version", "gdn_launch_count", "gdn_launch_count_reset", "gdn_kernel_name", "gdn_profiler_enable",
    "gdn_profiler_reset", "gdn_profiler_read", "gdn_prefill_noalloc", "gdn_decode_multi",
    "gdn_decode_step_indexed", "gdn_decode_multi_indexed", "gdn_prefill_indexed_workspace_size",
    "gdn_prefill_indexed", "gdn_gemm_bf16", "gdn_project_in", "gdn_project_out",
    "gdn_prefill_seqpar_workspace_size", "gdn_prefill_seqpar", "gdn_debug_wait_expiry",
    "gdn_rope_plan_init", "gdn_rope", "gdn_kv_page_bytes", "gdn_kv_append", "gdn_kv_read",
    "gdn_attention_workspace_size", "gdn_attention", "gdn_q4_packed_bytes", "gdn_q4_pack",
    "gdn_linear_q4_workspace_size", "gdn_linear_q4",
]


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class Config(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32), ("head_k_dim", ctypes.c_int32),
                ("head_v_dim", ctypes.c_int32), ("conv_width", ctypes.c_int32), ("l2_eps", ctypes.c_float),
                ("norm_eps", ctypes.c_float), ("q_scale", ctypes.c_float), ("io_dtype", ctypes.c_int32)]


class Params(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("norm_w", ctypes.c_void_p)]


ROPE_MAX_PAIRS = 128
ROPE_LAYOUTS = {"sections": 0, "interleaved": 1, "per_axis": 2}


class RopePlan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32), ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS),
                ("turn", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


class AttnConfig(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("io_dtype", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32)]


_lib = None


def lib():
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m linear_attention_recurrence_deltanet_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, U32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
        sig = {
            "gdn_conv_prefill": [P, P, P, P, P, I32, P, P, P],
            "gdn_conv_step": [P, P, P, I32, P, P, P],
            "gdn_prefill_workspace_size": [P, I64, I32, I32, P],
            "gdn_prefill": [P, P, P, P, P, P, P, P, I32, I32, U32, P, P, P, P, SZ, P],
            "gdn_prefill_noalloc": [P, P, P, P, P, P, P, P, I32, I32, U32, P, P, P, P],
            "gdn_decode_step": [P, P, P, P, P, P, I32, P, P, P, P],
            "gdn_decode_multi": [P, P, P, P, P, P, I32, I32, I32, P, P, P, P, P],
            "gdn_decode_step_indexed": [P, P, P, P, P, P, I32, P, I32, P, P, P, P],
            "gdn_decode_multi_indexed": [P, P, P, P, P, P, I32, I32, I32, P, P, I32, P, P, P, P],
            "gdn_prefill_indexed_workspace_size": [P, I64, I32, I32, P],
            "gdn_prefill_indexed": [P, P, P, P, P, P, P, P, I32, P, I32, I32, U32, P, P, P, P, SZ, P],
            "gdn_gemm_bf16": [P, I32, I32, P, I32, P, I32, P],
            "gdn_project_in": [P, P, I32, I32, P, P, P, P, P, P],
            "gdn_project_out": [P, P, I32, P, I32, P, P],
            "gdn_prefill_seqpar_workspace_size": [P, I64, I32, P],
            "gdn_prefill_seqpar": [P, P, P, P, P, P, I64, I32, U32, P, P, P, P, SZ, P, P],
            "gdn_rope_plan_init": [I32, ctypes.c_double, P, I32, P, I32, P],
            "gdn_rope": [P, I32, P, I64, P, I32, I32, I32, I32, P, I64, P],
            "gdn_kv_page_bytes": [P, P],
            "gdn_kv_append": [P, P, P, I64, P, I64, P, I64, P, P, P, I32, P, P, I64, P],
            "gdn_kv_read": [P, P, P, I32, P, P, P, P],
            "gdn_attention_workspace_size": [P, I64, I32, P],
            "gdn_attention": [P, P, I64, P, P, I32, P, P, P, P, SZ, P],
            "gdn_q4_packed_bytes": [I32, I32, I32, P],
            "gdn_q4_pack": [P, P, P, I32, I32, I32, P, P],
            "gdn_linear_q4_workspace_size": [I32, I32, I32, I32, I32, P],
            "gdn_linear_q4": [I32, P, I32, I32, P, I32, I32, P, P, SZ, P],
            "gdn_state_blob_size": [P, P],
            "gdn_state_save": [P, P, P, I32, P, SZ, P],
            "gdn_state_restore": [P, P, SZ, I32, P, P, P],
            "gdn_get_device_status": [P, P],
            "gdn_debug_wait_expiry": [ctypes.c_uint32, P],
            "gdn_profiler_enable": [I32],
            "gdn_profiler_reset": [],
            "gdn_profiler_read": [I32, P, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = I32
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_kernel_name.restype = ctypes.c_char_p
        L.gdn_kernel_name.argtypes = [I32]
        L.gdn_abi_version.restype = I32
        L.gdn_launch_count.restype = I64
        L.gdn_launch_count_reset.restype = None
        _lib = L
    return _lib


def last_error() -> str:
    return lib().gdn_last_error().decode()


def _check(rc: int):
    if rc != 0:
        raise GdnError(rc, last_error())


def make_config(geo) -> Config:
    """Config from an ``inputs.Geometry`` (or any object with the same fields)."""
    return Config(geo.num_k_heads, geo.num_v_heads, geo.head_k_dim, geo.head_v_dim, geo.conv_width, geo.l2_eps,
                  geo.norm_eps, geo.q_scale, BF16 if geo.io_dtype == "bf16" else F32)


def _p(t) -> Optional[int]:
    """Data pointer of a torch tensor / numpy array (None passes NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream=None) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return torch.cuda.current_stream().cuda_stream


def _host_cu(cu_host) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(cu_host), dtype=np.int32)


def _params(conv_w, A_log, dt_bias, norm_w) -> Params:
    return Params(_p(conv_w), _p(A_log), _p(dt_bias), _p(norm_w))


def conv_prefill(cfg, x, conv_w, cu_dev, cu_host, conv_state, y, stream=None):
    cu_h = _host_cu(cu_host)
    _check(lib().gdn_conv_prefill(ctypes.byref(cfg), _p(x), _p(conv_w), _p(cu_dev), cu_h.ctypes.data,
                                  cu_h.size - 1, _p(conv_state), _p(y), _stream(stream)))


def conv_step(cfg, x, conv_w, num_seqs, conv_state, y, stream=None):
    _check(lib().gdn_conv_step(ctypes.byref(cfg), _p(x), _p(conv_w), num_seqs, _p(conv_state), _p(y),
                               _stream(stream)))


def prefill_workspace_size(cfg, total_tokens: int, num_seqs: int, chunk_size: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_prefill_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs, chunk_size,
                                            ctypes.byref(out)))
    return out.value


def prefill(cfg, params, qkv, z, a, b, cu_dev, cu_host, chunk_size, flags, conv_state, state, o, workspace,
            workspace_bytes=None, stream=None):
    """gdn_prefill.  params = (conv_w, A_log, dt_bias, norm_w) device tensors."""
    cu_h = _host_cu(cu_host)
    prm = _params(*params)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().gdn_prefill(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), _p(cu_dev),
                             cu_h.ctypes.data, cu_h.size - 1, chunk_size, flags, _p(conv_state), _p(state), _p(o),
                             _p(workspace), workspace_bytes, _stream(stream)))


def prefill_noalloc(cfg, params, qkv, z, a, b, cu_dev, cu_host, chunk_size, flags, conv_state, state, o,
                    stream=None):
    """gdn_prefill_noalloc: gdn_prefill with the library's built-in scratch
    instead of a caller workspace (for callers that cannot allocate device
    memory); calls that overlap on the GPU share that scratch and race."""
    cu_h = _host_cu(cu_host)
    prm = _params(*params)
    _check(lib().gdn_prefill_noalloc(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), _p(cu_dev),
                                     cu_h.ctypes.data, cu_h.size - 1, chunk_size, flags, _p(conv_state), _p(state),
                                     _p(o), _stream(stream)))


def decode_step(cfg, params, qkv, z, a, b, num_seqs, conv_state, state, o, stream=None):
    prm = _params(*params)
    _check(lib().gdn_decode_step(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), num_seqs,
                                 _p(conv_state), _p(state), _p(o), _stream(stream)))


def decode_multi(cfg, params, qkv, z, a, b, num_seqs, num_tokens, commit, accept, conv_state, state, o,
                 stream=None):
    """gdn_decode_multi: num_tokens draft tokens per sequence in one pass.
    commit=False verifies (outputs only, caches untouched, accept None);
    commit=True applies accept[n] tokens (device int32, None = all)."""
    prm = _params(*params)
    _check(lib().gdn_decode_multi(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), num_seqs,
                                  num_tokens, 1 if commit else 0, _p(accept),
                                  _p(conv_state), _p(state), _p(o), _stream(stream)))


def decode_step_indexed(cfg, params, qkv, z, a, b, num_seqs, state_indices, num_slots, conv_state, state, o,
                        stream=None):
    """gdn_decode_step_indexed: row n of the batch uses pool slot
    state_indices[n] (device int32; negative = padding row)."""
    prm = _params(*params)
    _check(lib().gdn_decode_step_indexed(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b),
                                         num_seqs, _p(state_indices), num_slots, _p(conv_state), _p(state), _p(o),
                                         _stream(stream)))


def decode_multi_indexed(cfg, params, qkv, z, a, b, num_seqs, num_tokens, commit, accept, state_indices, num_slots,
                         conv_state, state, o, stream=None):
    """gdn_decode_multi_indexed: gdn_decode_multi over pool slots."""
    prm = _params(*params)
    _check(lib().gdn_decode_multi_indexed(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b),
                                          num_seqs, num_tokens, 1 if commit else 0, _p(accept), _p(state_indices),
                                          num_slots, _p(conv_state), _p(state), _p(o), _stream(stream)))


def prefill_indexed_workspace_size(cfg, total_tokens: int, num_seqs: int, chunk_size: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_prefill_indexed_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs, chunk_size,
                                                    ctypes.byref(out)))
    return out.value


def prefill_indexed(cfg, params, qkv, z, a, b, cu_dev, cu_host, state_indices, num_slots, chunk_size, flags,
                    conv_state, state, o, workspace, workspace_bytes=None, stream=None):
    """gdn_prefill_indexed: gdn_prefill over pool slots (a batch may mix
    prefill sequences with length-1 decode steps)."""
    cu_h = _host_cu(cu_host)
    prm = _params(*params)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().gdn_prefill_indexed(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), _p(cu_dev),
                                     cu_h.ctypes.data, cu_h.size - 1, _p(state_indices), num_slots, chunk_size, flags,
                                     _p(conv_state), _p(state), _p(o), _p(workspace), workspace_bytes,
                                     _stream(stream)))


def gemm_bf16(x, w, y, tile_n: int = 0, stream=None):
    """gdn_gemm_bf16: y [M, N] = x [M, K] @ w [N, K]^T, all bf16 (fp32 accumulation)."""
    M, K = x.shape[0], x.shape[1]
    N = w.shape[0]
    _check(lib().gdn_gemm_bf16(_p(x), M, K, _p(w), N, _p(y), tile_n, _stream(stream)))


def project_in(cfg, x, w_in, qkv, z, a, b, stream=None):
    """gdn_project_in: x [T, hidden] through w_in [C_conv + Hv*d_v + 2*Hv, hidden] into qkv, z, a, b."""
    _check(lib().gdn_project_in(ctypes.byref(cfg), _p(x), x.shape[0], x.shape[1], _p(w_in), _p(qkv), _p(z), _p(a),
                                _p(b), _stream(stream)))


def project_out(cfg, o, w_out, y, stream=None):
    """gdn_project_out: y [T, hidden] = o [T, Hv*d_v] @ w_out [hidden, Hv*d_v]^T."""
    _check(lib().gdn_project_out(ctypes.byref(cfg), _p(o), o.shape[0], _p(w_out), w_out.shape[0], _p(y),
                                 _stream(stream)))


def prefill_seqpar_workspace_size(cfg, total_tokens: int, segments: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_prefill_seqpar_workspace_size(ctypes.byref(cfg), total_tokens, segments, ctypes.byref(out)))
    return out.value


def prefill_seqpar(cfg, params, qkv, z, a, b, total_tokens, segments, flags, conv_state, state, o, workspace,
                   workspace_bytes=None, stream=None) -> int:
    """gdn_prefill_seqpar: one sequence of total_tokens tokens in `segments`
    chunk-aligned segments (0 = from the SM count); returns the count used."""
    prm = _params(*params)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    used = ctypes.c_int32(0)
    _check(lib().gdn_prefill_seqpar(ctypes.byref(cfg), ctypes.byref(prm), _p(qkv), _p(z), _p(a), _p(b), total_tokens,
                                    segments, flags, _p(conv_state), _p(state), _p(o), _p(workspace),
                                    workspace_bytes, ctypes.byref(used), _stream(stream)))
    return used.value


# ---------------------------------------------------------------- attention side and 4-bit projections
# These calls take tensors whose layout the C entry points cannot see, so the
# binding checks what it can (device, type, shape, strides) before it passes
# pointers on.  All tensors live on the current CUDA device.


def _need(ok: bool, message: str):
    if not ok:
        raise GdnError(-1, message)


class _Torch:
    """torch's types and the calls behind torch.cuda.current_device and current_stream, bound at the first use (the
    package imports without torch)."""
    bf16 = f32 = i32 = u8 = device = raw_stream = None


def _torch():
    import torch
    _Torch.bf16, _Torch.f32, _Torch.i32, _Torch.u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    _Torch.device = torch.cuda.current_device
    _Torch.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _io(dtype) -> int:
    if dtype is _Torch.bf16 and dtype is not None:
        return BF16
    if dtype is _Torch.f32 and dtype is not None:
        return F32
    name = str(dtype)
    if name in ("torch.bfloat16", "bf16"):
        return BF16
    if name in ("torch.float32", "f32"):
        return F32
    raise GdnError(-2, f"io type {name} is not bf16 or float32")


def _device(t, stream):
    """(current device, raw stream); t is on a CUDA device (_ptr and _heads check that it is the current one)."""
    if _Torch.device is None:
        _torch()
    if t.get_device() < 0:
        raise GdnError(-1, "tensors must be CUDA tensors")
    dev = _Torch.device()
    return dev, _Torch.raw_stream(dev) if stream is None else _stream(stream)


def _ptr(t, dev: int, name: str, dtype, numel: Optional[int] = None) -> int:
    """Pointer of a contiguous tensor of a type (and, if given, at least numel elements) on device dev."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise GdnError(-1, f"{name} must be a contiguous {dtype} tensor on device {dev}")
    if numel is not None and t.numel() < numel:
        raise GdnError(-1, f"{name} has {t.numel()} elements, {numel} are needed")
    return t.data_ptr()


def _heads(t, dev: int, name: str, io: int, T: int, H: int, D: int):
    """(pointer, elements between tokens) of rows [T, H, D] whose heads are contiguous within a token."""
    if (t.shape != (T, H, D) or t.dtype is not (_Torch.bf16 if io == BF16 else _Torch.f32) or t.get_device() != dev):
        raise GdnError(-1, f"{name} must be [{T}, {H}, {D}] in the io type on device {dev}, got {list(t.shape)} {t.dtype}")
    st = t.stride()
    if T > 0 and (st[2] != 1 or (H > 1 and st[1] != D)):
        raise GdnError(-1, f"{name}: a token's heads must be contiguous (strides {st})")
    return t.data_ptr(), st[0] if T > 1 else max(st[0], H * D)


def _cu_host(cu_host):
    """(array of int32, its pointer, sequences, tokens)"""
    if not (type(cu_host) is np.ndarray and cu_host.dtype == np.int32 and cu_host.flags.c_contiguous):
        cu_host = _host_cu(cu_host)
    n = cu_host.size - 1
    if n < 1:
        raise GdnError(-1, "cu_seqlens needs two entries or more")
    return cu_host, cu_host.ctypes.data, n, int(cu_host[n])


_PAGE_BYTES = {}  # kv_page_bytes by the sizes it depends on


def _cache(cfg, dev, cu_dev, n, kv_lens, pool, page_table) -> KvCache:
    _ptr(cu_dev, dev, "cu_seqlens", _Torch.i32, n + 1)
    key = (cfg.num_kv_heads, cfg.head_dim, cfg.page_size)
    size = _PAGE_BYTES.get(key)
    if size is None:
        size = _PAGE_BYTES[key] = kv_page_bytes(cfg)
    rows, pages = page_table.shape, pool.shape
    if len(rows) != 2 or rows[0] < n:
        raise GdnError(-1, "page_table must be [num_seqs, pages_per_seq]")
    if len(pages) != 2 or pages[1] != size:
        raise GdnError(-1, "pool must be [num_pages, kv_page_bytes]")
    return KvCache(_ptr(pool, dev, "pool", _Torch.u8), _ptr(page_table, dev, "page_table", _Torch.i32),
                   _ptr(kv_lens, dev, "kv_lens", _Torch.i32, n), pages[0], rows[1])


def make_attn_config(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int = 64, io_dtype="bf16",
                     softmax_scale: Optional[float] = None) -> AttnConfig:
    """gdn_attn_config; softmax_scale defaults to head_dim ** -0.5."""
    return AttnConfig(num_q_heads, num_kv_heads, head_dim, page_size,
                      head_dim ** -0.5 if softmax_scale is None else softmax_scale, _io(io_dtype))


def rope_plan(rotary_dim: int, theta: float = 10000.0, sections=None, layout: str = "sections",
              inv_freq=None) -> RopePlan:
    """gdn_rope_plan_init: the rotation of the first rotary_dim channels.  sections: pairs of each axis (1 to 3 of
    them, None = one axis); layout "sections", "interleaved" or "per_axis"; inv_freq: rotary_dim / 2 frequencies in
    radians per position in place of theta's."""
    _need(layout in ROPE_LAYOUTS, f"layout {layout!r} is none of {sorted(ROPE_LAYOUTS)}")
    plan = RopePlan()
    sec = None if sections is None else np.ascontiguousarray(sections, np.int32)
    _need(sec is None or sec.ndim == 1, "sections is a flat list")
    inv = None if inv_freq is None else np.ascontiguousarray(inv_freq, np.float64)
    _need(inv is None or inv.shape == (rotary_dim // 2,), f"inv_freq must have {rotary_dim // 2} values")
    _check(lib().gdn_rope_plan_init(rotary_dim, theta, _p(inv), 1 if sec is None else sec.size, _p(sec),
                                    ROPE_LAYOUTS[layout], ctypes.byref(plan)))
    return plan


def _positions(plan, positions, dev, T: int) -> int:
    shape = positions.shape
    if shape != (plan.num_axes, T) and not (plan.num_axes == 1 and shape == (T,)):
        raise GdnError(-1, f"positions must be [{plan.num_axes}, {T}], got {list(shape)}")
    return _ptr(positions, dev, "positions", _Torch.i32)


def rope(plan, x, positions, out, inverse: bool = False, stream=None):
    """gdn_rope: out = x [T, heads, head_dim] rotated (out may be x); positions [axes, T] int32."""
    dev, st = _device(x, stream)
    if x.dim() != 3:
        raise GdnError(-1, "x must be [tokens, heads, head_dim]")
    io, (T, H, D) = _io(x.dtype), x.shape
    px, ldx = _heads(x, dev, "x", io, T, H, D)
    po, ldo = _heads(out, dev, "out", io, T, H, D)
    _check(lib().gdn_rope(ctypes.byref(plan), io, px, ldx, _positions(plan, positions, dev, T), T, H, D,
                          1 if inverse else 0, po, ldo, st))


def kv_page_bytes(cfg) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_kv_page_bytes(ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def kv_append(cfg, plan, q, k, v, positions, cu_dev, cu_host, kv_lens, pool, page_table, q_out, stream=None):
    """gdn_kv_append: q [T, Hq, D] rotated into q_out, k and v [T, Hkv, D] into the 4-bit cache (k rotated).  plan None:
    no rotation; positions None: the cache positions; q and q_out may be None."""
    dev, st = _device(k, stream)
    cu_h, pcu, n, T = _cu_host(cu_host)
    io, D, hq, hkv = cfg.io_dtype, cfg.head_dim, cfg.num_q_heads, cfg.num_kv_heads
    c = _cache(cfg, dev, cu_dev, n, kv_lens, pool, page_table)
    pk, ldk = _heads(k, dev, "k", io, T, hkv, D)
    pv, ldv = _heads(v, dev, "v", io, T, hkv, D)
    pq, ldq = (None, 0) if q is None else _heads(q, dev, "q", io, T, hq, D)
    po, ldo = (None, 0) if q_out is None else _heads(q_out, dev, "q_out", io, T, hq, D)
    _check(lib().gdn_kv_append(ctypes.byref(cfg), None if plan is None else ctypes.byref(plan), pq, ldq, pk, ldk, pv,
                               ldv, None if positions is None or plan is None else _positions(plan, positions, dev, T),
                               cu_dev.data_ptr(), pcu, n, ctypes.byref(c), po, ldo, st))


def kv_read(cfg, cu_dev, cu_host, kv_lens, pool, page_table, k_out, v_out, stream=None):
    """gdn_kv_read: the cache's values for the last tokens of each sequence, k_out and v_out [T, Hkv, D]."""
    dev, st = _device(pool, stream)
    cu_h, pcu, n, T = _cu_host(cu_host)
    c = _cache(cfg, dev, cu_dev, n, kv_lens, pool, page_table)
    dt = _Torch.bf16 if cfg.io_dtype == BF16 else _Torch.f32
    need = T * cfg.num_kv_heads * cfg.head_dim
    _check(lib().gdn_kv_read(ctypes.byref(cfg), cu_dev.data_ptr(), pcu, n, ctypes.byref(c),
                             _ptr(k_out, dev, "k_out", dt, need), _ptr(v_out, dev, "v_out", dt, need), st))


def attention_workspace_size(cfg, total_tokens: int, num_seqs: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_attention_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs, ctypes.byref(out)))
    return out.value


def attention(cfg, q, cu_dev, cu_host, kv_lens, pool, page_table, o, lse=None, workspace=None, stream=None):
    """gdn_attention: causal attention of q [T, Hq, D] over the 4-bit cache into o [T, Hq, D] (and lse [T, Hq] fp32)."""
    dev, st = _device(q, stream)
    cu_h, pcu, n, T = _cu_host(cu_host)
    io, hq, D = cfg.io_dtype, cfg.num_q_heads, cfg.head_dim
    c = _cache(cfg, dev, cu_dev, n, kv_lens, pool, page_table)
    pq, ldq = _heads(q, dev, "q", io, T, hq, D)
    po = _ptr(o, dev, "o", _Torch.bf16 if io == BF16 else _Torch.f32, T * hq * D)
    pl = None if lse is None else _ptr(lse, dev, "lse", _Torch.f32, T * hq)
    pw, nw = (None, 0) if workspace is None else (_ptr(workspace, dev, "workspace", _Torch.u8), workspace.numel())
    _check(lib().gdn_attention(ctypes.byref(cfg), pq, ldq, cu_dev.data_ptr(), pcu, n, ctypes.byref(c), po, pl, pw, nw,
                               st))


class Q4Weight:
    """A weight [N, K] in 4 bits, packed for linear_q4 (see q4_pack)."""

    def __init__(self, data, N: int, K: int, group: int):
        self.data, self.N, self.K, self.group = data, N, K, group


_Q4_BYTES = {}  # gdn_q4_packed_bytes by (N, K, group)


def _q4_bytes(N: int, K: int, group: int) -> int:
    size = _Q4_BYTES.get((N, K, group))
    if size is None:
        out = ctypes.c_size_t()
        _check(lib().gdn_q4_packed_bytes(N, K, group, ctypes.byref(out)))
        size = _Q4_BYTES[N, K, group] = out.value
    return size


def q4_pack(codes, scales, biases, K: int, group: int, stream=None) -> Q4Weight:
    """gdn_q4_pack: codes uint8 [N, ceil(K / group) * group / 2] (channel 2i in the low half of byte i), scales and
    biases bf16 [N, ceil(K / group)]; a code c stands for scale * c + bias.  The packed weight is allocated on `stream`, as
    any tensor made there: another stream waits for it before it reads, and the caller keeps it until it has."""
    import torch
    dev, st = _device(codes, stream)
    _need(codes.dim() == 2, f"codes must be [N, ceil(K / group) * group / 2], got {list(codes.shape)}")
    N = codes.shape[0]
    size = _q4_bytes(N, K, group)
    G = -(-K // group)
    _need(tuple(codes.shape) == (N, G * group // 2), f"codes must be [{N}, {G * group // 2}], got {list(codes.shape)}")
    _need(tuple(scales.shape) == (N, G) and tuple(biases.shape) == (N, G), f"scales and biases must be [{N}, {G}]")
    # from the memory of the stream that writes it: what the current stream has freed may still be read there
    with torch.cuda.stream(torch.cuda.ExternalStream(st, dev) if st != _Torch.raw_stream(dev) else None):
        data = torch.empty(size, dtype=torch.uint8, device=codes.device)
    _check(lib().gdn_q4_pack(_ptr(codes, dev, "codes", _Torch.u8), _ptr(scales, dev, "scales", _Torch.bf16),
                             _ptr(biases, dev, "biases", _Torch.bf16), N, K, group, data.data_ptr(), st))
    return Q4Weight(data, N, K, group)


def linear_q4_workspace_size(M: int, N: int, K: int, group: int, io_dtype="bf16") -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_linear_q4_workspace_size(M, N, K, group, _io(io_dtype), ctypes.byref(out)))
    return out.value


def linear_q4(x, w: Q4Weight, y, workspace=None, stream=None):
    """gdn_linear_q4: y [M, N] = x [M, K] @ w^T for a packed 4-bit weight."""
    dev, st = _device(x, stream)
    shape, dt, N, K = x.shape, x.dtype, w.N, w.K
    if len(shape) != 2 or shape[1] != K:
        raise GdnError(-1, f"x must be [rows, {K}], got {list(shape)}")
    io, M = _io(dt), shape[0]
    if y.shape != (M, N):
        raise GdnError(-1, f"y must be [{M}, {N}], got {list(y.shape)}")
    pw, nw = (None, 0) if workspace is None else (_ptr(workspace, dev, "workspace", _Torch.u8), workspace.numel())
    pd = _ptr(w.data, dev, "w", _Torch.u8, _q4_bytes(N, K, w.group))
    _check(lib().gdn_linear_q4(io, _ptr(x, dev, "x", dt), M, K, pd, N, w.group, _ptr(y, dev, "y", dt), pw, nw, st))


def state_blob_size(cfg) -> int:
    out = ctypes.c_size_t()
    _check(lib().gdn_state_blob_size(ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def _nbytes(t) -> int:
    return t.nbytes if isinstance(t, np.ndarray) else t.numel() * t.element_size()


def state_save(cfg, conv_state, state, seq, blob, stream=None):
    _check(lib().gdn_state_save(ctypes.byref(cfg), _p(conv_state), _p(state), seq, _p(blob), _nbytes(blob),
                                _stream(stream)))


def state_restore(cfg, blob, seq, conv_state, state, stream=None):
    _check(lib().gdn_state_restore(ctypes.byref(cfg), _p(blob), _nbytes(blob), seq, _p(conv_state), _p(state),
                                   _stream(stream)))


def device_status(stream=None) -> int:
    code = ctypes.c_int32()
    _check(lib().gdn_get_device_status(ctypes.byref(code), _stream(stream)))
    return code.value


def debug_wait_expiry(limit_us: int, stream=None):
    """gdn_debug_wait_expiry: a kernel whose bounded wait always runs out
    after limit_us; the device status word then reads 1 (wait timeout)."""
    _check(lib().gdn_debug_wait_expiry(limit_us, _stream(stream)))


def abi_version() -> int:
    return lib().gdn_abi_version()


def launch_count() -> int:
    return lib().gdn_launch_count()


def launch_count_reset():
    lib().gdn_launch_count_reset()


def kernel_name(kid: int) -> str:
    return lib().gdn_kernel_name(kid).decode()


def profiler_enable(on: bool = True):
    _check(lib().gdn_profiler_enable(1 if on else 0))


def profiler_reset():
    _check(lib().gdn_profiler_reset())


def profiler_read(kid: int):
    """(launches, total device ms) of one kernel id since the last reset."""
    n, ms = ctypes.c_int64(), ctypes.c_double()
    _check(lib().gdn_profiler_read(kid, ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value
