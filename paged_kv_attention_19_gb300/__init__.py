"""Paged decode attention for GB300 (sm_103a): Python binding of the C ABI.

The binding only marshals arguments: every step of the decode runs in the CUDA
kernels of ``_lib/libpa_decode.so`` (declared in ``include/pa_decode.h``).
There is no CPU fallback: importing this package fails with ImportError if the
library has not been built (``python paged_kv_attention_19_gb300/build.py``).

Names follow the C ABI: ``pa_workspace_size``, ``pa_decode_gqa``,
``pa_decode_mla_absorbed``, ``pa_verify_gqa``, ``pa_decode_gqa_fp8``, ``pa_decode_gqa_nvfp4``,
``pa_decode_gqa_noalloc``, ``pa_kv_write``, ``pa_kv_write_fp8``, ``pa_kv_write_nvfp4``, ``pa_mla_cache_write``, ``pa_plan_step``,
``pa_qk_norm_rope_write``, ``pa_qk_norm_rope_write_fp8``, ``pa_qk_norm_rope_write_nvfp4``, ``pa_tree_gqa``, ``pa_tree_gqa_fp8``,
``pa_tree_gqa_nvfp4``, ``pa_tree_workspace_size``, ``pa_kv_compact``, ``pa_stream_gqa``, ``pa_stream_gqa_fp8``,
``pa_stream_gqa_nvfp4``, ``pa_stream_workspace_size``, ``pa_release_pages`` (the C ABI's ``_granted`` forms are
reached by the ``granted`` argument), ``pa_status_string``, ``pa_read_device_status``,
``pa_set_profile_events``, ``pa_last_launch_count``, ``pa_set_wait_limit_ns``, ``pa_last_cuda_error``,
``pa_last_cuda_error_string``.  The operators of tree drafting and of streams are called through a compiled module that
checks their tensors (``csrc/pa_binding.cpp``).  The tensor-taking
functions accept torch tensors (device memory, the layouts of the header) and
infer every size from their shapes.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpa_decode.so")
BINDING_PATH = os.path.join(_HERE, "_lib", "pa_binding.so")

PA_OK = 0
PA_ERR_INVALID_ARGUMENT = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_MISALIGNED = -3
PA_ERR_WORKSPACE_TOO_SMALL = -4
PA_ERR_CUDA = -5
PA_KIND_GQA = 0
PA_KIND_MLA_ABSORBED = 1
PA_DEV_BAD_PAGE = 0x1
PA_DEV_BAD_LEN = 0x2
PA_DEV_TIMEOUT = 0x4
PA_DEV_BAD_SLOT = 0x8
PA_DEV_NO_PAGES = 0x10
PA_DEV_BAD_POS = 0x20
PA_DEV_BAD_TREE = 0x40
PA_DEFAULT_WAIT_LIMIT_NS = 1_000_000_000

# Every symbol include/pa_decode.h declares, with its ctypes signature.
_P, _I, _F, _Z, _U32P = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
_LL = ctypes.c_longlong
SIGNATURES = {
    "pa_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "pa_decode_gqa": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _Z, _P]),
    "pa_decode_mla_absorbed": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _Z, _P]),
    "pa_decode_gqa_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "pa_verify_gqa": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _Z,
                           _P]),
    "pa_decode_gqa_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _F, _I,
                               _I, _P, _Z, _P]),
    "pa_decode_gqa_nvfp4": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _F, _I,
                                 _I, _P, _Z, _P]),
    "pa_kv_write_nvfp4": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _P, _P]),
    "pa_kv_write": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pa_kv_write_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _P, _P]),
    "pa_mla_cache_write": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "pa_plan_step": (_I, [_P] * 14 + [_I] * 5 + [_P, _P]),
    "pa_plan_step_granted": (_I, [_P] * 15 + [_I] * 5 + [_P, _P]),
    "pa_qk_norm_rope_write": (_I, [_P] * 11 + [_I] * 4 + [_LL] * 3 + [_I] * 3 + [_F] + [_I, _I, _P, _P]),
    "pa_qk_norm_rope_write_fp8": (_I, [_P] * 11 + [_I] * 4 + [_LL] * 3 + [_I] * 3 + [_F] * 3 + [_I, _I, _P, _P]),
    "pa_qk_norm_rope_write_nvfp4": (_I, [_P] * 11 + [_I] * 4 + [_LL] * 3 + [_I] * 3 + [_F] * 3 + [_I, _I, _P, _P]),
    "pa_tree_workspace_size": (_Z, [_I] * 8),
    "pa_tree_gqa": (_I, [_P] * 9 + [_I] * 10 + [_F, _I, _I, _P, _Z, _P]),
    "pa_tree_gqa_fp8": (_I, [_P] * 9 + [_I] * 10 + [_F, _F, _F, _I, _I, _P, _Z, _P]),
    "pa_tree_gqa_nvfp4": (_I, [_P] * 9 + [_I] * 10 + [_F, _F, _F, _I, _I, _P, _Z, _P]),
    "pa_tree_gqa_granted": (_I, [_P] * 10 + [_I] * 10 + [_F, _I, _I, _P, _Z, _P]),
    "pa_tree_gqa_fp8_granted": (_I, [_P] * 10 + [_I] * 10 + [_F, _F, _F, _I, _I, _P, _Z, _P]),
    "pa_tree_gqa_nvfp4_granted": (_I, [_P] * 10 + [_I] * 10 + [_F, _F, _F, _I, _I, _P, _Z, _P]),
    "pa_kv_compact": (_I, [_P] * 8 + [_I] * 7 + [_P, _P]),
    "pa_kv_compact_granted": (_I, [_P] * 9 + [_I] * 7 + [_P, _P]),
    "pa_stream_workspace_size": (_Z, [_I] * 8),
    "pa_stream_gqa": (_I, [_P] * 9 + [_I] * 10 + [_F, _I, _I, _I, _P, _Z, _P]),
    "pa_stream_gqa_fp8": (_I, [_P] * 9 + [_I] * 10 + [_F, _F, _F, _I, _I, _I, _P, _Z, _P]),
    "pa_stream_gqa_nvfp4": (_I, [_P] * 9 + [_I] * 10 + [_F, _F, _F, _I, _I, _I, _P, _Z, _P]),
    "pa_release_pages": (_I, [_P] * 12 + [_I] * 6 + [_P, _P]),
    "pa_status_string": (ctypes.c_char_p, [_I]),
    "pa_read_device_status": (_I, [_P, _P, _U32P]),
    "pa_set_profile_events": (_I, [_P, _P]),
    "pa_last_launch_count": (_I, []),
    "pa_set_wait_limit_ns": (_I, [ctypes.c_ulonglong]),
    "pa_last_cuda_error": (_I, []),
    "pa_last_cuda_error_string": (ctypes.c_char_p, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python paged_kv_attention_19_gb300/build.py` "
                          "(the decode has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class PaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = f"; {lib.pa_last_cuda_error_string().decode()}" if status == PA_ERR_CUDA else ""
        super().__init__(f"{what}: {pa_status_string(status)} ({status}){detail}")


def pa_status_string(status: int) -> str:
    return lib.pa_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != PA_OK:
        raise PaError(rc, what)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def pa_workspace_size(kind: int, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                      max_context_len: int, page_size: int, num_splits: int = 0) -> int:
    return int(lib.pa_workspace_size(kind, batch, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                     page_size, num_splits))


def pa_decode_gqa(q, k_pool, v_pool, block_table, context_lens, out, lse=None, *, scale: float,
                  workspace, window: int = 0, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """GQA paged decode.  q [B, Hq, D], pools [pages, P, Hkv, D] bf16; block_table [B, max_pages]
    int32; context_lens [B] int32; out [B, Hq, D] bf16; lse [B, Hq] fp32 or None; workspace: a
    device tensor of at least pa_workspace_size(...) bytes.  max_context_len defaults to
    max_pages * page_size (an upper bound that needs no device read)."""
    B, Hq, D = q.shape
    num_pages, P, Hkv, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if max_context_len is None:
        max_context_len = max_pages * P
    rc = lib.pa_decode_gqa(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(context_lens),
                           _ptr(out), _ptr(lse), B, Hq, Hkv, D, P, num_pages, max_pages, int(max_context_len),
                           float(scale), int(window), int(num_splits), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "pa_decode_gqa")


def pa_verify_gqa(q, k_pool, v_pool, block_table, context_lens, out, lse=None, *, scale: float,
                  workspace, window: int = 0, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """GQA multi-query verify.  q [B, Q, Hq, D]; out [B, Q, Hq, D]; lse [B, Q, Hq] or None;
    context_lens count the Q new tokens; the rest as for pa_decode_gqa."""
    B, Q, Hq, D = q.shape
    num_pages, P, Hkv, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if max_context_len is None:
        max_context_len = max_pages * P
    rc = lib.pa_verify_gqa(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(context_lens),
                           _ptr(out), _ptr(lse), B, Q, Hq, Hkv, D, P, num_pages, max_pages, int(max_context_len),
                           float(scale), int(window), int(num_splits), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "pa_verify_gqa")


def pa_decode_gqa_fp8(q, k_pool, v_pool, block_table, context_lens, out, lse=None, *, scale: float,
                      k_scale: float, v_scale: float, workspace, window: int = 0, num_splits: int = 0,
                      max_context_len=None, stream=None) -> None:
    """GQA decode (q [B, Hq, D]) or multi-query verify (q [B, Q, Hq, D]) over FP8 E4M3 pools
    [pages, P, Hkv, D] uint8 whose values are code * k_scale (keys) and code * v_scale (values);
    out and lse shaped like q without / with its last dim; the rest as for pa_verify_gqa."""
    if q.dim() == 3:
        B, Hq, D = q.shape
        Q = 1
    else:
        B, Q, Hq, D = q.shape
    num_pages, P, Hkv, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if max_context_len is None:
        max_context_len = max_pages * P
    rc = lib.pa_decode_gqa_fp8(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(context_lens),
                               _ptr(out), _ptr(lse), B, Q, Hq, Hkv, D, P, num_pages, max_pages,
                               int(max_context_len), float(scale), float(k_scale), float(v_scale), int(window),
                               int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    _check(rc, "pa_decode_gqa_fp8")


def pa_decode_gqa_nvfp4(q, k_pool, v_pool, block_table, context_lens, out, lse=None, *, scale: float,
                        k_scale: float, v_scale: float, workspace, window: int = 0, num_splits: int = 0,
                        max_context_len=None, stream=None) -> None:
    """GQA decode (q [B, Hq, D]) or multi-query verify (q [B, Q, Hq, D]) over NVFP4 pools
    [pages, P, Hkv, R] uint8 (R = nvfp4_row_bytes(D): code pairs, block scales, padding) whose
    values are e2m1(code) * e4m3(block scale) * k_scale (keys; v_scale for values); out and lse
    shaped like q without / with its last dim; the rest as for pa_verify_gqa."""
    if q.dim() == 3:
        B, Hq, D = q.shape
        Q = 1
    else:
        B, Q, Hq, D = q.shape
    num_pages, P, Hkv, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if max_context_len is None:
        max_context_len = max_pages * P
    rc = lib.pa_decode_gqa_nvfp4(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(context_lens),
                                 _ptr(out), _ptr(lse), B, Q, Hq, Hkv, D, P, num_pages, max_pages,
                                 int(max_context_len), float(scale), float(k_scale), float(v_scale), int(window),
                                 int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(rc, "pa_decode_gqa_nvfp4")


def nvfp4_row_bytes(head_dim: int) -> int:
    """Bytes of one NVFP4 pool row: head_dim / 2 code bytes and head_dim / 16 scale codes,
    padded to a multiple of 16."""
    return (head_dim // 2 + head_dim // 16 + 15) // 16 * 16


def pa_decode_mla_absorbed(q, cache, w_uk, w_uv, block_table, context_lens, out, lse=None, *, scale: float,
                           workspace, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """MLA absorbed decode.  q [B, H, 192], cache [pages, P, 576], w_uk / w_uv [H, 128, 512] bf16;
    out [B, H, 128] bf16; lse [B, H] fp32 or None."""
    B, H, _ = q.shape
    num_pages, P, _ = cache.shape
    max_pages = block_table.shape[1]
    if max_context_len is None:
        max_context_len = max_pages * P
    rc = lib.pa_decode_mla_absorbed(_ptr(q), _ptr(cache), _ptr(w_uk), _ptr(w_uv), _ptr(block_table),
                                    _ptr(context_lens), _ptr(out), _ptr(lse), B, H, P, num_pages, max_pages,
                                    int(max_context_len), float(scale), int(num_splits), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "pa_decode_mla_absorbed")


def pa_kv_write(k, v, slot_mapping, k_pool, v_pool, *, status=None, stream=None) -> None:
    """Paged KV write.  k, v [T, Hkv, D] bf16; slot_mapping [T] int64 (negative: padding, skipped);
    pools [pages, P, Hkv, D] bf16 (written at the named slots); status: optional uint32 device
    word that gets PA_DEV_BAD_SLOT for a slot past the pool."""
    T, Hkv, D = k.shape
    num_pages, P, _, _ = k_pool.shape
    _check(lib.pa_kv_write(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_pool), _ptr(v_pool), T, Hkv, D, P,
                           num_pages, _ptr(status), _stream(stream)), "pa_kv_write")


def pa_kv_write_fp8(k, v, slot_mapping, k_pool, v_pool, *, k_scale: float, v_scale: float, status=None,
                    stream=None) -> None:
    """FP8 paged KV write.  k, v [T, Hkv, D] bf16; pools [pages, P, Hkv, D] uint8 E4M3 codes of
    value / scale (nearest, ties to even, saturated at 448); the rest as for pa_kv_write."""
    T, Hkv, D = k.shape
    num_pages, P, _, _ = k_pool.shape
    _check(lib.pa_kv_write_fp8(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_pool), _ptr(v_pool), T, Hkv, D, P,
                               num_pages, float(k_scale), float(v_scale), _ptr(status), _stream(stream)),
           "pa_kv_write_fp8")


def pa_kv_write_nvfp4(k, v, slot_mapping, k_pool, v_pool, *, k_scale: float, v_scale: float, status=None,
                      stream=None) -> None:
    """NVFP4 paged KV write.  k, v [T, Hkv, D] bf16; pools [pages, P, Hkv, nvfp4_row_bytes(D)] uint8
    rows (E2M1 code pairs and E4M3 block scales of value / pool scale); the rest as for
    pa_kv_write."""
    T, Hkv, D = k.shape
    num_pages, P, _, _ = k_pool.shape
    _check(lib.pa_kv_write_nvfp4(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_pool), _ptr(v_pool), T, Hkv, D,
                                 P, num_pages, float(k_scale), float(v_scale), _ptr(status), _stream(stream)),
           "pa_kv_write_nvfp4")


def pa_mla_cache_write(c_lat, k_rope, slot_mapping, cache, *, status=None, stream=None) -> None:
    """MLA cache write.  c_lat [T, 512], k_rope [T, 64] bf16; cache [pages, P, 576] bf16."""
    T = c_lat.shape[0]
    num_pages, P, _ = cache.shape
    _check(lib.pa_mla_cache_write(_ptr(c_lat), _ptr(k_rope), _ptr(slot_mapping), _ptr(cache), T, P, num_pages,
                                  _ptr(status), _stream(stream)), "pa_mla_cache_write")


def _refuse(what: str, why: str):
    err = PaError(PA_ERR_INVALID_ARGUMENT, what)
    err.args = (f"{err.args[0]}: {why}",)
    raise err


_native_module = None


def _native():
    """The compiled calls (csrc/pa_binding.cpp), loaded at the first one: they need torch."""
    global _native_module
    if _native_module is None:
        import importlib.machinery
        import importlib.util
        import torch  # noqa: F401  (its libraries are the module's)
        if not os.path.exists(BINDING_PATH):
            raise ImportError(f"{BINDING_PATH} is not built; run `python paged_kv_attention_19_gb300/build.py`")
        loader = importlib.machinery.ExtensionFileLoader("pa_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("pa_binding", loader))
        loader.exec_module(module)
        _native_module = module
    return _native_module


def _done(what: str, answer) -> None:
    """The answer of a compiled call: None, a status, or what is wrong with an argument."""
    if answer is not None:
        if isinstance(answer, str):
            _refuse(what, answer)
        raise PaError(answer, what)


def pa_plan_step(context_lens, new_lens, held_pages, free_list, free_count, block_table, query_start, slot_mapping,
                 positions, *, page_size: int, context_lens_out=None, held_pages_out=None, free_count_out=None,
                 parents=None, tree_mask=None, granted=None, status=None, stream=None) -> None:
    """Plan of one step, all on the GPU.  context_lens, new_lens (negative: the row has ended) and
    held_pages [B] int32; free_list [num_pages] int32, a stack of which free_count [1] int32 entries
    are valid; block_table [B, max_pages] int32 gets the new pages' entries; query_start [B + 1] int32,
    slot_mapping [max_tokens] int64 and positions [max_tokens] int32 are written.  parents [max_tokens]
    int32 and tree_mask [max_tokens] int64 (the 64 mask bits) go together: drafted trees.  The _out
    arrays default to their inputs (updated in place).  granted: optional [B] int32, 1 for a row whose new
    tokens have their places and 0 for one that was refused or has ended; what pa_tree_gqa and
    pa_kv_compact take, so that they leave such a row alone.  status: optional int32 device word that gets
    PA_DEV_* bits (rows that found no pages: PA_DEV_NO_PAGES, their slots are -1)."""
    _done("pa_plan_step", (_native_module or _native()).plan_step(
        context_lens, new_lens, held_pages, free_list, free_count, block_table,
        context_lens if context_lens_out is None else context_lens_out,
        held_pages if held_pages_out is None else held_pages_out,
        free_count if free_count_out is None else free_count_out, query_start, slot_mapping, positions, parents,
        tree_mask, granted, status, page_size, stream))


def pa_qk_norm_rope_write(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, *,
                          eps: float = 1e-6, interleaved: bool = False, status=None, stream=None) -> None:
    """Per-head norms of q and k, position rotation and paged write.  q [T, Hq, D], k, v [T, Hkv, D] bf16,
    tokens any stride apart (views of one projection's output); q_weight, k_weight [D] bf16 or None (no
    norm); cos_sin [max_position, rot_dim] fp32 (cosines, then sines); positions [T] int32; slot_mapping
    [T] int64 (negative: padding, nothing written); q_out [T, Hq, D] bf16; pools [pages, P, Hkv, D] bf16;
    status: optional int32 device word for PA_DEV_* bits."""
    _done("pa_qk_norm_rope_write", (_native_module or _native()).qk_norm_rope_write(
        0, q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, status, eps,
        interleaved, 1.0, 1.0, stream))


def pa_qk_norm_rope_write_fp8(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, *,
                              k_scale: float, v_scale: float, eps: float = 1e-6, interleaved: bool = False,
                              status=None, stream=None) -> None:
    """The same into FP8 pools [pages, P, Hkv, D] uint8 (E4M3 codes of value / scale)."""
    _done("pa_qk_norm_rope_write_fp8", (_native_module or _native()).qk_norm_rope_write(
        1, q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, status, eps,
        interleaved, k_scale, v_scale, stream))


def pa_qk_norm_rope_write_nvfp4(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool,
                                *, k_scale: float, v_scale: float, eps: float = 1e-6, interleaved: bool = False,
                                status=None, stream=None) -> None:
    """The same into NVFP4 pools [pages, P, Hkv, nvfp4_row_bytes(D)] uint8."""
    _done("pa_qk_norm_rope_write_nvfp4", (_native_module or _native()).qk_norm_rope_write(
        2, q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, status, eps,
        interleaved, k_scale, v_scale, stream))


def pa_tree_workspace_size(batch: int, max_query: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           max_context_len: int, page_size: int, num_splits: int = 0) -> int:
    return int(lib.pa_tree_workspace_size(batch, max_query, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                          page_size, num_splits))


def pa_tree_gqa(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse=None, *, max_query: int,
                scale: float, workspace, granted=None, window: int = 0, num_splits: int = 0, max_context_len=None,
                stream=None) -> None:
    """Attention of drafted trees.  q [T, Hq, D] bf16: the rows' nodes one row after the other, row b's
    from query_start[b] to query_start[b + 1] ([B + 1] int32, at most max_query of them); tree_mask [T]
    int64: bit j set if the node attends to its row's node j; context_lens [B] int32 count the nodes;
    out [T, Hq, D] bf16 and lse [T, Hq] fp32 or None (tokens behind the last row stay as they were);
    pools and block_table as for pa_decode_gqa; workspace: workspace_for_tree(...).  granted: optional [B]
    int32 (pa_plan_step's); a row with 0 has no nodes in the cache, and its outputs stay as they were."""
    _done("pa_tree_gqa", (_native_module or _native()).tree_gqa(
        0, q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, granted, workspace, max_query,
        scale, 1.0, 1.0, window, num_splits, max_context_len, stream))


def pa_tree_gqa_fp8(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse=None, *,
                    max_query: int, scale: float, k_scale: float, v_scale: float, workspace, granted=None,
                    window: int = 0, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """The same over FP8 E4M3 pools [pages, P, Hkv, D] uint8."""
    _done("pa_tree_gqa_fp8", (_native_module or _native()).tree_gqa(
        1, q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, granted, workspace, max_query,
        scale, k_scale, v_scale, window, num_splits, max_context_len, stream))


def pa_tree_gqa_nvfp4(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse=None, *,
                      max_query: int, scale: float, k_scale: float, v_scale: float, workspace, granted=None,
                      window: int = 0, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """The same over NVFP4 pools [pages, P, Hkv, nvfp4_row_bytes(D)] uint8."""
    _done("pa_tree_gqa_nvfp4", (_native_module or _native()).tree_gqa(
        2, q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, granted, workspace, max_query,
        scale, k_scale, v_scale, window, num_splits, max_context_len, stream))


def pa_kv_compact(k_pool, v_pool, block_table, context_lens, query_start, accepted, num_accepted, *, context_lens_out,
                  granted=None, status=None, stream=None) -> None:
    """Accepted path: node accepted[b][i] (i < num_accepted[b]) of row b's tree becomes the row's token
    L - n_b + i, in every layer.  Pools [pages, P, Hkv, R] or [layers, pages, P, Hkv, R] of any format;
    accepted [B, max_accepted] int32 ascending; num_accepted [B] int32; context_lens_out [B] int32 (not
    context_lens itself) gets L - n_b + num_accepted.  granted: optional [B] int32 (pa_plan_step's).  A row
    with 0 there, and one of more than 64 new tokens, which is no tree, is left as it is: context_lens_out = L,
    its path is not read."""
    _done("pa_kv_compact", (_native_module or _native()).kv_compact(
        k_pool, v_pool, block_table, context_lens, query_start, accepted, num_accepted, granted, context_lens_out,
        status, stream))


def pa_stream_workspace_size(batch: int, max_query: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                             max_context_len: int, page_size: int, num_splits: int = 0) -> int:
    return int(lib.pa_stream_workspace_size(batch, max_query, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                            page_size, num_splits))


def pa_stream_gqa(q, k_pool, v_pool, block_table, context_lens, query_start, out, lse=None, *, max_query: int,
                  scale: float, workspace, window: int = 0, first: int = 0, granted=None, num_splits: int = 0,
                  max_context_len=None, stream=None) -> None:
    """Attention of each row's newest tokens: single tokens, chunks of prompts, whole prompts.  q [T, Hq, D]
    bf16: the rows' new tokens one row after the other, row b's from query_start[b] to query_start[b + 1]
    ([B + 1] int32, at most max_query of them); context_lens [B] int32 count them; out [T, Hq, D] bf16 and lse
    [T, Hq] fp32 or None (tokens behind the last row stay as they were); pools and block_table as for
    pa_decode_gqa.  The token at position p attends to those of [0, p]; under a window (> 0) to the `window` most
    recent ones and the row's `first` ones.  workspace: workspace_for_stream(...).  granted: optional [B] int32
    (pa_plan_step's); a row with 0 is left out and its outputs stay as they were.  Single tokens without first
    tokens are faster by pa_decode_gqa."""
    _done("pa_stream_gqa", (_native_module or _native()).stream_gqa(
        0, q, k_pool, v_pool, block_table, context_lens, query_start, out, lse, granted, workspace, max_query, scale,
        1.0, 1.0, window, first, num_splits, max_context_len, stream))


def pa_stream_gqa_fp8(q, k_pool, v_pool, block_table, context_lens, query_start, out, lse=None, *, max_query: int,
                      scale: float, k_scale: float, v_scale: float, workspace, window: int = 0, first: int = 0,
                      granted=None, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """The same over FP8 E4M3 pools [pages, P, Hkv, D] uint8."""
    _done("pa_stream_gqa_fp8", (_native_module or _native()).stream_gqa(
        1, q, k_pool, v_pool, block_table, context_lens, query_start, out, lse, granted, workspace, max_query, scale,
        k_scale, v_scale, window, first, num_splits, max_context_len, stream))


def pa_stream_gqa_nvfp4(q, k_pool, v_pool, block_table, context_lens, query_start, out, lse=None, *, max_query: int,
                        scale: float, k_scale: float, v_scale: float, workspace, window: int = 0, first: int = 0,
                        granted=None, num_splits: int = 0, max_context_len=None, stream=None) -> None:
    """The same over NVFP4 pools [pages, P, Hkv, nvfp4_row_bytes(D)] uint8."""
    _done("pa_stream_gqa_nvfp4", (_native_module or _native()).stream_gqa(
        2, q, k_pool, v_pool, block_table, context_lens, query_start, out, lse, granted, workspace, max_query, scale,
        k_scale, v_scale, window, first, num_splits, max_context_len, stream))


def pa_release_pages(context_lens, held_pages, window_start, free_list, free_count, block_table, *, page_size: int,
                     window: int, first: int = 0, ended=None, context_lens_out=None, held_pages_out=None,
                     window_start_out=None, free_count_out=None, block_table_out=None, status=None,
                     stream=None) -> None:
    """Gives back the pages that no later token sees: those wholly behind the window, but for the pages of the
    row's `first` tokens.  context_lens, held_pages (pa_plan_step's) and window_start [B] int32: a row's pages in
    [ceil(first / page_size), window_start) are gone already (0 for a new row; kept by the caller from step to
    step); free_list [num_pages] int32, a stack of which free_count [1] int32 entries are valid, gets the pages;
    block_table [B, max_pages] int32 gets -1 in their entries.  ended: optional [B] int32, not 0 for a row
    that gives back all it has left (a row that has released pages ends here, not by pa_plan_step).  The _out
    arrays default to their inputs (updated in place).  status: optional int32 device word for PA_DEV_* bits."""
    _done("pa_release_pages", (_native_module or _native()).release_pages(
        context_lens, held_pages, window_start, free_list, free_count, block_table,
        context_lens if context_lens_out is None else context_lens_out,
        held_pages if held_pages_out is None else held_pages_out,
        window_start if window_start_out is None else window_start_out,
        free_count if free_count_out is None else free_count_out,
        block_table if block_table_out is None else block_table_out, ended, status, page_size, window, first, stream))


def pa_read_device_status(workspace, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check(lib.pa_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(bits)),
           "pa_read_device_status")
    return int(bits.value)


def pa_set_profile_events(before=None, after=None) -> None:
    """Record torch.cuda.Event pair around the dominant kernel of later calls (None, None: off)."""
    def handle(ev):
        if ev is None:
            return None
        if ev.cuda_event == 0:  # torch creates the event lazily
            ev.record()
        return ev.cuda_event
    _check(lib.pa_set_profile_events(handle(before), handle(after)), "pa_set_profile_events")


def pa_last_launch_count() -> int:
    return int(lib.pa_last_launch_count())


def pa_set_wait_limit_ns(limit_ns: int = PA_DEFAULT_WAIT_LIMIT_NS) -> None:
    """Limit (global-timer ns) of the GQA split kernels' ring waits for later calls from this thread."""
    _check(lib.pa_set_wait_limit_ns(int(limit_ns)), "pa_set_wait_limit_ns")


def pa_last_cuda_error() -> int:
    return int(lib.pa_last_cuda_error())


def pa_last_cuda_error_string() -> str:
    return lib.pa_last_cuda_error_string().decode()


def workspace_for_gqa(q, k_pool, block_table, num_splits: int = 0, max_context_len=None, device=None):
    """Allocate a uint8 device workspace sized for a pa_decode_gqa call with these tensors."""
    import torch
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    _, P, Hkv, _ = k_pool.shape
    mcl = block_table.shape[1] * P if max_context_len is None else max_context_len
    n = pa_workspace_size(PA_KIND_GQA, B, Hq, Hkv, D, mcl, P, num_splits)
    if n == 0:
        raise PaError(PA_ERR_INVALID_ARGUMENT, "pa_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or q.device)


def workspace_for_mla(q, cache, block_table, num_splits: int = 0, max_context_len=None, device=None):
    import torch
    B, H, _ = q.shape
    _, P, _ = cache.shape
    mcl = block_table.shape[1] * P if max_context_len is None else max_context_len
    n = pa_workspace_size(PA_KIND_MLA_ABSORBED, B, H, 1, 576, mcl, P, num_splits)
    if n == 0:
        raise PaError(PA_ERR_INVALID_ARGUMENT, "pa_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or q.device)


def workspace_for_tree(q, k_pool, block_table, max_query: int, num_splits: int = 0, max_context_len=None, device=None):
    """Allocate a uint8 device workspace sized for a pa_tree_gqa call (of any cache format) with these tensors."""
    import torch
    Hq, D = q.shape[-2], q.shape[-1]
    P, Hkv = k_pool.shape[-3], k_pool.shape[-2]
    mcl = block_table.shape[1] * P if max_context_len is None else max_context_len
    n = pa_tree_workspace_size(block_table.shape[0], max_query, Hq, Hkv, D, mcl, P, num_splits)
    if n == 0:
        raise PaError(PA_ERR_INVALID_ARGUMENT, "pa_tree_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or q.device)


def workspace_for_stream(q, k_pool, block_table, max_query: int, num_splits: int = 0, max_context_len=None, device=None):
    """Allocate a uint8 device workspace sized for a pa_stream_gqa call (of any cache format) with these tensors."""
    import torch
    Hq, D = q.shape[-2], q.shape[-1]
    P, Hkv = k_pool.shape[-3], k_pool.shape[-2]
    mcl = block_table.shape[1] * P if max_context_len is None else max_context_len
    n = pa_stream_workspace_size(block_table.shape[0], max_query, Hq, Hkv, D, mcl, P, num_splits)
    if n == 0:
        raise PaError(PA_ERR_INVALID_ARGUMENT, "pa_stream_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or q.device)
