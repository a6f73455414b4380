"""GB300-native paged decode attention: Python binding of libvt_paged_attn.

The library (``_build/libvt_paged_attn.so``, built by ``build_lib.py``) does
every step of the decode on the GPU; this module only marshals arguments
through ctypes.  Functions named ``vt_*`` mirror the C entry points of
``include/vt_paged_attn.h`` one to one (pointers as Python ints); ``decode``
is a convenience wrapper that takes torch CUDA tensors.  There is no CPU
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from pathlib import Path

LIBRARY_PATH = Path(__file__).resolve().parent / "_build" / "libvt_paged_attn.so"

(VT_OK, VT_ERR_INVALID_ARG, VT_ERR_UNSUPPORTED, VT_ERR_CUDA, VT_ERR_OOM, VT_ERR_DEVICE_TIMEOUT,
 VT_ERR_SCRATCH_LIMIT) = range(7)
VT_BF16, VT_F32, VT_E4M3 = 0, 1, 2
BLOCK_SIZE = 32

EXPORTED = ("vt_paged_attn_decode", "vt_paged_attn_decode_noalloc", "vt_paged_attn_decode_fp8",
            "vt_paged_attn_decode_multi", "vt_paged_attn_decode_multi_fp8",
            "vt_rope_frequencies", "vt_rope", "vt_paged_kv_append", "vt_paged_kv_append_fp8",
            "vt_paged_attn_prefill", "vt_paged_attn_prefill_fp8", "vt_paged_attn_prefill_workspace_bytes",
            "vt_paged_step_tables", "vt_tree_masks", "vt_norm_rope", "vt_paged_kv_norm_append",
            "vt_paged_kv_norm_append_fp8", "vt_paged_attn_prefill_tree", "vt_paged_attn_prefill_tree_fp8",
            "vt_paged_kv_keep_path", "vt_call",
            "vt_paged_attn_last_plan",
            "vt_paged_attn_set_override", "vt_paged_attn_set_overlap", "vt_paged_attn_set_segment_cost",
            "vt_paged_attn_set_workspace", "vt_paged_attn_set_test_wait",
            "vt_paged_attn_device_status", "vt_paged_attn_device_status_detail", "vt_paged_attn_workspace_bytes",
            "vt_paged_attn_release", "vt_status_string", "vt_last_cuda_error", "vt_paged_attn_version")
VT_NOALLOC_SCRATCH_BYTES = 8 << 20
VT_MIN_WORKSPACE_BYTES = 4096
(VT_ROPE_PLAIN, VT_ROPE_LINEAR, VT_ROPE_NTK, VT_ROPE_YARN, VT_ROPE_BANDED) = range(5)


class VtError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: status {status}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class vt_plan(ctypes.Structure):
    _fields_ = [("grid_ctas", ctypes.c_int), ("ctas_per_sm", ctypes.c_int), ("num_sms", ctypes.c_int),
                ("consumer_warps", ctypes.c_int), ("tensor_cores", ctypes.c_int), ("stages", ctypes.c_int), ("group_tile", ctypes.c_int),
                ("subgroups", ctypes.c_int), ("min_units_per_cta", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("smem_bytes", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t), ("launch_overlap", ctypes.c_int),
                ("segment_cost", ctypes.c_int), ("scratch_source", ctypes.c_int), ("q_len", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class vt_rope_stretch(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


_lib = None
_lock = threading.Lock()


def library() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not LIBRARY_PATH.exists():
                raise RuntimeError(
                    f"{LIBRARY_PATH} is missing: build it with "
                    "`python -m paged_attention_decode_kv_gb300.build_lib` (needs nvcc)")
            lib = ctypes.CDLL(str(LIBRARY_PATH))
            c_int, c_void, c_float, c_size = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
            lib.vt_paged_attn_decode.argtypes = [c_void] * 6 + [c_int] * 5 + [c_float, c_int, c_void, c_int,
                                                                               c_int, c_int]
            lib.vt_paged_attn_decode.restype = c_int
            lib.vt_paged_attn_decode_noalloc.argtypes = lib.vt_paged_attn_decode.argtypes
            lib.vt_paged_attn_decode_noalloc.restype = c_int
            lib.vt_paged_attn_decode_fp8.argtypes = [c_void] * 8 + [c_int] * 5 + [c_float, c_int, c_void, c_int,
                                                                                   c_int]
            lib.vt_paged_attn_decode_fp8.restype = c_int
            lib.vt_paged_attn_decode_multi.argtypes = [c_void] * 6 + [c_int] * 6 + [c_float, c_int, c_void, c_int,
                                                                                    c_int, c_int]
            lib.vt_paged_attn_decode_multi.restype = c_int
            lib.vt_paged_attn_decode_multi_fp8.argtypes = [c_void] * 8 + [c_int] * 6 + [c_float, c_int, c_void,
                                                                                         c_int, c_int]
            lib.vt_paged_attn_decode_multi_fp8.restype = c_int
            c_long, c_double = ctypes.c_longlong, ctypes.c_double
            lib.vt_rope_frequencies.argtypes = [ctypes.POINTER(c_double), ctypes.POINTER(c_float), c_int, c_double,
                                                ctypes.POINTER(vt_rope_stretch)]
            lib.vt_rope_frequencies.restype = c_int
            lib.vt_rope.argtypes = [c_void] * 4 + [c_int] * 5 + [c_float, c_long, c_long, c_void, c_int]
            lib.vt_rope.restype = c_int
            tail = [c_int] * 8 + [c_float, c_long, c_long, c_long, c_void, c_int, c_int]
            lib.vt_paged_kv_append.argtypes = [c_void] * 11 + tail + [c_int]
            lib.vt_paged_kv_append.restype = c_int
            lib.vt_paged_kv_append_fp8.argtypes = [c_void] * 13 + tail
            lib.vt_paged_kv_append_fp8.restype = c_int
            tail = [c_int] * 6 + [c_float, c_int, c_void, c_int, c_int]
            lib.vt_paged_attn_prefill.argtypes = [c_void] * 7 + tail + [c_int]
            lib.vt_paged_attn_prefill.restype = c_int
            lib.vt_paged_attn_prefill_fp8.argtypes = [c_void] * 9 + tail
            lib.vt_paged_attn_prefill_fp8.restype = c_int
            lib.vt_paged_attn_prefill_workspace_bytes.argtypes = [c_int, c_int]
            lib.vt_paged_attn_prefill_workspace_bytes.restype = c_size
            lib.vt_paged_step_tables.argtypes = [c_void] * 9 + [c_int] * 3 + [c_void] + [c_int] * 2
            lib.vt_paged_step_tables.restype = c_int
            lib.vt_tree_masks.argtypes = [c_void] * 5 + [c_int] * 3 + [c_void]
            lib.vt_tree_masks.restype = c_int
            lib.vt_norm_rope.argtypes = [c_void] * 5 + [c_int] * 5 + [c_float] * 2 + [c_long] * 3 + [c_void, c_int]
            lib.vt_norm_rope.restype = c_int
            tail = [c_int] * 8 + [c_float] * 2 + [c_long] * 5 + [c_void, c_int, c_int]
            lib.vt_paged_kv_norm_append.argtypes = [c_void] * 13 + tail + [c_int]
            lib.vt_paged_kv_norm_append.restype = c_int
            lib.vt_paged_kv_norm_append_fp8.argtypes = [c_void] * 15 + tail
            lib.vt_paged_kv_norm_append_fp8.restype = c_int
            tail = [c_int] * 7 + [c_float, c_int, c_void, c_int, c_int]
            lib.vt_paged_attn_prefill_tree.argtypes = [c_void] * 8 + tail + [c_int]
            lib.vt_paged_attn_prefill_tree.restype = c_int
            lib.vt_paged_attn_prefill_tree_fp8.argtypes = [c_void] * 10 + tail
            lib.vt_paged_attn_prefill_tree_fp8.restype = c_int
            lib.vt_paged_kv_keep_path.argtypes = [c_void] * 8 + [c_int] * 7 + [c_long] * 2 + [c_void] + [c_int] * 3
            lib.vt_paged_kv_keep_path.restype = c_int
            lib.vt_call.argtypes = [ctypes.c_char_p]
            lib.vt_call.restype = c_int
            lib.vt_paged_attn_last_plan.argtypes = [ctypes.POINTER(vt_plan)]
            lib.vt_paged_attn_last_plan.restype = c_int
            lib.vt_paged_attn_set_override.argtypes = [c_int, c_int]
            lib.vt_paged_attn_set_override.restype = c_int
            lib.vt_paged_attn_set_overlap.argtypes = [c_int]
            lib.vt_paged_attn_set_overlap.restype = c_int
            lib.vt_paged_attn_set_segment_cost.argtypes = [c_int]
            lib.vt_paged_attn_set_segment_cost.restype = c_int
            lib.vt_paged_attn_set_workspace.argtypes = [c_void, c_size, c_void]
            lib.vt_paged_attn_set_workspace.restype = c_int
            lib.vt_paged_attn_set_test_wait.argtypes = [ctypes.c_longlong, c_int, c_int]
            lib.vt_paged_attn_set_test_wait.restype = c_int
            lib.vt_paged_attn_device_status.argtypes = [c_void, ctypes.POINTER(ctypes.c_uint)]
            lib.vt_paged_attn_device_status.restype = c_int
            lib.vt_paged_attn_device_status_detail.argtypes = [c_void, ctypes.POINTER(ctypes.c_uint), c_int]
            lib.vt_paged_attn_device_status_detail.restype = c_int
            lib.vt_paged_attn_workspace_bytes.argtypes = [c_int] * 5
            lib.vt_paged_attn_workspace_bytes.restype = c_size
            lib.vt_paged_attn_release.argtypes = []
            lib.vt_paged_attn_release.restype = None
            lib.vt_status_string.argtypes = [c_int]
            lib.vt_status_string.restype = ctypes.c_char_p
            lib.vt_last_cuda_error.argtypes = []
            lib.vt_last_cuda_error.restype = ctypes.c_char_p
            lib.vt_paged_attn_version.argtypes = []
            lib.vt_paged_attn_version.restype = c_int
            _lib = lib
    return _lib


def _check(status: int, where: str) -> None:
    if status != VT_OK:
        lib = library()
        detail = lib.vt_status_string(status).decode()
        cuda = lib.vt_last_cuda_error().decode()
        if cuda:
            detail += f"; {cuda}"
        raise VtError(status, where, detail)


# ---- C entry points, same names -------------------------------------------
def vt_paged_attn_decode(out, q, k_cache, v_cache, block_tables, context_lens, num_seqs, num_q_heads,
                         num_kv_heads, head_dim, block_size, scale, window, stream, max_blocks_per_seq,
                         num_blocks, dtype) -> int:
    """Raw call: pointers and the stream handle are ints; returns the status code."""
    return library().vt_paged_attn_decode(out, q, k_cache, v_cache, block_tables, context_lens, num_seqs,
                                          num_q_heads, num_kv_heads, head_dim, block_size, float(scale),
                                          int(window), stream, max_blocks_per_seq, num_blocks, dtype)


def vt_paged_attn_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, num_seqs, num_q_heads,
                                 num_kv_heads, head_dim, block_size, scale, window, stream, max_blocks_per_seq,
                                 num_blocks, dtype) -> int:
    """Raw call of the allocation-free entry point (scratch in a fixed static
    device array instead of a library allocation); returns the status code."""
    return library().vt_paged_attn_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                                                  num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                  float(scale), int(window), stream, max_blocks_per_seq,
                                                  num_blocks, dtype)


def vt_paged_attn_decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, num_seqs, q_len, num_q_heads,
                               num_kv_heads, head_dim, block_size, scale, window, stream, max_blocks_per_seq,
                               num_blocks, dtype) -> int:
    """Raw call of the multi-token decode (q_len new tokens per sequence,
    causal within them); returns the status code."""
    return library().vt_paged_attn_decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, num_seqs,
                                                q_len, num_q_heads, num_kv_heads, head_dim, block_size, float(scale),
                                                int(window), stream, max_blocks_per_seq, num_blocks, dtype)


def vt_paged_attn_decode_multi_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                   num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, scale, window,
                                   stream, max_blocks_per_seq, num_blocks) -> int:
    """Raw call of the multi-token decode over an FP8 (E4M3) KV cache; returns
    the status code."""
    return library().vt_paged_attn_decode_multi_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                                    context_lens, num_seqs, q_len, num_q_heads, num_kv_heads,
                                                    head_dim, block_size, float(scale), int(window), stream,
                                                    max_blocks_per_seq, num_blocks)


def vt_paged_attn_decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, num_seqs,
                             num_q_heads, num_kv_heads, head_dim, block_size, scale, window, stream,
                             max_blocks_per_seq, num_blocks) -> int:
    """Raw call of the FP8 (E4M3) KV-cache decode; returns the status code."""
    return library().vt_paged_attn_decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                              context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                              block_size, float(scale), int(window), stream, max_blocks_per_seq,
                                              num_blocks)


def vt_rope_frequencies(rot_dim, base, stretch=None):
    """(status, list of rot_dim // 2 radians per token, amplitude); stretch is
    a vt_rope_stretch or None."""
    inv = (ctypes.c_double * max(1, rot_dim // 2))()
    amplitude = ctypes.c_float(0.0)
    st = library().vt_rope_frequencies(inv, ctypes.byref(amplitude), rot_dim, float(base),
                                       ctypes.byref(stretch) if stretch is not None else None)
    return st, list(inv)[:max(0, rot_dim // 2)], float(amplitude.value)


def vt_rope(out, x, positions, inv_freq, num_tokens, num_heads, head_dim, rot_dim, interleaved, amplitude, x_stride,
            out_stride, stream, dtype) -> int:
    """Raw call of the rotary positions; returns the status code."""
    return library().vt_rope(out, x, positions, inv_freq, num_tokens, num_heads, head_dim, rot_dim, int(interleaved),
                             float(amplitude), x_stride, out_stride, stream, dtype)


def vt_paged_kv_append(k_cache, v_cache, q_out, k, v, q, q_starts, block_tables, context_lens, positions, inv_freq,
                       num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, rot_dim, interleaved,
                       amplitude, q_stride, k_stride, v_stride, stream, max_blocks_per_seq, num_blocks, dtype) -> int:
    """Raw call of the append to the paged cache; returns the status code."""
    return library().vt_paged_kv_append(k_cache, v_cache, q_out, k, v, q, q_starts, block_tables, context_lens,
                                        positions, inv_freq, num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                        head_dim, block_size, rot_dim, int(interleaved), float(amplitude), q_stride,
                                        k_stride, v_stride, stream, max_blocks_per_seq, num_blocks, dtype)


def vt_paged_kv_append_fp8(k_cache, v_cache, q_out, k, v, q, k_scale, v_scale, q_starts, block_tables, context_lens,
                           positions, inv_freq, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                           rot_dim, interleaved, amplitude, q_stride, k_stride, v_stride, stream, max_blocks_per_seq,
                           num_blocks) -> int:
    """Raw call of the append to an FP8 (E4M3) cache; returns the status code."""
    return library().vt_paged_kv_append_fp8(k_cache, v_cache, q_out, k, v, q, k_scale, v_scale, q_starts,
                                            block_tables, context_lens, positions, inv_freq, num_seqs, num_tokens,
                                            num_q_heads, num_kv_heads, head_dim, block_size, rot_dim,
                                            int(interleaved), float(amplitude), q_stride, k_stride, v_stride, stream,
                                            max_blocks_per_seq, num_blocks)


def vt_paged_attn_prefill(out, q, k_cache, v_cache, q_starts, block_tables, context_lens, num_seqs, num_tokens,
                          num_q_heads, num_kv_heads, head_dim, block_size, scale, window, stream, max_blocks_per_seq,
                          num_blocks, dtype) -> int:
    """Raw call of the ragged prefill; returns the status code."""
    return library().vt_paged_attn_prefill(out, q, k_cache, v_cache, q_starts, block_tables, context_lens, num_seqs,
                                           num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, float(scale),
                                           int(window), stream, max_blocks_per_seq, num_blocks, dtype)


def vt_paged_attn_prefill_fp8(out, q, k_cache, v_cache, k_scale, v_scale, q_starts, block_tables, context_lens,
                              num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, scale, window,
                              stream, max_blocks_per_seq, num_blocks) -> int:
    """Raw call of the ragged prefill over an FP8 (E4M3) cache; returns the
    status code."""
    return library().vt_paged_attn_prefill_fp8(out, q, k_cache, v_cache, k_scale, v_scale, q_starts, block_tables,
                                               context_lens, num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                               head_dim, block_size, float(scale), int(window), stream,
                                               max_blocks_per_seq, num_blocks)


def vt_paged_attn_prefill_workspace_bytes(head_dim, dtype) -> int:
    return int(library().vt_paged_attn_prefill_workspace_bytes(head_dim, dtype))


def vt_paged_step_tables(block_tables, context_lens, free_pages, counters, q_starts, positions, slots, keep_lens,
                         new_lens, num_seqs, num_tokens, block_size, stream, max_blocks_per_seq, num_blocks) -> int:
    """Raw call of the step's page tables; returns the status code."""
    return library().vt_paged_step_tables(block_tables, context_lens, free_pages, counters, q_starts, positions,
                                          slots, keep_lens, new_lens, num_seqs, num_tokens, block_size, stream,
                                          max_blocks_per_seq, num_blocks)


def vt_tree_masks(masks, positions, parents, q_starts, context_lens, num_seqs, num_tokens, mask_words, stream) -> int:
    """Raw call of the drafted trees' masks; returns the status code."""
    return library().vt_tree_masks(masks, positions, parents, q_starts, context_lens, num_seqs, num_tokens,
                                   mask_words, stream)


def vt_norm_rope(out, x, weight, positions, inv_freq, num_tokens, num_heads, head_dim, rot_dim, interleaved,
                 amplitude, eps, x_stride, out_stride, weight_stride, stream, dtype) -> int:
    """Raw call of the heads' norm and rotation; returns the status code."""
    return library().vt_norm_rope(out, x, weight, positions, inv_freq, num_tokens, num_heads, head_dim, rot_dim,
                                  int(interleaved), float(amplitude), float(eps), x_stride, out_stride,
                                  weight_stride, stream, dtype)


def vt_paged_kv_norm_append(k_cache, v_cache, q_out, k, v, q, k_weight, q_weight, q_starts, block_tables,
                            context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads, num_kv_heads,
                            head_dim, block_size, rot_dim, interleaved, amplitude, eps, q_stride, k_stride, v_stride,
                            q_weight_stride, k_weight_stride, stream, max_blocks_per_seq, num_blocks, dtype) -> int:
    """Raw call of the append of normed queries and keys; returns the status code."""
    return library().vt_paged_kv_norm_append(k_cache, v_cache, q_out, k, v, q, k_weight, q_weight, q_starts,
                                             block_tables, context_lens, positions, inv_freq, num_seqs, num_tokens,
                                             num_q_heads, num_kv_heads, head_dim, block_size, rot_dim,
                                             int(interleaved), float(amplitude), float(eps), q_stride, k_stride,
                                             v_stride, q_weight_stride, k_weight_stride, stream, max_blocks_per_seq,
                                             num_blocks, dtype)


def vt_paged_kv_norm_append_fp8(k_cache, v_cache, q_out, k, v, q, k_weight, q_weight, k_scale, v_scale, q_starts,
                                block_tables, context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                num_kv_heads, head_dim, block_size, rot_dim, interleaved, amplitude, eps, q_stride,
                                k_stride, v_stride, q_weight_stride, k_weight_stride, stream, max_blocks_per_seq,
                                num_blocks) -> int:
    """Raw call of the append of normed queries and keys to an FP8 (E4M3)
    cache; returns the status code."""
    return library().vt_paged_kv_norm_append_fp8(k_cache, v_cache, q_out, k, v, q, k_weight, q_weight, k_scale,
                                                 v_scale, q_starts, block_tables, context_lens, positions, inv_freq,
                                                 num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                                 block_size, rot_dim, int(interleaved), float(amplitude), float(eps),
                                                 q_stride, k_stride, v_stride, q_weight_stride, k_weight_stride,
                                                 stream, max_blocks_per_seq, num_blocks)


def vt_paged_attn_prefill_tree(out, q, k_cache, v_cache, masks, q_starts, block_tables, context_lens, num_seqs,
                               num_tokens, mask_words, num_q_heads, num_kv_heads, head_dim, block_size, scale, window,
                               stream, max_blocks_per_seq, num_blocks, dtype) -> int:
    """Raw call of the drafted trees' attention; returns the status code."""
    return library().vt_paged_attn_prefill_tree(out, q, k_cache, v_cache, masks, q_starts, block_tables,
                                                context_lens, num_seqs, num_tokens, mask_words, num_q_heads,
                                                num_kv_heads, head_dim, block_size, float(scale), int(window), stream,
                                                max_blocks_per_seq, num_blocks, dtype)


def vt_paged_attn_prefill_tree_fp8(out, q, k_cache, v_cache, k_scale, v_scale, masks, q_starts, block_tables,
                                   context_lens, num_seqs, num_tokens, mask_words, num_q_heads, num_kv_heads,
                                   head_dim, block_size, scale, window, stream, max_blocks_per_seq,
                                   num_blocks) -> int:
    """Raw call of the drafted trees' attention over an FP8 (E4M3) cache;
    returns the status code."""
    return library().vt_paged_attn_prefill_tree_fp8(out, q, k_cache, v_cache, k_scale, v_scale, masks, q_starts,
                                                    block_tables, context_lens, num_seqs, num_tokens, mask_words,
                                                    num_q_heads, num_kv_heads, head_dim, block_size, float(scale),
                                                    int(window), stream, max_blocks_per_seq, num_blocks)


def vt_paged_kv_keep_path(k_cache, v_cache, kept_lens, accepted, masks, q_starts, block_tables, context_lens,
                          num_seqs, num_tokens, mask_words, num_layers, num_kv_heads, head_dim, block_size,
                          k_layer_stride, v_layer_stride, stream, max_blocks_per_seq, num_blocks, dtype) -> int:
    """Raw call that moves accepted branches to consecutive slots; returns the
    status code."""
    return library().vt_paged_kv_keep_path(k_cache, v_cache, kept_lens, accepted, masks, q_starts, block_tables,
                                           context_lens, num_seqs, num_tokens, mask_words, num_layers, num_kv_heads,
                                           head_dim, block_size, k_layer_stride, v_layer_stride, stream,
                                           max_blocks_per_seq, num_blocks, dtype)


def vt_call(args) -> int:
    """Raw call of an operator by its arguments in 8-byte slots (bytes, see
    vt_op and vt_arg); returns the status code."""
    return library().vt_call(args)


def vt_paged_attn_last_plan() -> dict:
    p = vt_plan()
    _check(library().vt_paged_attn_last_plan(ctypes.byref(p)), "vt_paged_attn_last_plan")
    return p.as_dict()


def vt_paged_attn_set_override(grid_ctas: int = 0, min_units_per_cta: int = 0) -> None:
    """Force the CTA count and/or the minimum work per CTA (0: automatic)."""
    _check(library().vt_paged_attn_set_override(grid_ctas, min_units_per_cta), "vt_paged_attn_set_override")


def vt_paged_attn_set_overlap(enabled: bool) -> None:
    """Launch decodes as programmatic dependents of the previous kernel on the
    stream (that kernel must not write context_lens or block_tables)."""
    _check(library().vt_paged_attn_set_overlap(1 if enabled else 0), "vt_paged_attn_set_overlap")


def vt_paged_attn_set_segment_cost(tiles: int = -1) -> None:
    """Partition weight of a (sequence, kv head) boundary in tiles (-1: default, 2; 6 for FP8 or multi-token)."""
    _check(library().vt_paged_attn_set_segment_cost(tiles), "vt_paged_attn_set_segment_cost")


def vt_paged_attn_set_workspace(dev_ptr: int, nbytes: int, stream=None) -> None:
    """Use caller-owned device memory [dev_ptr, dev_ptr + nbytes) as the split
    workspace of the current device (dev_ptr 0: back to the library's own)."""
    _check(library().vt_paged_attn_set_workspace(dev_ptr or None, nbytes, _stream_handle(stream)),
           "vt_paged_attn_set_workspace")


def vt_paged_attn_set_test_wait(wait_limit_cycles: int = 0, withhold_cta: int = -1, withhold_tile: int = -1) -> None:
    """Test hook: shorten the kernel's bounded waits and make one CTA withhold
    a tile, so a wait gives up (0, -1, -1 restores normal operation)."""
    _check(library().vt_paged_attn_set_test_wait(wait_limit_cycles, withhold_cta, withhold_tile),
           "vt_paged_attn_set_test_wait")


def vt_paged_attn_device_status(stream=None) -> int:
    """Status word of bounded waits that gave up (0 = none); clears it."""
    word = ctypes.c_uint(0)
    library().vt_paged_attn_device_status(_stream_handle(stream), ctypes.byref(word))
    return int(word.value)


def vt_paged_attn_device_status_detail(stream=None, n_words: int = 5) -> list:
    """First n_words of the device status area (not cleared): status bits, then
    where the first bounded wait that gave up was (1 + CTA, bit | thread << 8,
    barrier address, parity)."""
    words = (ctypes.c_uint * n_words)()
    _check(library().vt_paged_attn_device_status_detail(_stream_handle(stream), words, n_words),
           "vt_paged_attn_device_status_detail")
    return [int(x) for x in words]


def vt_paged_attn_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, dtype) -> int:
    return int(library().vt_paged_attn_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, dtype))


def vt_paged_attn_release() -> None:
    library().vt_paged_attn_release()


def vt_status_string(status: int) -> str:
    return library().vt_status_string(status).decode()


def vt_paged_attn_version() -> int:
    return int(library().vt_paged_attn_version())


# ---- torch convenience -------------------------------------------------------
def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return VT_BF16
    if t.dtype == torch.float32:
        return VT_F32
    raise TypeError(f"storage dtype must be bfloat16 or float32, got {t.dtype}")


def decode(q, k_cache, v_cache, block_tables, context_lens, scale=None, window: int = 0, out=None,
           stream=None):
    """Decode attention for torch CUDA tensors.

    q [B][Hq][D]; k_cache, v_cache [num_blocks][32][Hkv][D]; block_tables
    [B][max_blocks] int32; context_lens [B] int32.  Returns out [B][Hq][D]
    (allocated unless given).  Asynchronous on ``stream`` (default: current).
    """
    import torch
    B, Hq, D = q.shape
    nb, P, Hkv, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache/v_cache must be [num_blocks][32][Hkv][head_dim] matching q")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_tables", block_tables),
                    ("context_lens", context_lens)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor shaped and typed like q")
    if scale is None:
        scale = D ** -0.5
    st = vt_paged_attn_decode(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                              block_tables.data_ptr(), context_lens.data_ptr(), B, Hq, Hkv, D, P, scale,
                              window, _stream_handle(stream), block_tables.shape[1], nb, dtype_code(q))
    _check(st, "vt_paged_attn_decode")
    return out


def decode_fp8(q, k_codes, v_codes, k_scale, v_scale, block_tables, context_lens, scale=None, window: int = 0,
               out=None, stream=None):
    """Decode attention over an FP8 (E4M3) KV cache, for torch CUDA tensors.

    q [B][Hq][D] bf16, or [B][q_len][Hq][D] for several new tokens per
    sequence (vt_paged_attn_decode_multi_fp8); k_codes, v_codes
    [num_blocks][32][Hkv][D] uint8 E4M3 codes (or torch.float8_e4m3fn);
    k_scale, v_scale [Hkv] float32.  Returns out shaped like q, bf16
    (allocated unless given).  Asynchronous on ``stream``.
    """
    import torch
    if q.dim() == 4:
        B, q_len, Hq, D = q.shape
    else:
        B, Hq, D = q.shape
        q_len = 0
    if k_codes.dtype == torch.float8_e4m3fn:
        k_codes = k_codes.view(torch.uint8)
    if v_codes.dtype == torch.float8_e4m3fn:
        v_codes = v_codes.view(torch.uint8)
    nb, P, Hkv, D2 = k_codes.shape
    if D2 != D or v_codes.shape != k_codes.shape:
        raise ValueError("k_codes/v_codes must be [num_blocks][32][Hkv][head_dim] matching q")
    for name, t in (("q", q), ("k_codes", k_codes), ("v_codes", v_codes), ("k_scale", k_scale),
                    ("v_scale", v_scale), ("block_tables", block_tables), ("context_lens", context_lens)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dtype != torch.bfloat16 or k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8:
        raise TypeError("q must be bfloat16 and the caches uint8 E4M3 codes")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or k_scale.numel() != Hkv or \
            v_scale.numel() != Hkv:
        raise TypeError("k_scale and v_scale must be float32 [num_kv_heads]")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor shaped and typed like q")
    if scale is None:
        scale = D ** -0.5
    if q_len:
        st = vt_paged_attn_decode_multi_fp8(out.data_ptr(), q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                                            k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(),
                                            context_lens.data_ptr(), B, q_len, Hq, Hkv, D, P, scale, window,
                                            _stream_handle(stream), block_tables.shape[1], nb)
        _check(st, "vt_paged_attn_decode_multi_fp8")
    else:
        st = vt_paged_attn_decode_fp8(out.data_ptr(), q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                                      k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(),
                                      context_lens.data_ptr(), B, Hq, Hkv, D, P, scale, window,
                                      _stream_handle(stream), block_tables.shape[1], nb)
        _check(st, "vt_paged_attn_decode_fp8")
    return out


def decode_multi(q, k_cache, v_cache, block_tables, context_lens, scale=None, window: int = 0, out=None,
                 stream=None):
    """Multi-token decode for torch CUDA tensors: q [B][q_len][Hq][D]; the new
    tokens are the last q_len of each sequence's context_lens[b] cached tokens
    and attend causally.  Returns out [B][q_len][Hq][D]."""
    import torch
    B, q_len, Hq, D = q.shape
    nb, P, Hkv, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache/v_cache must be [num_blocks][32][Hkv][head_dim] matching q")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_tables", block_tables),
                    ("context_lens", context_lens)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor shaped and typed like q")
    if scale is None:
        scale = D ** -0.5
    st = vt_paged_attn_decode_multi(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                    block_tables.data_ptr(), context_lens.data_ptr(), B, q_len, Hq, Hkv, D, P,
                                    scale, window, _stream_handle(stream), block_tables.shape[1], nb,
                                    dtype_code(q))
    _check(st, "vt_paged_attn_decode_multi")
    return out


def rope_frequencies(rot_dim: int, base: float = 10000.0, kind: int = VT_ROPE_PLAIN, factor: float = 1.0,
                     original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Frequencies for ``rope`` and ``append``: (inv_freq float64 [rot_dim / 2]
    on ``device``, amplitude).  ``kind`` is a VT_ROPE_* stretch for contexts
    longer than the trained one (vt_rope_frequencies)."""
    import torch
    st, inv, amplitude = vt_rope_frequencies(
        rot_dim, base, vt_rope_stretch(kind, factor, original_context, beta_fast, beta_slow))
    _check(st, "vt_rope_frequencies")
    return torch.tensor(inv, dtype=torch.float64, device=device), amplitude


_torch = None


def _t():
    """torch, imported at the first call that takes tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


# The checks below run on every call of operators that take a few microseconds
# on the GPU: plain comparisons, no helper objects.
def _row_stride(name, t, T, H, D, dtype, index):
    """Checks packed rows [T][H][D] whose heads are contiguous; the token
    stride in elements."""
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != (T, H, D):
        raise ValueError(f"{name} must be [{T}][{H}][{D}], got {tuple(t.shape)}")
    row, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{name} must have contiguous heads (only the token stride is free)")
    return row if T > 1 else H * D


def _check_plain(name, t, dtype, index):
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_ragged(torch, k_cache, v_cache, kv, q_starts, block_tables, context_lens, index):
    """(num_seqs, max_blocks) of a ragged batch over caches of type kv."""
    int32 = torch.int32
    # (in line what _check_plain says of each: five calls cost a microsecond)
    if not (k_cache.get_device() == v_cache.get_device() == q_starts.get_device() == block_tables.get_device()
            == context_lens.get_device() == index and k_cache.dtype is kv and v_cache.dtype is kv
            and q_starts.dtype is int32 and block_tables.dtype is int32 and context_lens.dtype is int32
            and k_cache.is_contiguous() and v_cache.is_contiguous() and q_starts.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()):
        _check_plain("k_cache", k_cache, kv, index)
        _check_plain("v_cache", v_cache, kv, index)
        _check_plain("q_starts", q_starts, int32, index)
        _check_plain("block_tables", block_tables, int32, index)
        _check_plain("context_lens", context_lens, int32, index)
    B = context_lens.numel()
    if q_starts.numel() != B + 1 or block_tables.dim() != 2:
        raise ValueError("q_starts must be [num_seqs + 1] and block_tables [num_seqs][max_blocks]")
    rows, max_blocks = block_tables.shape
    if rows != B:
        raise ValueError("q_starts must be [num_seqs + 1] and block_tables [num_seqs][max_blocks]")
    return B, max_blocks


def _check_scales(torch, k_scale, v_scale, heads, index):
    _check_plain("k_scale", k_scale, torch.float32, index)
    _check_plain("v_scale", v_scale, torch.float32, index)
    if k_scale.numel() != heads or v_scale.numel() != heads:
        raise TypeError("k_scale and v_scale must be float32 [num_kv_heads]")


def _codes(torch, k, v):
    """Caches of codes, of one type (whose name does not matter: a view takes 3 us)."""
    dtype = k.dtype
    if dtype is v.dtype and (dtype is torch.float8_e4m3fn or dtype is torch.uint8):
        return k, v
    for t in (k, v):
        if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
            raise TypeError("the caches must be uint8 or float8_e4m3fn E4M3 codes")
    return k.view(torch.uint8), v.view(torch.uint8)


def _check_freq(torch, inv_freq, index):
    """(pointer, rot_dim) of a frequency table, or of none."""
    if inv_freq is None:
        return 0, 0
    if not (inv_freq.dtype is torch.float64 and inv_freq.get_device() == index and inv_freq.is_contiguous()):
        _check_plain("inv_freq", inv_freq, torch.float64, index)
    n = inv_freq.numel()
    return (inv_freq.data_ptr(), 2 * n) if n else (0, 0)


def _cuda_index(name, t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _io_code(torch, dtype):
    if dtype is torch.bfloat16:
        return VT_BF16
    if dtype is torch.float32:
        return VT_F32
    raise TypeError(f"storage dtype must be bfloat16 or float32, got {dtype}")


def _launch(torch, index, stream, where, call, before, after):
    """call(*before, stream handle, *after) with the tensors' device current;
    raises VtError."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_on(torch, index, stream)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            status = call(*before, handle, *after)
    else:
        status = call(*before, handle, *after)
    if status != VT_OK:
        _check(status, where)


# vt_call's arguments: the operator, their number, and each operator's own (the stream's handle among them).
_TAIL = "8q2d8q"
_STEP_TABLES, _TREE_MASKS = (1, 15, struct.Struct("17q")), (2, 9, struct.Struct("11q"))
_NORM_ROPE = 3, 17, struct.Struct("12q2d5q")
_NORM_APPEND, _NORM_APPEND_FP8 = (4, 32, struct.Struct("15q" + _TAIL + "q")), (5, 33, struct.Struct("17q" + _TAIL))
_PREFILL_TREE, _PREFILL_TREE_FP8 = (6, 21, struct.Struct("17qd5q")), (7, 22, struct.Struct("19qd4q"))
_KEEP_PATH = 8, 21, struct.Struct("23q")


def _launch_packed(torch, index, stream, where, op, before, after):
    """``_launch`` through vt_call (0 for a null pointer): ctypes takes 0.1 us an argument."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_on(torch, index, stream)
    number, count, layout = op
    args = layout.pack(number, count, *before, handle, *after)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            status = library().vt_call(args)
    else:
        status = library().vt_call(args)
    if status != VT_OK:
        _check(status, where)


def _empty_on(torch, shape, dtype, index, stream):
    """Memory of the stream that will write it: a block that the current
    stream has given back may still be read there."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=index)


def _stream_on(torch, index, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def rope(x, positions, inv_freq, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Rotary positions on torch CUDA tensors.

    x [T][H][D] bf16 or fp32 (token stride free, e.g. the queries of a fused
    projection); positions [T] int32; inv_freq float64 [rot_dim / 2] (see
    ``rope_frequencies``).  Returns out [T][H][D] (allocated unless given; x
    itself rotates in place).  A negative position turns back, so the gradient
    of ``rope(x, p)`` is ``rope(grad, -p)``.  Asynchronous on ``stream``, whose
    memory an allocated result is."""
    torch = _t()
    index = _cuda_index("x", x)
    io = x.dtype
    code = _io_code(torch, io)
    T, H, D = x.shape
    x_stride = _row_stride("x", x, T, H, D, io, index)
    _check_plain("positions", positions, torch.int32, index)
    if positions.numel() != T:
        raise ValueError("positions must be [tokens]")
    freq, rot = _check_freq(torch, inv_freq, index)
    if out is None:
        out = torch.empty((T, H, D), dtype=io, device=x.device) if stream is None else \
            _empty_on(torch, (T, H, D), io, index, stream)
    out_stride = _row_stride("out", out, T, H, D, io, index)
    _launch(torch, index, stream, "vt_rope", library().vt_rope,
            (out.data_ptr(), x.data_ptr(), positions.data_ptr(), freq, T, H, D, rot, 1 if interleaved else 0, amplitude,
             x_stride, out_stride), (code,))
    return out


def _append(torch, k, v, k_cache, v_cache, scales, q_starts, block_tables, context_lens, q, q_out, positions,
            inv_freq, interleaved, amplitude, stream, norm=None):
    index = _cuda_index("k", k)
    T, Hkv, D = k.shape
    fp8 = scales is not None
    io = torch.bfloat16 if fp8 else k_cache.dtype
    code = 0 if fp8 else _io_code(torch, io)
    ks = _row_stride("k", k, T, Hkv, D, io, index)
    vs = _row_stride("v", v, T, Hkv, D, io, index)
    B, max_blocks = _check_ragged(torch, k_cache, v_cache, k_cache.dtype, q_starts, block_tables, context_lens, index)
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != Hkv or shape[3] != D or v_cache.shape != shape:
        raise ValueError("k_cache/v_cache must be [num_blocks][32][Hkv][head_dim] matching k")
    freq, rot = _check_freq(torch, inv_freq, index)
    Hq = qs = 0
    q_ptr = out_ptr = pos_ptr = 0
    if q is not None:
        Hq = q.shape[1]
        qs = _row_stride("q", q, T, Hq, D, io, index)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=io, device=q.device) if stream is None else \
                _empty_on(torch, (T, Hq, D), io, index, stream)
        else:
            _check_plain("q_out", q_out, io, index)
            if q_out.shape != q.shape:
                raise ValueError("q_out must be shaped like q")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if positions is not None:
        _check_plain("positions", positions, torch.int32, index)
        if positions.numel() != T:
            raise ValueError("positions must be [tokens]")
        pos_ptr = positions.data_ptr()
    head = (k_cache.data_ptr(), v_cache.data_ptr(), out_ptr, k.data_ptr(), v.data_ptr(), q_ptr)
    rest = (q_starts.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), pos_ptr, freq, B, T, Hq, Hkv, D,
            shape[1], rot, 1 if interleaved else 0, amplitude)
    if norm is None:
        rest += (qs, ks, vs)
    else:
        k_weight, q_weight, eps = norm
        kw, kw_stride = _weight(torch, "k_weight", k_weight, Hkv, D, index)
        qw, qw_stride = (0, 0) if q is None else _weight(torch, "q_weight", q_weight, Hq, D, index)
        head += (kw, qw)
        rest += (eps, qs, ks, vs, qw_stride, kw_stride)
        if fp8:
            _check_scales(torch, *scales, Hkv, index)
            _launch_packed(torch, index, stream, "vt_paged_kv_norm_append_fp8", _NORM_APPEND_FP8,
                           head + (scales[0].data_ptr(), scales[1].data_ptr()) + rest, (max_blocks, shape[0]))
        else:
            _launch_packed(torch, index, stream, "vt_paged_kv_norm_append", _NORM_APPEND, head + rest,
                           (max_blocks, shape[0], code))
        return q_out
    if fp8:
        _check_scales(torch, *scales, Hkv, index)
        _launch(torch, index, stream, "vt_paged_kv_append_fp8", library().vt_paged_kv_append_fp8,
                head + (scales[0].data_ptr(), scales[1].data_ptr()) + rest, (max_blocks, shape[0]))
    else:
        _launch(torch, index, stream, "vt_paged_kv_append", library().vt_paged_kv_append, head + rest,
                (max_blocks, shape[0], code))
    return q_out


def append(k, v, k_cache, v_cache, q_starts, block_tables, context_lens, q=None, q_out=None, positions=None,
           inv_freq=None, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """Writes the keys and values of new tokens into the paged cache, keys and
    queries rotated on the way.

    k, v [T][Hkv][D] and q [T][Hq][D] (token strides free); sequence b owns
    rows q_starts[b]:q_starts[b + 1], the last of its context_lens[b] tokens;
    caches [num_blocks][32][Hkv][D] of the rows' type.  Rotates at each
    token's place in its context, or at positions [T]; without inv_freq it
    rotates nothing.  Returns the rotated queries [T][Hq][D] (q_out, allocated
    unless given; None without q).  Asynchronous on ``stream``, whose memory
    an allocated result is."""
    return _append(_t(), k, v, k_cache, v_cache, None, q_starts, block_tables, context_lens, q, q_out, positions,
                   inv_freq, interleaved, amplitude, stream)


def append_fp8(k, v, k_codes, v_codes, k_scale, v_scale, q_starts, block_tables, context_lens, q=None, q_out=None,
               positions=None, inv_freq=None, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """``append`` into an FP8 (E4M3) cache of codes with a scale per kv head
    (rows bf16; codes uint8 or torch.float8_e4m3fn)."""
    torch = _t()
    return _append(torch, k, v, *_codes(torch, k_codes, v_codes), (k_scale, v_scale), q_starts,
                   block_tables, context_lens, q, q_out, positions, inv_freq, interleaved, amplitude, stream)


def _given(name, t):
    if t is None:
        raise ValueError(f"{name} must be given")
    return t


def _weight(torch, name, weight, H, D, index):
    """(pointer, stride from head to head) of the norm's weights, [D] or [H][D]."""
    shape = _given(name, weight).shape
    if not (weight.dtype is torch.float32 and weight.get_device() == index and weight.is_contiguous()):
        _check_plain(name, weight, torch.float32, index)
    if shape == (D,):
        return weight.data_ptr(), 0
    if shape == (H, D):
        return weight.data_ptr(), D
    raise ValueError(f"{name} must be [{D}] or [{H}][{D}], got {tuple(shape)}")


def norm_rope(x, weight, positions=None, inv_freq=None, eps: float = 1e-6, interleaved: bool = False,
              amplitude: float = 1.0, out=None, stream=None):
    """RMS norm of each head's row, then ``rope``'s rotation, rounded once.

    x [T][H][D] bf16 or fp32 (token stride free); weight float32 [D], or [H][D]
    with a row for each head; y = x / sqrt(mean(x^2) + eps) * weight is turned
    by positions [T] int32 and inv_freq (without inv_freq it is not turned).
    Returns out [T][H][D] (allocated unless given; x itself works in place).
    Asynchronous on ``stream``, whose memory an allocated result is."""
    torch = _t()
    index = _cuda_index("x", x)
    io = x.dtype
    code = _io_code(torch, io)
    T, H, D = x.shape
    x_stride = _row_stride("x", x, T, H, D, io, index)
    w, w_stride = _weight(torch, "weight", weight, H, D, index)
    freq, rot = _check_freq(torch, inv_freq, index)
    pos = 0
    if positions is not None:
        _check_plain("positions", positions, torch.int32, index)
        if positions.numel() != T:
            raise ValueError("positions must be [tokens]")
        pos = positions.data_ptr()
    elif rot:
        raise ValueError("inv_freq needs positions")
    if out is None:
        out = torch.empty((T, H, D), dtype=io, device=x.device) if stream is None else \
            _empty_on(torch, (T, H, D), io, index, stream)
    out_stride = _row_stride("out", out, T, H, D, io, index)
    _launch_packed(torch, index, stream, "vt_norm_rope", _NORM_ROPE,
                   (out.data_ptr(), x.data_ptr(), w, pos, freq, T, H, D, rot, 1 if interleaved else 0, amplitude, eps,
                    x_stride, out_stride, w_stride), (code,))
    return out


def norm_append(k, v, k_weight, k_cache, v_cache, q_starts, block_tables, context_lens, q=None, q_weight=None,
                eps: float = 1e-6, q_out=None, positions=None, inv_freq=None, interleaved: bool = False,
                amplitude: float = 1.0, stream=None):
    """``append`` of queries and keys that are normed first (``norm_rope``), in
    the same pass: k_weight float32 [D] or [Hkv][D], q_weight [D] or [Hq][D]
    where q is given.  Values are not normed."""
    return _append(_t(), k, v, k_cache, v_cache, None, q_starts, block_tables, context_lens, q, q_out, positions,
                   inv_freq, interleaved, amplitude, stream, (k_weight, q_weight, eps))


def norm_append_fp8(k, v, k_weight, k_codes, v_codes, k_scale, v_scale, q_starts, block_tables, context_lens, q=None,
                    q_weight=None, eps: float = 1e-6, q_out=None, positions=None, inv_freq=None,
                    interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """``norm_append`` into an FP8 (E4M3) cache of codes with a scale per kv
    head (rows bf16; codes uint8 or torch.float8_e4m3fn)."""
    torch = _t()
    return _append(torch, k, v, *_codes(torch, k_codes, v_codes), (k_scale, v_scale), q_starts,
                   block_tables, context_lens, q, q_out, positions, inv_freq, interleaved, amplitude, stream,
                   (k_weight, q_weight, eps))


def _prefill(torch, q, k_cache, v_cache, scales, q_starts, block_tables, context_lens, scale, window, out, stream,
             masks=None):
    index = _cuda_index("q", q)
    if q.dim() != 3:
        raise ValueError("q must be [tokens][heads][head_dim]")
    T, Hq, D = q.shape
    fp8 = scales is not None
    io = torch.bfloat16 if fp8 else q.dtype
    code = 0 if fp8 else _io_code(torch, io)
    _check_plain("q", q, io, index)
    B, max_blocks = _check_ragged(torch, k_cache, v_cache, k_cache.dtype if fp8 else io, q_starts, block_tables,
                                  context_lens, index)
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != D or v_cache.shape != shape:
        raise ValueError("k_cache/v_cache must be [num_blocks][32][Hkv][head_dim] matching q")
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty_on(torch, (T, Hq, D), io, index, stream)
    else:
        _check_plain("out", out, io, index)
        if out.shape != q.shape:
            raise ValueError("out must be shaped like q")
    if scale is None:
        scale = D ** -0.5
    head = (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr())
    rest = (q_starts.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), B, T, Hq, shape[2], D, shape[1],
            scale, window)
    if masks is not None:
        words = _check_masks(torch, masks, T, index)
        rest = (masks.data_ptr(),) + rest[:5] + (words,) + rest[5:]
        if fp8:
            _check_scales(torch, *scales, shape[2], index)
            _launch_packed(torch, index, stream, "vt_paged_attn_prefill_tree_fp8", _PREFILL_TREE_FP8,
                           head + (scales[0].data_ptr(), scales[1].data_ptr()) + rest, (max_blocks, shape[0]))
        else:
            _launch_packed(torch, index, stream, "vt_paged_attn_prefill_tree", _PREFILL_TREE,
                           head + rest, (max_blocks, shape[0], code))
    elif fp8:
        _check_scales(torch, *scales, shape[2], index)
        _launch(torch, index, stream, "vt_paged_attn_prefill_fp8", library().vt_paged_attn_prefill_fp8,
                head + (scales[0].data_ptr(), scales[1].data_ptr()) + rest, (max_blocks, shape[0]))
    else:
        _launch(torch, index, stream, "vt_paged_attn_prefill", library().vt_paged_attn_prefill, head + rest,
                (max_blocks, shape[0], code))
    return out


def prefill(q, k_cache, v_cache, q_starts, block_tables, context_lens, scale=None, window: int = 0, out=None,
            stream=None):
    """Attention of a ragged batch of chunks of new tokens over the paged
    cache (which holds their keys and values already, see ``append``).

    q [T][Hq][D]: sequence b owns rows q_starts[b]:q_starts[b + 1], the last of
    its context_lens[b] tokens, attending causally; q_starts [B + 1] int32, the
    rest as for ``decode``.  Returns out [T][Hq][D] (allocated unless given;
    rows behind the last sequence are not written).  Asynchronous on
    ``stream``, whose memory an allocated result is."""
    return _prefill(_t(), q, k_cache, v_cache, None, q_starts, block_tables, context_lens, scale, window, out, stream)


def prefill_fp8(q, k_codes, v_codes, k_scale, v_scale, q_starts, block_tables, context_lens, scale=None,
                window: int = 0, out=None, stream=None):
    """``prefill`` over an FP8 (E4M3) cache (q and out bf16; codes uint8 or
    torch.float8_e4m3fn with a float32 scale per kv head)."""
    torch = _t()
    return _prefill(torch, q, *_codes(torch, k_codes, v_codes), (k_scale, v_scale), q_starts,
                    block_tables, context_lens, scale, window, out, stream)


def _check_masks(torch, masks, T, index):
    """Words of a row of masks [T][words]."""
    if not (masks.dtype is torch.int32 and masks.get_device() == index and masks.is_contiguous()):
        _check_plain("masks", masks, torch.int32, index)
    shape = masks.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"masks must be [{T}][words], got {tuple(shape)}")
    return shape[1]


def prefill_tree(q, k_cache, v_cache, masks, q_starts, block_tables, context_lens, scale=None, window: int = 0,
                 out=None, stream=None):
    """Attention of trees of drafted tokens over the paged cache (which holds
    their keys and values already, see ``append`` and ``norm_append``).

    As ``prefill``, but a row sees every token before its sequence's first new
    one, and new token i where bit i of its mask is set (masks int32
    [T][words], see ``tree_masks``); with a window the last ``window`` of
    those.  A row that sees nothing is 0."""
    return _prefill(_t(), q, k_cache, v_cache, None, q_starts, block_tables, context_lens, scale, window, out, stream,
                    _given("masks", masks))


def prefill_tree_fp8(q, k_codes, v_codes, k_scale, v_scale, masks, q_starts, block_tables, context_lens, scale=None,
                     window: int = 0, out=None, stream=None):
    """``prefill_tree`` over an FP8 (E4M3) cache (q and out bf16; codes uint8 or
    torch.float8_e4m3fn with a float32 scale per kv head)."""
    torch = _t()
    return _prefill(torch, q, *_codes(torch, k_codes, v_codes), (k_scale, v_scale), q_starts,
                    block_tables, context_lens, scale, window, out, stream, _given("masks", masks))


def tree_masks(parents, q_starts, context_lens, words=None, masks=None, positions=None, stream=None):
    """Masks and positions of trees of drafted tokens, from each one's parent.

    parents [T] int32: the place within its sequence's rows of the token that
    a row follows (less than its own), -1 where it follows the context.
    q_starts and context_lens as for ``append``, the drafted tokens counted in.
    Returns (masks [T][words] int32, positions [T] int32): bit i of a row's
    mask says that it sees its sequence's i-th new token (itself and those it
    follows), and its position is the context's end plus the number it follows.
    ``words`` (32 tokens each, 32 at most) is read off masks where they are
    given.  Rows behind the last sequence are not written.  Asynchronous on
    ``stream``, whose memory allocated results are."""
    torch = _t()
    index = _cuda_index("parents", parents)
    int32 = torch.int32
    if not (q_starts.get_device() == context_lens.get_device() == index and parents.dtype is int32
            and q_starts.dtype is int32 and context_lens.dtype is int32 and parents.is_contiguous()
            and q_starts.is_contiguous() and context_lens.is_contiguous()):
        for name, t in (("parents", parents), ("q_starts", q_starts), ("context_lens", context_lens)):
            _check_plain(name, t, int32, index)
    shape, B = parents.shape, context_lens.numel()
    if len(shape) != 1 or q_starts.numel() != B + 1:
        raise ValueError("parents must be [tokens] and q_starts [num_seqs + 1]")
    T = shape[0]
    if masks is None:
        if words is None:
            raise ValueError("give words or masks")
        masks = torch.empty((T, words), dtype=int32, device=parents.device) if stream is None else \
            _empty_on(torch, (T, words), int32, index, stream)
    elif words is not None and masks.shape[-1] != words:
        raise ValueError("masks must be [tokens][words]")
    words = _check_masks(torch, masks, T, index)
    positions = _int32_out(torch, "positions", positions, T, index, stream)
    _launch_packed(torch, index, stream, "vt_tree_masks", _TREE_MASKS,
                   (masks.data_ptr(), positions.data_ptr(), parents.data_ptr(), q_starts.data_ptr(),
                    context_lens.data_ptr(), B, T, words), ())
    return masks, positions


def _int32_out(torch, name, t, n, index, stream):
    """An int32 result [n], allocated unless given."""
    if t is None:
        return torch.empty((n,), dtype=torch.int32, device=index) if stream is None else \
            _empty_on(torch, (n,), torch.int32, index, stream)
    if not (t.dtype is torch.int32 and t.get_device() == index and t.is_contiguous()):
        _check_plain(name, t, torch.int32, index)
    if t.numel() != n:
        raise ValueError(f"{name} must be [{n}]")
    return t


def step_tables(context_lens, new_lens, block_tables, free_pages, counters, num_tokens: int, keep_lens=None,
                q_starts=None, positions=None, slots=None, stream=None):
    """Page tables of the next step, on the GPU, from request lengths.

    Sequence b keeps keep_lens[b] of its context_lens[b] tokens (all without
    keep_lens) and gets new_lens[b] new ones: pages behind what it keeps go
    back to the stack of free pages, pages for the new tokens come from its
    top, and block_tables, context_lens, free_pages [num_blocks] and
    counters [2] (pages on the stack, sequences refused) are updated in place.
    Returns (q_starts [B + 1], positions [num_tokens], slots [num_tokens]),
    allocated unless given: the rows of the packed batch, their positions and
    their slots (page * 32 + place).  Sequences from the first on whose pages
    or rows do not fit get none, nor do those with a table too short or
    lengths that are none (counters[1] of them in all): rows lie as granted, so
    what was packed by the lengths asked for is then out of place
    (vt_paged_step_tables).  Asynchronous on ``stream``, whose memory
    allocated results are."""
    torch = _t()
    index = _cuda_index("context_lens", context_lens)
    int32 = torch.int32
    # (in line what _check_plain says of each)
    if not (new_lens.get_device() == block_tables.get_device() == free_pages.get_device() == counters.get_device()
            == index and context_lens.dtype is int32 and new_lens.dtype is int32 and block_tables.dtype is int32
            and free_pages.dtype is int32 and counters.dtype is int32 and context_lens.is_contiguous()
            and new_lens.is_contiguous() and block_tables.is_contiguous() and free_pages.is_contiguous()
            and counters.is_contiguous()):
        for name, t in (("context_lens", context_lens), ("new_lens", new_lens), ("block_tables", block_tables),
                        ("free_pages", free_pages), ("counters", counters)):
            _check_plain(name, t, int32, index)
    B, table = context_lens.numel(), block_tables.shape
    if new_lens.numel() != B or len(table) != 2 or table[0] != B or counters.numel() != 2:
        raise ValueError("new_lens must be [num_seqs], block_tables [num_seqs][max_blocks] and counters [2]")
    keep = 0
    if keep_lens is not None:
        if not (keep_lens.dtype is int32 and keep_lens.get_device() == index and keep_lens.is_contiguous()):
            _check_plain("keep_lens", keep_lens, int32, index)
        if keep_lens.numel() != B:
            raise ValueError("keep_lens must be [num_seqs]")
        keep = keep_lens.data_ptr()
    q_starts = _int32_out(torch, "q_starts", q_starts, B + 1, index, stream)
    positions = _int32_out(torch, "positions", positions, num_tokens, index, stream)
    slots = _int32_out(torch, "slots", slots, num_tokens, index, stream)
    _launch_packed(torch, index, stream, "vt_paged_step_tables", _STEP_TABLES,
                   (block_tables.data_ptr(), context_lens.data_ptr(), free_pages.data_ptr(), counters.data_ptr(),
                    q_starts.data_ptr(), positions.data_ptr(), slots.data_ptr(), keep, new_lens.data_ptr(), B,
                    num_tokens, BLOCK_SIZE), (table[1], free_pages.numel()))
    return q_starts, positions, slots


def keep_path(accepted, masks, k_cache, v_cache, q_starts, block_tables, context_lens, kept_lens=None, stream=None):
    """Moves each sequence's accepted branch to consecutive slots.

    accepted [B] int32: the place within its sequence's rows of the last
    accepted drafted token, -1 for none; the tokens its row of masks names
    (``tree_masks``) go to the slots right behind the context they were
    drafted for.  k_cache, v_cache [num_blocks][32][Hkv][D], or
    [layers][num_blocks][32][Hkv][D] (layer stride free) for all layers in one
    launch; bf16, fp32 or E4M3 codes.  Returns kept_lens [B] (allocated unless
    given): the contexts that are left, ``step_tables``' keep_lens.
    Asynchronous on ``stream``, whose memory an allocated result is."""
    torch = _t()
    index = _cuda_index("accepted", accepted)
    int32 = torch.int32
    if k_cache.dtype is torch.float8_e4m3fn or k_cache.dtype is torch.uint8:
        k_cache, v_cache = _codes(torch, k_cache, v_cache)
        code = VT_E4M3
    else:
        code = _io_code(torch, k_cache.dtype)
    kv = k_cache.dtype
    shape = k_cache.shape
    if len(shape) not in (4, 5) or v_cache.shape != shape:
        raise ValueError("k_cache/v_cache must be [num_blocks][32][Hkv][head_dim], or layers of it")
    layers = shape[0] if len(shape) == 5 else 1
    strides = (0, 0)
    if len(shape) == 5 and layers:
        inner = (shape[2] * shape[3] * shape[4], shape[3] * shape[4], shape[4], 1)
        strides = k_cache.stride(), v_cache.stride()
        if not (k_cache.get_device() == v_cache.get_device() == index and v_cache.dtype is kv
                and strides[0][1:] == inner and strides[1][1:] == inner):
            _check_plain("k_cache", k_cache[0], kv, index)  # (a view of one layer takes 3 us)
            _check_plain("v_cache", v_cache[0], kv, index)
        strides = (strides[0][0], strides[1][0]) if layers > 1 else (0, 0)
    else:
        _check_plain("k_cache", k_cache, kv, index)
        _check_plain("v_cache", v_cache, kv, index)
    if not (q_starts.get_device() == block_tables.get_device() == context_lens.get_device() == index
            and accepted.dtype is int32 and q_starts.dtype is int32 and block_tables.dtype is int32
            and context_lens.dtype is int32 and accepted.is_contiguous() and q_starts.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()):
        for name, t in (("accepted", accepted), ("q_starts", q_starts), ("block_tables", block_tables),
                        ("context_lens", context_lens)):
            _check_plain(name, t, int32, index)
    B, table = context_lens.numel(), block_tables.shape
    if accepted.numel() != B or q_starts.numel() != B + 1 or len(table) != 2 or table[0] != B:
        raise ValueError("accepted must be [num_seqs], q_starts [num_seqs + 1] and block_tables "
                         "[num_seqs][max_blocks]")
    words = _check_masks(torch, masks, masks.shape[0], index)
    kept_lens = _int32_out(torch, "kept_lens", kept_lens, B, index, stream)
    _launch_packed(torch, index, stream, "vt_paged_kv_keep_path", _KEEP_PATH,
                   (k_cache.data_ptr(), v_cache.data_ptr(), kept_lens.data_ptr(), accepted.data_ptr(), masks.data_ptr(),
                    q_starts.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), B, masks.shape[0], words,
                    layers, shape[-2], shape[-1], shape[-3], strides[0], strides[1]), (table[1], shape[-4], code))
    return kept_lens
