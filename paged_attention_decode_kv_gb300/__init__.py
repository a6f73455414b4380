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


def _codes(torch, t):
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError("the caches must be uint8 or float8_e4m3fn E4M3 codes")
    return t


def _check_freq(torch, inv_freq, index):
    """(pointer, rot_dim) of a frequency table, or of none."""
    if inv_freq is None:
        return None, 0
    _check_plain("inv_freq", inv_freq, torch.float64, index)
    n = inv_freq.numel()
    return (inv_freq.data_ptr(), 2 * n) if n else (None, 0)


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
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            status = call(*before, _stream_on(torch, index, stream), *after)
    else:
        status = call(*before, _stream_on(torch, index, stream), *after)
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
            inv_freq, interleaved, amplitude, stream):
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
    q_ptr = out_ptr = pos_ptr = None
    if q is not None:
        Hq = q.shape[1]
        qs = _row_stride("q", q, T, Hq, D, io, index)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=io, device=q.device) if stream is None else \
                _empty_on(torch, (T, Hq, D), io, index, stream)
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
            shape[1], rot, 1 if interleaved else 0, amplitude, qs, ks, vs)
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
    return _append(torch, k, v, _codes(torch, k_codes), _codes(torch, v_codes), (k_scale, v_scale), q_starts,
                   block_tables, context_lens, q, q_out, positions, inv_freq, interleaved, amplitude, stream)


def _prefill(torch, q, k_cache, v_cache, scales, q_starts, block_tables, context_lens, scale, window, out, stream):
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
    if fp8:
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
    return _prefill(torch, q, _codes(torch, k_codes), _codes(torch, v_codes), (k_scale, v_scale), q_starts,
                    block_tables, context_lens, scale, window, out, stream)
