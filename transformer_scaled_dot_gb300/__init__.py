"""GB300 (sm_103a) multi-head scaled dot-product attention.

A thin Python binding over the C ABI of libtsd_attention.so
(include/tsd_attention.h). Each function has the name and the parameters of
its C entry point and only marshals arguments: tensor arguments may be
torch tensors (their data_ptr() is passed) or raw device addresses (int);
`stream` may be a torch.cuda.Stream, a raw cudaStream_t (int), or None for
torch's current stream. A non-OK status raises AttnError.

There is no fallback: if the native library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

__all__ = [
    "ATTN_OK", "ATTN_ERR_INVALID", "ATTN_ERR_UNSUPPORTED", "ATTN_ERR_CUDA",
    "ATTN_ERR_DEVICE_TIMEOUT", "ATTN_ERR_DEVICE_INDEX", "ATTN_ERR_DEVICE_VALUE",
    "ATTN_MASK_NONE", "ATTN_MASK_CAUSAL", "ATTN_MASK_KEY_PADDING",
    "AttnError", "library", "library_path", "EXPORTED_SYMBOLS",
    "attn_forward", "attn_forward_strided", "attn_forward_f32", "mha_workspace_bytes",
    "mha_forward", "attn_get_device_status", "attn_last_cuda_error", "attn_status_string",
    "attn_selftest_wait_timeout", "mha_project_qkv", "mha_project_out", "mha_forward_noalloc",
    "mha_concat_heads", "mha_forward_launches", "attn_forward_window", "attn_decode",
    "attn_decode_workspace_bytes", "encoder_layer_forward", "encoder_layer_workspace_bytes",
    "MHA_NOALLOC_SCRATCH_BYTES", "attn_host_workspace_bytes", "attn_forward_host",
    "mha_host_workspace_bytes", "mha_forward_host", "encoder_layer_host_workspace_bytes",
    "encoder_layer_forward_host", "attn_decode_host_workspace_bytes", "attn_decode_host",
    "attn_forward_window_host", "mha_forward_host_async", "attn_host_join",
    "attn_decode_host_async", "encoder_layer_forward_host_async",
    "ATTN_ROPE_NONE", "ATTN_ROPE_HALVES", "ATTN_ROPE_PAIRS", "attn_cache_append",
    "attn_cache_append_q4", "attn_decode_paged_workspace_bytes", "attn_decode_paged",
    "attn_decode_paged_q4", "attn_cache_fork", "attn_cache_release", "attn_cache_pages_workspace_bytes",
    "attn_cache_reserve", "attn_cache_compact", "attn_cache_copy", "attn_cache_copy_q4",
    "beam_select_workspace_bytes", "beam_select", "beam_select_f32",
]

ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_DEVICE_TIMEOUT, \
    ATTN_ERR_DEVICE_INDEX, ATTN_ERR_DEVICE_VALUE = range(7)
ATTN_MASK_NONE, ATTN_MASK_CAUSAL, ATTN_MASK_KEY_PADDING = 0, 1, 2
ATTN_ROPE_NONE, ATTN_ROPE_HALVES, ATTN_ROPE_PAIRS = 0, 1, 2

EXPORTED_SYMBOLS = (
    "attn_forward", "attn_forward_strided", "attn_forward_f32", "mha_workspace_bytes",
    "mha_forward", "attn_get_device_status", "attn_last_cuda_error", "attn_status_string",
    "attn_selftest_wait_timeout", "mha_project_qkv", "mha_project_out", "mha_forward_noalloc",
    "mha_concat_heads", "mha_forward_launches", "attn_forward_window", "attn_decode",
    "attn_decode_workspace_bytes", "encoder_layer_forward", "encoder_layer_workspace_bytes",
    "attn_host_workspace_bytes", "attn_forward_host", "mha_host_workspace_bytes",
    "mha_forward_host", "encoder_layer_host_workspace_bytes", "encoder_layer_forward_host",
    "attn_decode_host_workspace_bytes", "attn_decode_host", "attn_forward_window_host",
    "mha_forward_host_async", "attn_host_join", "attn_decode_host_async",
    "encoder_layer_forward_host_async", "attn_cache_append", "attn_cache_append_q4",
    "attn_decode_paged_workspace_bytes", "attn_decode_paged", "attn_decode_paged_q4",
    "attn_cache_fork", "attn_cache_release", "attn_cache_pages_workspace_bytes",
    "attn_cache_reserve", "attn_cache_compact", "attn_cache_copy", "attn_cache_copy_q4",
    "beam_select_workspace_bytes", "beam_select", "beam_select_f32",
)

# TSD_MHA_NOALLOC_SCRATCH_BYTES of the header: the fixed scratch of mha_forward_noalloc
MHA_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024

_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = library().attn_status_string(status).decode()
        extra = ""
        if status == ATTN_ERR_CUDA:
            extra = f" (cudaError {library().attn_last_cuda_error()})"
        super().__init__(f"{where}: {name}{extra}")


def library_path() -> str:
    return _build.LIB_PATH


def library():
    """Loads libtsd_attention.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, i, i64, f, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    lib.attn_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, f, st]
    lib.attn_forward_strided.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, vp, i64, i64, i64,
                                         vp, i64, i64, i64, i, i, i, i, i, i, i, vp, f, st]
    lib.attn_forward_f32.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, f, st]
    lib.mha_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.mha_workspace_bytes.restype = ctypes.c_size_t
    lib.mha_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, f, vp,
                                ctypes.c_size_t, st]
    lib.mha_project_qkv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, st]
    lib.mha_concat_heads.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, f, vp,
                                     ctypes.c_size_t, st]
    lib.mha_project_out.argtypes = [vp, vp, vp, i, i, i, i, i, st]
    lib.mha_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, f,
                                        st]
    lib.attn_get_device_status.argtypes = [st]
    lib.attn_last_cuda_error.argtypes = []
    lib.attn_status_string.argtypes = [i]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_selftest_wait_timeout.argtypes = [i, st]
    lib.mha_forward_launches.argtypes = [i, i, i, i, i, i, i, i]
    lib.attn_forward_window.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, i, i, f, st]
    lib.attn_decode_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_decode.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, f, vp, ctypes.c_size_t, st]
    lib.encoder_layer_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.encoder_layer_workspace_bytes.restype = ctypes.c_size_t
    lib.encoder_layer_forward.argtypes = [vp] * 14 + [i] * 7 + [vp, f, f, vp, ctypes.c_size_t, st]
    sz = ctypes.c_size_t
    for name, n in (("attn_host_workspace_bytes", 6), ("mha_host_workspace_bytes", 7),
                    ("encoder_layer_host_workspace_bytes", 6),
                    ("attn_decode_host_workspace_bytes", 6)):
        getattr(lib, name).argtypes = [i] * n
        getattr(lib, name).restype = sz
    lib.attn_forward_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, f, vp, sz, st]
    lib.attn_forward_window_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, i, i, f, vp,
                                             sz, st]
    lib.mha_forward_host.argtypes = [vp] * 7 + [i] * 8 + [vp, f, vp, sz, st]
    lib.mha_forward_host_async.argtypes = [vp] * 7 + [i] * 8 + [vp, f, vp, sz, st]
    lib.attn_host_join.argtypes = [st]
    lib.encoder_layer_forward_host.argtypes = [vp] * 14 + [i] * 7 + [vp, f, f, vp, sz, st]
    lib.encoder_layer_forward_host_async.argtypes = lib.encoder_layer_forward_host.argtypes
    lib.attn_decode_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, f, vp, sz, st]
    lib.attn_decode_host_async.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, f, vp, sz, st]
    lib.attn_cache_append.argtypes = [vp, i64, i64, i64, vp, vp, i64, i64, i64] + [vp] * 8 + \
        [i] * 11 + [st]
    lib.attn_cache_append_q4.argtypes = [vp, i64, i64, i64, vp, vp, i64, i64, i64] + [vp] * 6 + \
        [f, f] + [vp] * 4 + [i] * 11 + [st]
    lib.attn_decode_paged_workspace_bytes.argtypes = [i] * 7
    lib.attn_decode_paged_workspace_bytes.restype = sz
    lib.attn_decode_paged.argtypes = [vp] * 7 + [i] * 9 + [f, vp, sz, st]
    lib.attn_decode_paged_q4.argtypes = [vp] * 5 + [f, f] + [vp] * 4 + [i] * 9 + [f, vp, sz, st]
    lib.attn_cache_fork.argtypes = [vp] * 4 + [i] * 3 + [st]
    lib.attn_cache_release.argtypes = [vp] * 3 + [i] * 4 + [st]
    lib.attn_cache_pages_workspace_bytes.argtypes = [i, i]
    lib.attn_cache_pages_workspace_bytes.restype = sz
    lib.attn_cache_reserve.argtypes = [vp] * 7 + [i] * 5 + [vp, sz, st]
    lib.attn_cache_compact.argtypes = [vp] * 7 + [i] * 5 + [vp, sz, st]
    lib.attn_cache_copy.argtypes = [vp] * 4 + [i, i, i64] + [i] * 4 + [st]
    lib.attn_cache_copy_q4.argtypes = [vp] * 6 + [i, i, i64] + [i] * 4 + [st]
    lib.beam_select_workspace_bytes.argtypes = [i] * 3
    lib.beam_select_workspace_bytes.restype = sz
    for name in ("beam_select", "beam_select_f32"):
        getattr(lib, name).argtypes = [vp, i64, vp, vp, i, i, i, i, ctypes.c_double] + [vp] * 7 + [sz, st]
        getattr(lib, name).restype = ctypes.c_int
    for name in ("attn_cache_fork", "attn_cache_release", "attn_cache_reserve",
                 "attn_cache_compact", "attn_cache_copy", "attn_cache_copy_q4",
                 "attn_forward", "attn_forward_strided", "attn_forward_f32", "mha_forward",
                 "attn_cache_append", "attn_cache_append_q4", "attn_decode_paged",
                 "attn_decode_paged_q4", "attn_get_device_status", "attn_last_cuda_error", "attn_selftest_wait_timeout",
                 "mha_project_qkv", "mha_project_out", "mha_forward_noalloc", "mha_concat_heads",
                 "mha_forward_launches", "attn_forward_window", "attn_decode",
                 "encoder_layer_forward", "attn_forward_host", "mha_forward_host",
                 "encoder_layer_forward_host", "attn_decode_host", "attn_forward_window_host",
                 "mha_forward_host_async", "attn_host_join", "attn_decode_host_async",
                 "encoder_layer_forward_host_async"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


_tensor_types = set()  # that have had a data_ptr()


def _ptr(x):
    """Address of a torch tensor (device or host), a numpy array (host), or an int."""
    if type(x) in _tensor_types:
        return x.data_ptr()
    if x is None or isinstance(x, int):
        return x
    if not hasattr(x, "data_ptr"):
        return x.ctypes.data
    _tensor_types.add(type(x))
    return x.data_ptr()


_raw_stream = _device = None  # torch's, from the first call that finds CUDA up


def _current_stream():
    """torch's current stream, as a raw cudaStream_t. torch.cuda.current_stream() makes a Stream
    object first (2.9 us against 0.2 us on the Grace host, more than a short kernel's launch),
    so its raw form is asked where torch has it and CUDA is up."""
    global _raw_stream, _device
    if _raw_stream is not None:
        return _raw_stream(_device())
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = raw
    return raw(_device())


def _stream(s):
    if s is None:
        return _current_stream() if _raw_stream is None else _raw_stream(_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def attn_forward(q, k, v, out, B, h, n_q, n_k, d_k, d_v, mask_kind=ATTN_MASK_NONE, kv_lens=None,
                 scale=0.0, stream=None):
    _check(library().attn_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, h, n_q, n_k, d_k, d_v,
                                  mask_kind, _ptr(kv_lens), scale, _stream(stream)), "attn_forward")


def attn_forward_window(q, k, v, out, B, h, n_q, n_k, d_k, d_v, window_left, window_right,
                        mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, stream=None):
    """Restricted self-attention: query i sees keys [i - window_left, i + window_right]
    (-1 = no bound on that side)."""
    _check(library().attn_forward_window(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, h, n_q, n_k,
                                         d_k, d_v, mask_kind, _ptr(kv_lens), window_left,
                                         window_right, scale, _stream(stream)),
           "attn_forward_window")


def attn_decode_workspace_bytes(B, h, n_q, n_max, d_v) -> int:
    return int(library().attn_decode_workspace_bytes(B, h, n_q, n_max, d_v))


def attn_decode(q, k_cache, v_cache, out, B, h, n_q, n_max, d_k, d_v, cache_lens=None, scale=0.0,
                workspace=None, workspace_bytes=0, stream=None):
    """One decoding step: the n_q newest tokens' queries against an n_max-row
    key/value cache (cache_lens[b] valid rows, None = n_max)."""
    _check(library().attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), B, h, n_q,
                                 n_max, d_k, d_v, _ptr(cache_lens), scale, _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "attn_decode")


def attn_cache_append(q, q_sb, q_sh, q_sr, k, v, kv_sb, kv_sh, kv_sr, q_out, k_out, k_cache,
                      v_cache, page_table, cache_lens, new_lens, rope, rope_rows, rope_dim,
                      rope_kind, B, h, h_kv, n_new, d, n_pages, page_size, max_pages, stream=None):
    """Writes the new tokens' keys (rotated by their positions) and values into a paged
    bf16 cache [n_pages, h_kv, page_size, d], and the rotated queries into q_out."""
    _check(library().attn_cache_append(
        _ptr(q), q_sb, q_sh, q_sr, _ptr(k), _ptr(v), kv_sb, kv_sh, kv_sr, _ptr(q_out), _ptr(k_out),
        _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(cache_lens), _ptr(new_lens),
        _ptr(rope), rope_rows, rope_dim, rope_kind, B, h, h_kv, n_new, d, n_pages, page_size,
        max_pages, _stream(stream)), "attn_cache_append")


def attn_cache_append_q4(q, q_sb, q_sh, q_sr, k, v, kv_sb, kv_sh, kv_sr, q_out, k_out, k_codes,
                         k_scales, v_codes, v_scales, k_factor, v_factor, page_table, cache_lens,
                         new_lens, rope, rope_rows, rope_dim, rope_kind, B, h, h_kv, n_new, d,
                         n_pages, page_size, max_pages, stream=None):
    """attn_cache_append into a paged cache of 4-bit codes [.., d / 2] with a scale per 16
    columns [.., d / 16]."""
    _check(library().attn_cache_append_q4(
        _ptr(q), q_sb, q_sh, q_sr, _ptr(k), _ptr(v), kv_sb, kv_sh, kv_sr, _ptr(q_out), _ptr(k_out),
        _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), k_factor, v_factor,
        _ptr(page_table), _ptr(cache_lens), _ptr(new_lens), _ptr(rope), rope_rows, rope_dim,
        rope_kind, B, h, h_kv, n_new, d, n_pages, page_size, max_pages, _stream(stream)),
        "attn_cache_append_q4")


def attn_decode_paged_workspace_bytes(B, h, h_kv, n_q, d, page_size, max_pages) -> int:
    return int(library().attn_decode_paged_workspace_bytes(B, h, h_kv, n_q, d, page_size,
                                                           max_pages))


def attn_decode_paged(q, k_cache, v_cache, out, page_table, cache_lens, new_lens, B, h, h_kv, n_q,
                      d, n_pages, page_size, max_pages, mask_kind=ATTN_MASK_CAUSAL, scale=0.0,
                      workspace=None, workspace_bytes=0, stream=None):
    """One decoding step over a paged bf16 cache: n_q queries per sequence, h / h_kv query
    heads to a key head, causal from the end of the cache or without a mask."""
    _check(library().attn_decode_paged(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(page_table), _ptr(cache_lens),
        _ptr(new_lens), B, h, h_kv, n_q, d, n_pages, page_size, max_pages, mask_kind, scale,
        _ptr(workspace), workspace_bytes, _stream(stream)), "attn_decode_paged")


def attn_decode_paged_q4(q, k_codes, k_scales, v_codes, v_scales, k_factor, v_factor, out,
                         page_table, cache_lens, new_lens, B, h, h_kv, n_q, d, n_pages, page_size,
                         max_pages, mask_kind=ATTN_MASK_CAUSAL, scale=0.0, workspace=None,
                         workspace_bytes=0, stream=None):
    """attn_decode_paged over a paged cache of 4-bit codes and their scales."""
    _check(library().attn_decode_paged_q4(
        _ptr(q), _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), k_factor, v_factor,
        _ptr(out), _ptr(page_table), _ptr(cache_lens), _ptr(new_lens), B, h, h_kv, n_q, d, n_pages,
        page_size, max_pages, mask_kind, scale, _ptr(workspace), workspace_bytes,
        _stream(stream)), "attn_decode_paged_q4")


def attn_cache_fork(page_table, cache_lens, ref_counts, parents, B, n_pages, max_pages,
                    stream=None):
    """Row r of the page table becomes row parents[r] (-1: empty), all at once and in place;
    ref_counts, and cache_lens unless None, follow."""
    _check(library().attn_cache_fork(_ptr(page_table), _ptr(cache_lens), _ptr(ref_counts),
                                     _ptr(parents), B, n_pages, max_pages, _stream(stream)),
           "attn_cache_fork")


def attn_cache_release(page_table, ref_counts, keep_lens, B, n_pages, page_size, max_pages,
                       stream=None):
    """Row b gives back the pages past its first keep_lens[b] rows (None: all; negative: none)."""
    _check(library().attn_cache_release(_ptr(page_table), _ptr(ref_counts), _ptr(keep_lens), B,
                                        n_pages, page_size, max_pages, _stream(stream)),
           "attn_cache_release")


def attn_cache_pages_workspace_bytes(B, n_pages) -> int:
    return int(library().attn_cache_pages_workspace_bytes(B, n_pages))


def attn_cache_reserve(page_table, ref_counts, cache_lens, new_lens, copies, n_copies, n_missing,
                       B, n_new, n_pages, page_size, max_pages, workspace=None, workspace_bytes=0,
                       stream=None):
    """Pages of their own for the new tokens of every row, the lowest free ones first; the copies
    that attn_cache_copy has to make of pages that were shared go into `copies`."""
    _check(library().attn_cache_reserve(
        _ptr(page_table), _ptr(ref_counts), _ptr(cache_lens), _ptr(new_lens), _ptr(copies),
        _ptr(n_copies), _ptr(n_missing), B, n_new, n_pages, page_size, max_pages, _ptr(workspace),
        workspace_bytes, _stream(stream)), "attn_cache_reserve")


def attn_cache_compact(page_table, ref_counts, table_out, counts_out, copies, n_copies, n_used, B,
                       n_pages, page_size, max_pages, max_copies, workspace=None,
                       workspace_bytes=0, stream=None):
    """The table and counts with the used pages at the front of the pool, and the copies that
    attn_cache_copy has to make for it."""
    _check(library().attn_cache_compact(
        _ptr(page_table), _ptr(ref_counts), _ptr(table_out), _ptr(counts_out), _ptr(copies),
        _ptr(n_copies), _ptr(n_used), B, n_pages, page_size, max_pages, max_copies,
        _ptr(workspace), workspace_bytes, _stream(stream)), "attn_cache_compact")


def attn_cache_copy(k_cache, v_cache, copies, n_copies, max_copies, n_layers, layer_rows, h_kv, d,
                    n_pages, page_size, stream=None):
    """Copies rows of pages by a list [max_copies, 3] of (from, to, rows), in all layers."""
    _check(library().attn_cache_copy(_ptr(k_cache), _ptr(v_cache), _ptr(copies), _ptr(n_copies),
                                     max_copies, n_layers, layer_rows, h_kv, d, n_pages,
                                     page_size, _stream(stream)), "attn_cache_copy")


def attn_cache_copy_q4(k_codes, k_scales, v_codes, v_scales, copies, n_copies, max_copies,
                       n_layers, layer_rows, h_kv, d, n_pages, page_size, stream=None):
    """attn_cache_copy of a 4-bit cache's codes and scales."""
    _check(library().attn_cache_copy_q4(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes),
                                        _ptr(v_scales), _ptr(copies), _ptr(n_copies), max_copies,
                                        n_layers, layer_rows, h_kv, d, n_pages, page_size,
                                        _stream(stream)), "attn_cache_copy_q4")


def beam_select_workspace_bytes(B, beams, vocab) -> int:
    return int(library().beam_select_workspace_bytes(B, beams, vocab))


def beam_select(logits, row_stride, scores, lengths, B, beams, vocab, end, alpha, tokens, parents,
                new_scores, ended_scores=None, ended_rows=None, ended_lengths=None,
                workspace=None, workspace_bytes=0, stream=None):
    """One step of beam search: the next beams of each sentence from its beams' bf16 logits, and
    the hypotheses that ended (end = -1: no end token)."""
    _check(library().beam_select(
        _ptr(logits), row_stride, _ptr(scores), _ptr(lengths), B, beams, vocab, end, alpha,
        _ptr(tokens), _ptr(parents), _ptr(new_scores), _ptr(ended_scores), _ptr(ended_rows),
        _ptr(ended_lengths), _ptr(workspace), workspace_bytes, _stream(stream)), "beam_select")


def beam_select_f32(logits, row_stride, scores, lengths, B, beams, vocab, end, alpha, tokens,
                    parents, new_scores, ended_scores=None, ended_rows=None, ended_lengths=None,
                    workspace=None, workspace_bytes=0, stream=None):
    """beam_select of fp32 logits."""
    _check(library().beam_select_f32(
        _ptr(logits), row_stride, _ptr(scores), _ptr(lengths), B, beams, vocab, end, alpha,
        _ptr(tokens), _ptr(parents), _ptr(new_scores), _ptr(ended_scores), _ptr(ended_rows),
        _ptr(ended_lengths), _ptr(workspace), workspace_bytes, _stream(stream)), "beam_select_f32")


def encoder_layer_workspace_bytes(B, n, d_model, h, d_k, d_ff) -> int:
    return int(library().encoder_layer_workspace_bytes(B, n, d_model, h, d_k, d_ff))


def encoder_layer_forward(x, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1, w_2, b_2,
                          ln2_gamma, ln2_beta, out, B, n, d_model, h, d_k, d_ff,
                          mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, eps=1e-6,
                          workspace=None, workspace_bytes=0, stream=None):
    """LayerNorm_2(y + FFN(y)), y = LayerNorm_1(x + MultiHead(x, x)) (post-LN encoder layer)."""
    ptrs = [_ptr(t) for t in (x, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1, w_2, b_2,
                              ln2_gamma, ln2_beta, out)]
    _check(library().encoder_layer_forward(*ptrs, B, n, d_model, h, d_k, d_ff, mask_kind,
                                           _ptr(kv_lens), scale, eps, _ptr(workspace),
                                           workspace_bytes, _stream(stream)),
           "encoder_layer_forward")


def attn_forward_strided(q, q_sb, q_sh, q_sr, k, k_sb, k_sh, k_sr, v, v_sb, v_sh, v_sr,
                         out, o_sb, o_sh, o_sr, B, h, n_q, n_k, d_k, d_v,
                         mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, stream=None):
    _check(library().attn_forward_strided(
        _ptr(q), q_sb, q_sh, q_sr, _ptr(k), k_sb, k_sh, k_sr, _ptr(v), v_sb, v_sh, v_sr,
        _ptr(out), o_sb, o_sh, o_sr, B, h, n_q, n_k, d_k, d_v, mask_kind, _ptr(kv_lens), scale,
        _stream(stream)), "attn_forward_strided")


def attn_forward_f32(q, k, v, out, B, h, n_q, n_k, d_k, d_v, mask_kind=ATTN_MASK_NONE,
                     kv_lens=None, scale=0.0, stream=None):
    _check(library().attn_forward_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, h, n_q, n_k, d_k,
                                      d_v, mask_kind, _ptr(kv_lens), scale, _stream(stream)),
           "attn_forward_f32")


def mha_workspace_bytes(B, n_q, n_k, h, d_k, d_v) -> int:
    return int(library().mha_workspace_bytes(B, n_q, n_k, h, d_k, d_v))


def mha_forward(x_q, x_kv, w_q, w_k, w_v, w_o, out, B, n_q, n_k, d_model, h, d_k, d_v,
                mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, workspace=None,
                workspace_bytes=0, stream=None):
    _check(library().mha_forward(_ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                 _ptr(w_o), _ptr(out), B, n_q, n_k, d_model, h, d_k, d_v,
                                 mask_kind, _ptr(kv_lens), scale, _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "mha_forward")


def mha_forward_launches(B, n_q, n_k, d_model, h, d_k, d_v, self_attention) -> int:
    """Kernels mha_forward launches for these sizes (1, 2 or 3; 0 for no
    work; -1 for sizes it rejects)."""
    return int(library().mha_forward_launches(B, n_q, n_k, d_model, h, d_k, d_v,
                                              1 if self_attention else 0))


def mha_concat_heads(x_q, x_kv, w_q, w_k, w_v, concat, B, n_q, n_k, d_model, h, d_k, d_v,
                     mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, workspace=None,
                     workspace_bytes=0, stream=None):
    _check(library().mha_concat_heads(_ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                      _ptr(concat), B, n_q, n_k, d_model, h, d_k, d_v, mask_kind,
                                      _ptr(kv_lens), scale, _ptr(workspace), workspace_bytes,
                                      _stream(stream)), "mha_concat_heads")


def mha_project_qkv(x_q, x_kv, w_q, w_k, w_v, q_out, k_out, v_out, B, n_q, n_k, d_model, h, d_k,
                    d_v, stream=None):
    _check(library().mha_project_qkv(_ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                     _ptr(q_out), _ptr(k_out), _ptr(v_out), B, n_q, n_k, d_model,
                                     h, d_k, d_v, _stream(stream)), "mha_project_qkv")


def mha_project_out(concat, w_o, out, B, n_q, d_model, h, d_v, stream=None):
    _check(library().mha_project_out(_ptr(concat), _ptr(w_o), _ptr(out), B, n_q, d_model, h, d_v,
                                     _stream(stream)), "mha_project_out")


def mha_forward_noalloc(x_q, x_kv, w_q, w_k, w_v, w_o, out, B, n_q, n_k, d_model, h, d_k, d_v,
                        mask_kind=ATTN_MASK_NONE, kv_lens=None, scale=0.0, stream=None):
    """mha_forward on the library's fixed device scratch (no workspace argument;
    for callers that cannot allocate device memory)."""
    _check(library().mha_forward_noalloc(_ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                         _ptr(w_o), _ptr(out), B, n_q, n_k, d_model, h, d_k, d_v,
                                         mask_kind, _ptr(kv_lens), scale, _stream(stream)),
           "mha_forward_noalloc")


def attn_get_device_status(stream=None) -> int:
    """Returns the status code (does not raise on ATTN_ERR_DEVICE_*)."""
    return int(library().attn_get_device_status(_stream(stream)))


def attn_last_cuda_error() -> int:
    return int(library().attn_last_cuda_error())


def attn_status_string(status: int) -> str:
    return library().attn_status_string(status).decode()


def attn_selftest_wait_timeout(limit_us: int, stream=None):
    _check(library().attn_selftest_wait_timeout(limit_us, _stream(stream)),
           "attn_selftest_wait_timeout")


# ---------------------------------------------------------------- host buffers
# The *_host entry points take the step's inputs and result in host memory
# (pinned for asynchronous copies) and stage them through the workspace.

def attn_host_workspace_bytes(B, h, n_q, n_k, d_k, d_v) -> int:
    return int(library().attn_host_workspace_bytes(B, h, n_q, n_k, d_k, d_v))


def attn_forward_host(q_host, k_host, v_host, out_host, B, h, n_q, n_k, d_k, d_v,
                      mask_kind=ATTN_MASK_NONE, kv_lens_host=None, scale=0.0, workspace=None,
                      workspace_bytes=0, stream=None):
    _check(library().attn_forward_host(_ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(out_host),
                                       B, h, n_q, n_k, d_k, d_v, mask_kind, _ptr(kv_lens_host),
                                       scale, _ptr(workspace), workspace_bytes, _stream(stream)),
           "attn_forward_host")


def attn_forward_window_host(q_host, k_host, v_host, out_host, B, h, n_q, n_k, d_k, d_v,
                             window_left, window_right, mask_kind=ATTN_MASK_NONE,
                             kv_lens_host=None, scale=0.0, workspace=None, workspace_bytes=0,
                             stream=None):
    _check(library().attn_forward_window_host(_ptr(q_host), _ptr(k_host), _ptr(v_host),
                                              _ptr(out_host), B, h, n_q, n_k, d_k, d_v, mask_kind,
                                              _ptr(kv_lens_host), window_left, window_right,
                                              scale, _ptr(workspace), workspace_bytes,
                                              _stream(stream)),
           "attn_forward_window_host")


def mha_host_workspace_bytes(B, n_q, n_k, d_model, h, d_k, d_v) -> int:
    return int(library().mha_host_workspace_bytes(B, n_q, n_k, d_model, h, d_k, d_v))


def mha_forward_host(x_q_host, x_kv_host, w_q, w_k, w_v, w_o, out_host, B, n_q, n_k, d_model, h,
                     d_k, d_v, mask_kind=ATTN_MASK_NONE, kv_lens_host=None, scale=0.0,
                     workspace=None, workspace_bytes=0, stream=None):
    _check(library().mha_forward_host(_ptr(x_q_host), _ptr(x_kv_host), _ptr(w_q), _ptr(w_k),
                                      _ptr(w_v), _ptr(w_o), _ptr(out_host), B, n_q, n_k, d_model,
                                      h, d_k, d_v, mask_kind, _ptr(kv_lens_host), scale,
                                      _ptr(workspace), workspace_bytes, _stream(stream)),
           "mha_forward_host")


def mha_forward_host_async(x_q_host, x_kv_host, w_q, w_k, w_v, w_o, out_host, B, n_q, n_k,
                           d_model, h, d_k, d_v, mask_kind=ATTN_MASK_NONE, kv_lens_host=None,
                           scale=0.0, workspace=None, workspace_bytes=0, stream=None):
    """mha_forward_host with the result copy on the library's result stream:
    out_host is complete once `stream` has passed a later attn_host_join."""
    _check(library().mha_forward_host_async(_ptr(x_q_host), _ptr(x_kv_host), _ptr(w_q),
                                            _ptr(w_k), _ptr(w_v), _ptr(w_o), _ptr(out_host), B,
                                            n_q, n_k, d_model, h, d_k, d_v, mask_kind,
                                            _ptr(kv_lens_host), scale, _ptr(workspace),
                                            workspace_bytes, _stream(stream)),
           "mha_forward_host_async")


def attn_host_join(stream=None):
    _check(library().attn_host_join(_stream(stream)), "attn_host_join")


def encoder_layer_host_workspace_bytes(B, n, d_model, h, d_k, d_ff) -> int:
    return int(library().encoder_layer_host_workspace_bytes(B, n, d_model, h, d_k, d_ff))


def encoder_layer_forward_host(x_host, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1, w_2,
                               b_2, ln2_gamma, ln2_beta, out_host, B, n, d_model, h, d_k, d_ff,
                               mask_kind=ATTN_MASK_NONE, kv_lens_host=None, scale=0.0, eps=1e-6,
                               workspace=None, workspace_bytes=0, stream=None):
    ptrs = [_ptr(t) for t in (x_host, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1, w_2, b_2,
                              ln2_gamma, ln2_beta, out_host)]
    _check(library().encoder_layer_forward_host(*ptrs, B, n, d_model, h, d_k, d_ff, mask_kind,
                                                _ptr(kv_lens_host), scale, eps, _ptr(workspace),
                                                workspace_bytes, _stream(stream)),
           "encoder_layer_forward_host")


def encoder_layer_forward_host_async(x_host, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1,
                                     w_2, b_2, ln2_gamma, ln2_beta, out_host, B, n, d_model, h,
                                     d_k, d_ff, mask_kind=ATTN_MASK_NONE, kv_lens_host=None,
                                     scale=0.0, eps=1e-6, workspace=None, workspace_bytes=0,
                                     stream=None):
    """encoder_layer_forward_host with the result copy on the library's result
    stream: out_host is complete once `stream` has passed a later attn_host_join."""
    ptrs = [_ptr(t) for t in (x_host, w_q, w_k, w_v, w_o, ln1_gamma, ln1_beta, w_1, b_1, w_2, b_2,
                              ln2_gamma, ln2_beta, out_host)]
    _check(library().encoder_layer_forward_host_async(*ptrs, B, n, d_model, h, d_k, d_ff,
                                                      mask_kind, _ptr(kv_lens_host), scale, eps,
                                                      _ptr(workspace), workspace_bytes,
                                                      _stream(stream)),
           "encoder_layer_forward_host_async")


def attn_decode_host_workspace_bytes(B, h, n_q, n_max, d_k, d_v) -> int:
    return int(library().attn_decode_host_workspace_bytes(B, h, n_q, n_max, d_k, d_v))


def attn_decode_host(q_host, k_cache, v_cache, out_host, B, h, n_q, n_max, d_k, d_v,
                     cache_lens_host=None, scale=0.0, workspace=None, workspace_bytes=0,
                     stream=None):
    _check(library().attn_decode_host(_ptr(q_host), _ptr(k_cache), _ptr(v_cache), _ptr(out_host),
                                      B, h, n_q, n_max, d_k, d_v, _ptr(cache_lens_host), scale,
                                      _ptr(workspace), workspace_bytes, _stream(stream)),
           "attn_decode_host")


def attn_decode_host_async(q_host, k_cache, v_cache, out_host, B, h, n_q, n_max, d_k, d_v,
                           cache_lens_host=None, scale=0.0, workspace=None, workspace_bytes=0,
                           stream=None):
    """attn_decode_host with the result copy on the library's result stream:
    out_host is complete once `stream` has passed a later attn_host_join."""
    _check(library().attn_decode_host_async(_ptr(q_host), _ptr(k_cache), _ptr(v_cache),
                                            _ptr(out_host), B, h, n_q, n_max, d_k, d_v,
                                            _ptr(cache_lens_host), scale, _ptr(workspace),
                                            workspace_bytes, _stream(stream)),
           "attn_decode_host_async")
