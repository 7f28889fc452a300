"""Thin ctypes binding of libpa (include/pa.h): argument marshalling only.

Every function takes CUDA torch tensors, passes their device pointers and the
current torch stream to the C ABI, and raises ``PagedAttentionError`` on a
non-OK status.  There is no CPU path: the library must be built
(``paged_kv_cache_251_gb300.build``) and the tensors must live on a GPU.
"""
from __future__ import annotations

import ctypes
import functools
import math
from pathlib import Path

import torch

LIB_PATH = Path(__file__).resolve().parent / "_lib" / "libpa.so"

PA_OK, PA_ERR_INVALID_ARGUMENT, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE_TOO_SMALL, PA_ERR_CUDA = range(5)
PA_F32, PA_F16, PA_BF16, PA_I8, PA_E4M3 = 0, 1, 2, 3, 4
DEVERR_BAD_BLOCK, DEVERR_BAD_SLOT, DEVERR_BAD_PAIR, DEVERR_TIMEOUT, DEVERR_BAD_LEN, DEVERR_BAD_LAUNCH = 1, 2, 4, 8, 16, 32
DEVERR_BAD_INDEX, DEVERR_BAD_COUNT = 64, 128

DTYPE_CODE = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
# rotary frequency scalings of pa_rope_frequencies
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
# 8-bit caches: code pools are int8 or float8_e4m3fn tensors, scales float32
CODE_DTYPE = {torch.int8: PA_I8, torch.float8_e4m3fn: PA_E4M3}


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_lib.pa_status_string(status).decode()}: {detail}")
        self.status = status


def _load():
    if not LIB_PATH.exists():
        raise ImportError(f"libpa.so is not built ({LIB_PATH}); run paged_kv_cache_251_gb300.build.build()")
    lib = ctypes.CDLL(str(LIB_PATH))
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.pa_decode_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.pa_decode_workspace_size.restype = SZ
    lib.pa_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, I, I, P, SZ, P, P]
    lib.pa_decode.restype = I
    lib.pa_decode_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, I, I, P, P]
    lib.pa_decode_noalloc.restype = I
    lib.pa_decode_contiguous.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_contiguous.restype = I
    lib.pa_decode_noalloc_max_scratch.argtypes = []
    lib.pa_decode_noalloc_max_scratch.restype = SZ
    lib.pa_append_kv.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P, P]
    lib.pa_append_kv.restype = I
    lib.pa_copy_blocks.argtypes = [P, I, P, P, I, I, I, I, I, P, P]
    lib.pa_copy_blocks.restype = I
    lib.pa_decode_shared_prefix.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_shared_prefix.restype = I
    lib.pa_decode_shared_prefix_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    lib.pa_decode_shared_prefix_workspace_size.restype = SZ
    lib.pa_swap_blocks.argtypes = [P, I, P, P, P, P, I, I, I, I, I, I, P, P]
    lib.pa_swap_blocks.restype = I
    lib.pa_quant_page_bytes.argtypes = [I, I]
    lib.pa_quant_page_bytes.restype = SZ
    lib.pa_append_kv_quant.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, P, P]
    lib.pa_append_kv_quant.restype = I
    lib.pa_decode_quant.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_quant.restype = I
    lib.pa_copy_blocks_quant.argtypes = [P, I, P, P, I, I, I, I, P, P]
    lib.pa_copy_blocks_quant.restype = I
    lib.pa_swap_blocks_quant.argtypes = [P, I, P, P, P, P, I, I, I, I, I, P, P]
    lib.pa_swap_blocks_quant.restype = I
    D, LL = ctypes.c_double, ctypes.c_longlong
    lib.pa_rope_frequencies.argtypes = [P, I, D, I, D, D, D, D]
    lib.pa_rope_frequencies.restype = I
    lib.pa_rope.argtypes = [P, P, P, P, I, I, I, I, LL, LL, I, I, F, I, P]
    lib.pa_rope.restype = I
    lib.pa_rope_append_kv.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, LL, LL, LL, I, I, I, F, I, P, P]
    lib.pa_rope_append_kv.restype = I
    lib.pa_decode_tree.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_tree.restype = I
    lib.pa_decode_tree_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    lib.pa_decode_tree_workspace_size.restype = SZ
    lib.pa_decode_scored.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, LL, I, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_scored.restype = I
    lib.pa_decode_scored_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.pa_decode_scored_workspace_size.restype = SZ
    lib.pa_evict_select.argtypes = [P, P, P, P, P, I, I, I, I, LL, P, P]
    lib.pa_evict_select.restype = I
    lib.pa_compact_kv.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P]
    lib.pa_compact_kv.restype = I
    lib.pa_verify_drafts.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, LL, LL, I, P, P]
    lib.pa_verify_drafts.restype = I
    lib.pa_append_kv_block_quant.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.pa_append_kv_block_quant.restype = I
    lib.pa_append_kv_block_quant_workspace_size.argtypes = [I, I, I]
    lib.pa_append_kv_block_quant_workspace_size.restype = SZ
    lib.pa_decode_block_quant.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, I, I, P, SZ, P, P]
    lib.pa_decode_block_quant.restype = I
    lib.pa_decode_block_quant_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.pa_decode_block_quant_workspace_size.restype = SZ
    lib.pa_pages_update.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, SZ, P, P]
    lib.pa_pages_update.restype = I
    lib.pa_pages_compact.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, SZ, P, P]
    lib.pa_pages_compact.restype = I
    lib.pa_pages_workspace_size.argtypes = [I, I]
    lib.pa_pages_workspace_size.restype = SZ
    lib.pa_copy_pages.argtypes = [P, I, P, P, I, I, P, P]
    lib.pa_copy_pages.restype = I
    lib.pa_status_string.argtypes = [I]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_last_error_detail.argtypes = []
    lib.pa_last_error_detail.restype = ctypes.c_char_p
    lib.pa_version.argtypes = []
    lib.pa_version.restype = I
    return lib


_lib = _load()


def _check(status: int) -> None:
    if status != PA_OK:
        raise PagedAttentionError(status, _lib.pa_last_error_detail().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _own_workspace(stream, make, *args) -> torch.Tensor | None:
    """make(*args) for a call on `stream` that was given no workspace: the memory
    belongs to that stream (the call's own end is no end for the GPU; memory of
    another stream could be handed out there while the kernels still use it)."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("every tensor must be a contiguous CUDA tensor")


def pa_decode_workspace_size(num_seqs: int, num_heads: int, head_dim: int, block_size: int,
                             max_blocks_per_seq: int, window: int = 0, partition_size: int = 0) -> int:
    return int(_lib.pa_decode_workspace_size(num_seqs, num_heads, head_dim, block_size,
                                             max_blocks_per_seq, window, partition_size))


def workspace_for(q: torch.Tensor, block_size: int, max_blocks_per_seq: int, window: int = 0,
                  partition_size: int = 0) -> torch.Tensor | None:
    """A workspace tensor sized by pa_decode_workspace_size (None if 0 bytes)."""
    N, H, d = q.shape
    n = pa_decode_workspace_size(N, H, d, block_size, max_blocks_per_seq, window, partition_size)
    if n == 0:
        return None
    return torch.empty((n + 15) // 16 * 4, dtype=torch.float32, device=q.device)


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int | None = None,
              scale: float | None = None, window: int = 0, partition_size: int = 0,
              workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_s^T) V_s over sequence s's cached
    tokens, read through block_tables[s] (see include/pa.h)."""
    _cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace, err_word)
    N, H, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if q.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if workspace is None:
        workspace = _own_workspace(stream, workspace_for, q, bs, block_tables.shape[1], window, partition_size)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                          _ptr(context_lens), N, H, num_kv_heads, d, bs, float(scale), int(window),
                          DTYPE_CODE[q.dtype], DTYPE_CODE[out.dtype], block_tables.shape[1], nb,
                          int(partition_size), _ptr(workspace), ws_bytes, _ptr(err_word), _stream(stream)))
    return out


def pa_decode_shared_prefix_workspace_size(num_seqs: int, num_heads: int, head_dim: int, block_size: int,
                                           max_blocks_per_seq: int, partition_size: int, group_size: int,
                                           dtype: torch.dtype) -> int:
    return int(_lib.pa_decode_shared_prefix_workspace_size(num_seqs, num_heads, head_dim, block_size,
                                                           max_blocks_per_seq, partition_size, group_size,
                                                           DTYPE_CODE[dtype]))


def pa_decode_shared_prefix(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, shared_lens: torch.Tensor,
                            group_size: int, num_kv_heads: int | None = None, scale: float | None = None,
                            partition_size: int = 0, workspace: torch.Tensor | None = None,
                            err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_decode for consecutive groups of group_size sequences whose first
    shared_lens[g] tokens are the same blocks: each shared block is read once
    per group (see include/pa.h)."""
    _cuda(out, q, k_cache, v_cache, block_tables, context_lens, shared_lens, workspace, err_word)
    N, H, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for t in (block_tables, context_lens, shared_lens):
        if t.dtype != torch.int32:
            raise TypeError("block_tables, context_lens and shared_lens must be int32")
    if q.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if workspace is None:
        n = pa_decode_shared_prefix_workspace_size(N, H, d, bs, block_tables.shape[1], partition_size, group_size,
                                                   q.dtype)
        workspace = _own_workspace(stream, _bytes, max(n, 16), q.device)
    _check(_lib.pa_decode_shared_prefix(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                        _ptr(context_lens), _ptr(shared_lens), int(group_size), N, H, num_kv_heads,
                                        d, bs, float(scale), DTYPE_CODE[q.dtype], DTYPE_CODE[out.dtype],
                                        block_tables.shape[1], nb, int(partition_size), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(err_word),
                                        _stream(stream)))
    return out


def pa_decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int | None = None,
                      scale: float | None = None, window: int = 0, partition_size: int = 0,
                      err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_decode for callers that cannot allocate device memory: the partials'
    scratch is the library's built-in array (pa_decode_noalloc_max_scratch()
    bytes), shared by all calls on a device, so calls must not overlap on the
    GPU.  This wrapper allocates nothing either."""
    _cuda(out, q, k_cache, v_cache, block_tables, context_lens, err_word)
    N, H, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if q.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    _check(_lib.pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                  _ptr(context_lens), N, H, num_kv_heads, d, bs, float(scale), int(window),
                                  DTYPE_CODE[q.dtype], DTYPE_CODE[out.dtype], block_tables.shape[1], nb,
                                  int(partition_size), _ptr(err_word), _stream(stream)))
    return out


def pa_decode_contiguous(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         context_lens: torch.Tensor, num_kv_heads: int | None = None, scale: float | None = None,
                         window: int = 0, partition_size: int = 0, workspace: torch.Tensor | None = None,
                         err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_decode over contiguous caches [N, H_kv, L, d] (no block table; see
    include/pa.h)."""
    _cuda(out, q, k_cache, v_cache, context_lens, workspace, err_word)
    N, H, d = q.shape
    n2, hkv, L, d2 = k_cache.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if context_lens.dtype != torch.int32:
        raise TypeError("context_lens must be int32")
    if q.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if workspace is None:
        workspace = _own_workspace(stream, workspace_for, q, 16, max(1, L // 16), window, partition_size)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode_contiguous(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(context_lens), N, H,
                                     num_kv_heads, d, L, float(scale), int(window), DTYPE_CODE[q.dtype],
                                     DTYPE_CODE[out.dtype], int(partition_size), _ptr(workspace), ws_bytes,
                                     _ptr(err_word), _stream(stream)))
    return out


def pa_decode_noalloc_max_scratch() -> int:
    return int(_lib.pa_decode_noalloc_max_scratch())


def pa_append_kv(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Store token i's K/V rows at slot_mapping[i] (see include/pa.h)."""
    _cuda(k, v, slot_mapping, k_cache, v_cache, err_word)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("k, v and the caches must share one dtype")
    nb, hkv, bs, d = k_cache.shape
    _check(_lib.pa_append_kv(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                             slot_mapping.numel(), hkv, d, bs, nb, DTYPE_CODE[k_cache.dtype],
                             _ptr(err_word), _stream(stream)))


def pa_copy_blocks(src_dst_pairs: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   err_word: torch.Tensor | None = None, stream=None) -> None:
    """Copy block src onto block dst (K and V, all kv heads) for every pair."""
    _cuda(src_dst_pairs, k_cache, v_cache, err_word)
    if src_dst_pairs.dtype != torch.int64:
        raise TypeError("src_dst_pairs must be int64")
    nb, hkv, bs, d = k_cache.shape
    _check(_lib.pa_copy_blocks(_ptr(src_dst_pairs), src_dst_pairs.numel() // 2, _ptr(k_cache),
                               _ptr(v_cache), hkv, d, bs, nb, DTYPE_CODE[k_cache.dtype],
                               _ptr(err_word), _stream(stream)))


def pa_swap_blocks(src_dst_pairs: torch.Tensor, src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor,
                   dst_v: torch.Tensor, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Copy block src of (src_k, src_v) onto block dst of (dst_k, dst_v) for
    every pair.  Pools and pairs may be CUDA tensors or pinned host tensors
    (the GPU reads / writes host memory directly)."""
    for t in (src_dst_pairs, src_k, src_v, dst_k, dst_v):
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools and pairs must be contiguous CUDA tensors or pinned host tensors")
    if err_word is not None:
        _cuda(err_word)
    if src_dst_pairs.dtype != torch.int64:
        raise TypeError("src_dst_pairs must be int64")
    if src_k.dtype != dst_k.dtype or src_v.dtype != src_k.dtype or dst_v.dtype != src_k.dtype:
        raise TypeError("both pools must share one dtype")
    snb, hkv, bs, d = src_k.shape
    dnb, hkv2, bs2, d2 = dst_k.shape
    if (hkv, bs, d) != (hkv2, bs2, d2) or src_v.shape != src_k.shape or dst_v.shape != dst_k.shape:
        raise ValueError("both pools must share the block layout")
    _check(_lib.pa_swap_blocks(_ptr(src_dst_pairs), src_dst_pairs.numel() // 2, _ptr(src_k), _ptr(src_v),
                               _ptr(dst_k), _ptr(dst_v), snb, dnb, hkv, d, bs, DTYPE_CODE[src_k.dtype],
                               _ptr(err_word), _stream(stream)))


def pa_quant_page_bytes(head_dim: int, block_size: int) -> int:
    """Bytes of one (block, kv head) page of an 8-bit pool: block_size code rows
    of head_dim bytes, then the rows holding their fp32 scales."""
    return int(_lib.pa_quant_page_bytes(head_dim, block_size))


def quant_pool_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int) -> tuple:
    """Shape of an 8-bit pool tensor: [num_blocks, H_kv, page rows, head_dim]."""
    return (num_blocks, num_kv_heads, pa_quant_page_bytes(head_dim, block_size) // head_dim, head_dim)


def _pool_block_size(pool: torch.Tensor) -> int:
    if pool.dtype not in CODE_DTYPE or pool.dim() != 4:
        raise TypeError("8-bit pools are int8 / float8_e4m3fn tensors [num_blocks, H_kv, page rows, head_dim]")
    rows, d = pool.shape[2], pool.shape[3]
    for bs in (8, 16, 32):
        if pa_quant_page_bytes(d, bs) == rows * d:
            return bs
    raise ValueError(f"a {rows}-row page at head_dim {d} matches no block size")


def pa_append_kv_quant(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Quantise token i's K/V rows (fp32/fp16/bf16) into the 8-bit pages at
    slot_mapping[i]: codes into the slot's row, the row scale into the page's
    scale rows (see include/pa.h)."""
    _cuda(k, v, slot_mapping, k_cache, v_cache, err_word)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    bs = _pool_block_size(k_cache)
    if k.dtype != v.dtype or k_cache.dtype != v_cache.dtype or k_cache.shape != v_cache.shape:
        raise TypeError("k and v share one dtype, the page pools another and one shape")
    nb, hkv, _, d = k_cache.shape
    _check(_lib.pa_append_kv_quant(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                   slot_mapping.numel(), hkv, d, bs, nb, DTYPE_CODE[k.dtype],
                                   CODE_DTYPE[k_cache.dtype], _ptr(err_word), _stream(stream)))


def pa_decode_quant(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int | None = None,
                    scale: float | None = None, window: int = 0, partition_size: int = 0,
                    workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """pa_decode over 8-bit pages: every cached element is code * scale of its
    row (see include/pa.h)."""
    _cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace, err_word)
    N, H, d = q.shape
    bs = _pool_block_size(k_cache)
    nb, hkv, _, d2 = k_cache.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
        raise TypeError("k_cache and v_cache must share one code dtype and shape")
    if workspace is None:
        workspace = _own_workspace(stream, workspace_for, q, bs, block_tables.shape[1], window, partition_size)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode_quant(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                _ptr(context_lens), N, H, num_kv_heads, d, bs, float(scale), int(window),
                                DTYPE_CODE[q.dtype], CODE_DTYPE[k_cache.dtype], DTYPE_CODE[out.dtype],
                                block_tables.shape[1], nb, int(partition_size), _ptr(workspace), ws_bytes,
                                _ptr(err_word), _stream(stream)))
    return out


def pa_copy_blocks_quant(src_dst_pairs: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         err_word: torch.Tensor | None = None, stream=None) -> None:
    """pa_copy_blocks for 8-bit pools: whole pages (codes and scales)."""
    _cuda(src_dst_pairs, k_cache, v_cache, err_word)
    if src_dst_pairs.dtype != torch.int64:
        raise TypeError("src_dst_pairs must be int64")
    bs = _pool_block_size(k_cache)
    nb, hkv, _, d = k_cache.shape
    _check(_lib.pa_copy_blocks_quant(_ptr(src_dst_pairs), src_dst_pairs.numel() // 2, _ptr(k_cache),
                                     _ptr(v_cache), hkv, d, bs, nb, _ptr(err_word), _stream(stream)))


def pa_swap_blocks_quant(src_dst_pairs: torch.Tensor, src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor,
                         dst_v: torch.Tensor, err_word: torch.Tensor | None = None, stream=None) -> None:
    """pa_swap_blocks for 8-bit pools: whole pages (CUDA or pinned host tensors)."""
    for t in (src_dst_pairs, src_k, src_v, dst_k, dst_v):
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools and pairs must be contiguous CUDA tensors or pinned host tensors")
    if err_word is not None:
        _cuda(err_word)
    if src_dst_pairs.dtype != torch.int64:
        raise TypeError("src_dst_pairs must be int64")
    bs = _pool_block_size(src_k)
    snb, hkv, rows, d = src_k.shape
    dnb, hkv2, rows2, d2 = dst_k.shape
    if (hkv, rows, d) != (hkv2, rows2, d2) or src_k.dtype != dst_k.dtype:
        raise ValueError("both pools must share the page layout and code dtype")
    _check(_lib.pa_swap_blocks_quant(_ptr(src_dst_pairs), src_dst_pairs.numel() // 2, _ptr(src_k), _ptr(src_v),
                                     _ptr(dst_k), _ptr(dst_v), snb, dnb, hkv, d, bs, _ptr(err_word),
                                     _stream(stream)))


# ---------------------------------------------------------------------------
# Serving-step operators (rotary positions, tree attention, scored decode,
# eviction)


# These calls are short beside their launch, so their checks are written to cost
# little: one pass over the tensors, addresses passed as integers.


def _dense(first: torch.Tensor, *rest) -> int:
    """The CUDA device index that all tensors share; each must be contiguous."""
    dev = first.get_device()
    if dev < 0 or not first.is_contiguous():
        raise ValueError("every tensor must be a contiguous CUDA tensor")
    for t in rest:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            if t.is_cuda and t.is_contiguous():
                raise ValueError("every tensor must be on one device")
            raise ValueError("every tensor must be a contiguous CUDA tensor")
    return dev


# The current stream's handle and the current device, by torch's inner names where it
# has them (the public ones make objects on the way, of a call of 11 us), else by the
# public ones.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: torch.cuda.current_device())


def _call(fn, dev: int, stream, *args) -> None:
    """Run a library call on `stream` (default: the device's current one) with
    device `dev` current."""
    if stream is None:
        raw = _raw_stream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError("the stream is on another device than the tensors")
        raw = stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != PA_OK:
        _check(status)


def _shapes(*checks) -> None:
    """Tensor, shape, name, and so on: the tensors (None aside) have those shapes."""
    for i in range(0, len(checks), 3):
        t = checks[i]
        if t is not None and t.shape != checks[i + 1]:
            raise ValueError(f"{checks[i + 2]} has shape {tuple(t.shape)}, expected {tuple(checks[i + 1])}")


def _int32(*checks) -> None:
    """Tensor, name, and so on: the tensors (None aside) are int32."""
    i32 = torch.int32
    for i in range(0, len(checks), 2):
        t = checks[i]
        if t is not None and t.dtype is not i32:
            raise TypeError(f"{checks[i + 1]} must be int32")


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _ws_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.nbytes


def _ws(nbytes: int, device) -> torch.Tensor | None:
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=device) if nbytes else None


def _rows(t: torch.Tensor, name: str) -> int:
    """The row stride, in elements, of a [tokens, heads, d] tensor whose rows are
    dense (a slice of a wider projection, for instance)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    at = t.stride()
    if n and ((h > 1 and at[1] != d) or at[2] != 1):
        raise ValueError(f"{name}: each token's heads must be dense")
    return at[0] if n > 1 else h * d


def pa_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                        original_len: float = 0.0, low: float = 1.0, high: float = 4.0) -> torch.Tensor:
    """Rotation frequencies (radians per position) as a CPU double tensor
    [rot_dim / 2]: scaling "none", "linear", "base" or "ramp" (see
    include/pa.h).  Copy it to the GPU once and pass it to the rope calls."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"unknown scaling {scaling!r}")
    out = torch.empty(max(rot_dim // 2, 1), dtype=torch.float64)
    _check(_lib.pa_rope_frequencies(_ptr(out), int(rot_dim), float(base), ROPE_SCALING[scaling], float(factor),
                                    float(original_len), float(low), float(high)))
    return out


def pa_rope(out: torch.Tensor, x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
            interleaved: bool = False, inverse: bool = False, mscale: float = 1.0, stream=None) -> torch.Tensor:
    """out[i, h] = x[i, h] rotated to positions[i] (back by it when inverse:
    the gradient of the rotation).  rot_dim is 2 * freqs.numel(); out may be x."""
    dev = _dense(positions, freqs)
    if x.get_device() != dev or out.get_device() != dev:
        raise ValueError("every tensor must be a CUDA tensor on one device")
    n, h, d = x.shape
    _shapes(out, x.shape, "out", positions, (n,), "positions")
    if positions.dtype != torch.int32 or freqs.dtype != torch.float64 or freqs.dim() != 1:
        raise TypeError("positions must be int32 and freqs a double vector")
    if out.dtype != x.dtype:
        raise TypeError("out and x must share one dtype")
    _call(_lib.pa_rope, dev, stream, out.data_ptr(), x.data_ptr(), positions.data_ptr(), freqs.data_ptr(), n, h, d,
          2 * freqs.numel(), _rows(x, "x"), _rows(out, "out"), int(interleaved), -1 if inverse else 1, float(mscale),
          DTYPE_CODE[x.dtype])
    return out


def pa_rope_append_kv(q_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      positions: torch.Tensor, slot_mapping: torch.Tensor, freqs: torch.Tensor,
                      k_cache: torch.Tensor, v_cache: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                      err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotate q into q_out and k into its cache slots, store v in its slots (see
    include/pa.h).  q, k and v may be slices of one projection: their rows may
    be any distance apart."""
    dev = _dense(q_out, positions, slot_mapping, freqs, k_cache, v_cache, err_word)
    if q.get_device() != dev or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("every tensor must be a CUDA tensor on one device")
    n, h, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _shapes(q_out, q.shape, "q_out", k, (n, hkv, d), "k", v, (n, hkv, d), "v", k_cache, (nb, hkv, bs, d), "k_cache",
            v_cache, k_cache.shape, "v_cache", positions, (n,), "positions", slot_mapping, (n,), "slot_mapping")
    if positions.dtype != torch.int32 or slot_mapping.dtype != torch.int64:
        raise TypeError("positions must be int32 and slot_mapping int64")
    if freqs.dtype != torch.float64 or freqs.dim() != 1:
        raise TypeError("freqs must be a double vector")
    dt = q.dtype
    if q_out.dtype != dt or k.dtype != dt or v.dtype != dt or k_cache.dtype != dt or v_cache.dtype != dt:
        raise TypeError("q, k, v, q_out and the caches must share one dtype")
    _call(_lib.pa_rope_append_kv, dev, stream, q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          positions.data_ptr(), slot_mapping.data_ptr(), freqs.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), n, h,
          hkv, d, 2 * freqs.numel(), _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), bs, nb, int(interleaved),
          float(mscale), DTYPE_CODE[dt], _addr(err_word))
    return q_out


def pa_decode_tree_workspace_size(num_seqs: int, num_draft: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                  block_size: int, max_blocks_per_seq: int, dtype: torch.dtype) -> int:
    return int(_lib.pa_decode_tree_workspace_size(num_seqs, num_draft, num_heads, num_kv_heads, head_dim, block_size,
                                                  max_blocks_per_seq, DTYPE_CODE[dtype]))


def tree_workspace_for(q: torch.Tensor, k_cache: torch.Tensor, max_blocks_per_seq: int) -> torch.Tensor | None:
    """A workspace tensor for pa_decode_tree (None if 0 bytes)."""
    n, t, h, d = q.shape
    return _ws(pa_decode_tree_workspace_size(n, t, h, k_cache.shape[1], d, k_cache.shape[2], max_blocks_per_seq,
                                             k_cache.dtype), q.device)


def tree_mask_from_parents(parents: torch.Tensor) -> torch.Tensor:
    """The mask of pa_decode_tree for trees given by parents, an integer tensor
    [N, T]: parents[s, i] < i is the drafted token before token i, or negative
    when it follows the last committed token.  A token attends itself and its
    ancestors.  Returns int64 [N, T, ceil(T / 64)] on the device of parents.  Works
    on the host: parents on a GPU are waited for and copied, so not during a capture."""
    n, t = parents.shape
    p = parents.to("cpu", torch.int64)
    if bool((p >= torch.arange(t)).any()):
        raise ValueError("a token's parent must come before it")
    seen = torch.zeros((n, t, t), dtype=torch.bool)
    rows = torch.arange(n)
    for i in range(t):
        up = p[:, i]
        seen[:, i] = seen[rows, up.clamp_min(0)] & (up >= 0)[:, None]
        seen[:, i, i] = True
    words = (t + 63) // 64
    bits = torch.zeros((n, t, words * 64), dtype=torch.int64)
    bits[:, :, :t] = seen
    one = torch.ones(64, dtype=torch.int64) << torch.arange(64)
    return (bits.view(n, t, words, 64) * one).sum(-1).to(parents.device)


def _check_paged(q, k_cache, v_cache, block_tables, context_lens, n, h, d) -> tuple:
    nb, hkv, bs, d2 = k_cache.shape
    _shapes(k_cache, (nb, hkv, bs, d), "k_cache", v_cache, k_cache.shape, "v_cache", context_lens, (n,),
            "context_lens")
    if block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("block_tables must be [N, max_blocks_per_seq]")
    _int32(block_tables, "block_tables", context_lens, "context_lens")
    if q.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    return nb, hkv, bs


def pa_decode_tree(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor, tree_mask: torch.Tensor | None = None,
                   draft_lens: torch.Tensor | None = None, scale: float | None = None,
                   workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Attention of each sequence's drafted tokens (q, out: [N, T, H, d]) over
    its committed tokens and the drafted ones its mask names; the drafted
    tokens are the last draft_lens[s] of the context_lens[s] cached ones.
    tree_mask None: a chain (see include/pa.h)."""
    dev = _dense(out, q, k_cache, v_cache, block_tables, context_lens, tree_mask, draft_lens, workspace, err_word)
    n, t, h, d = q.shape
    nb, hkv, bs = _check_paged(q, k_cache, v_cache, block_tables, context_lens, n, h, d)
    _shapes(out, q.shape, "out")
    _int32(draft_lens, "draft_lens")
    _shapes(draft_lens, (n,), "draft_lens")
    if tree_mask is not None:
        if tree_mask.dtype != torch.int64:
            raise TypeError("tree_mask must be int64 (64 bits a word)")
        _shapes(tree_mask, (n, t, (t + 63) // 64), "tree_mask")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = _own_workspace(stream, tree_workspace_for, q, k_cache, block_tables.shape[1])
    _call(_lib.pa_decode_tree, dev, stream, out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          block_tables.data_ptr(), context_lens.data_ptr(), _addr(draft_lens), _addr(tree_mask), n, t, h, hkv, d, bs,
          float(scale), DTYPE_CODE[q.dtype], DTYPE_CODE[out.dtype], block_tables.shape[1], nb, _addr(workspace),
          _ws_bytes(workspace), _addr(err_word))
    return out


def pa_decode_scored_workspace_size(num_seqs: int, num_heads: int, head_dim: int, block_size: int,
                                    max_blocks_per_seq: int, partition_size: int = 0) -> int:
    return int(_lib.pa_decode_scored_workspace_size(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq,
                                                    partition_size))


def scored_workspace_for(q: torch.Tensor, k_cache: torch.Tensor, max_blocks_per_seq: int,
                         partition_size: int = 0) -> torch.Tensor | None:
    """A workspace tensor for pa_decode_scored (None if 0 bytes)."""
    n, h, d = q.shape
    return _ws(pa_decode_scored_workspace_size(n, h, d, k_cache.shape[2], max_blocks_per_seq, partition_size),
               q.device)


def pa_decode_scored(out: torch.Tensor, scores_out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                     scores_in: torch.Tensor | None = None, scale: float | None = None, partition_size: int = 0,
                     workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """pa_decode, and scores_out[s, kvh, t] = scores_in[s, kvh, t] (None: 0) +
    the softmax weights token t gets from the kv head's query heads (see
    include/pa.h).  Scores are fp32 [N, H_kv, at least max_blocks * block_size]."""
    dev = _dense(out, scores_out, q, k_cache, v_cache, block_tables, context_lens, scores_in, workspace, err_word)
    n, h, d = q.shape
    nb, hkv, bs = _check_paged(q, k_cache, v_cache, block_tables, context_lens, n, h, d)
    _shapes(out, q.shape, "out")
    if scores_out.dim() != 3 or scores_out.shape[:2] != (n, hkv):
        raise ValueError("scores_out must be [N, H_kv, tokens]")
    if scores_in is not None:
        _shapes(scores_in, scores_out.shape, "scores_in")
    if scores_out.dtype != torch.float32 or (scores_in is not None and scores_in.dtype != torch.float32):
        raise TypeError("scores must be float32")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = _own_workspace(stream, scored_workspace_for, q, k_cache, block_tables.shape[1], partition_size)
    _call(_lib.pa_decode_scored, dev, stream, out.data_ptr(), scores_out.data_ptr(), _addr(scores_in), q.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), n, h, hkv, d, bs,
          float(scale), scores_out.shape[2], DTYPE_CODE[q.dtype], DTYPE_CODE[out.dtype], block_tables.shape[1], nb,
          int(partition_size), _addr(workspace), _ws_bytes(workspace), _addr(err_word))
    return out


def pa_evict_select(keep: torch.Tensor, new_lens: torch.Tensor, scores_out: torch.Tensor | None,
                    scores: torch.Tensor, context_lens: torch.Tensor, budget: int, recent: int,
                    err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The cached tokens every kv head keeps: its `recent` last ones and those of
    the others with the largest scores, `budget` in all, ascending in keep
    [N, H_kv, budget] (-1 past new_lens); their scores move to the front of
    scores_out (which may be scores, or None).  See include/pa.h."""
    dev = _dense(keep, new_lens, scores_out, scores, context_lens, err_word)
    if scores.dim() != 3 or scores.dtype != torch.float32:
        raise TypeError("scores must be float32 [N, H_kv, tokens]")
    n, hkv, stride = scores.shape
    if scores_out is not None:
        _shapes(scores_out, scores.shape, "scores_out")
        if scores_out.dtype != torch.float32:
            raise TypeError("scores_out must be float32")
    _shapes(keep, (n, hkv, budget), "keep", new_lens, (n,), "new_lens", context_lens, (n,), "context_lens")
    _int32(keep, "keep", new_lens, "new_lens", context_lens, "context_lens")
    _call(_lib.pa_evict_select, dev, stream, keep.data_ptr(), new_lens.data_ptr(), _addr(scores_out),
          scores.data_ptr(), context_lens.data_ptr(), n, hkv, int(budget), int(recent), stride, _addr(err_word))
    return keep


def pa_compact_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, keep: torch.Tensor, keep_lens: torch.Tensor,
                  block_tables: torch.Tensor, dst_block_tables: torch.Tensor | None = None,
                  base_lens: torch.Tensor | None = None, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Token base_lens[s] + i takes the K/V rows of token base_lens[s] +
    keep[s, h, i], for i < keep_lens[s] (keep [N, H_kv or 1, n]): in place, or
    into the blocks of dst_block_tables.  See include/pa.h."""
    dev = _dense(k_cache, v_cache, keep, keep_lens, block_tables, dst_block_tables, base_lens, err_word)
    nb, hkv, bs, d = k_cache.shape
    _shapes(v_cache, k_cache.shape, "v_cache")
    if v_cache.dtype != k_cache.dtype:
        raise TypeError("the caches must share one dtype")
    if keep.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("keep must be [N, H_kv or 1, n] and block_tables [N, max_blocks_per_seq]")
    n = keep.shape[0]
    _int32(keep, "keep", keep_lens, "keep_lens", block_tables, "block_tables", dst_block_tables, "dst_block_tables",
           base_lens, "base_lens")
    _shapes(keep_lens, (n,), "keep_lens", base_lens, (n,), "base_lens")
    if block_tables.shape[0] != n or (dst_block_tables is not None and
                                      (dst_block_tables.dim() != 2 or dst_block_tables.shape[0] != n)):
        raise ValueError("block_tables and dst_block_tables must be [N, max_blocks_per_seq]")
    _call(_lib.pa_compact_kv, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), keep.data_ptr(),
          keep_lens.data_ptr(), _addr(base_lens), block_tables.data_ptr(), _addr(dst_block_tables), n, keep.shape[1],
          keep.shape[2], hkv, d, bs, block_tables.shape[1],
          0 if dst_block_tables is None else dst_block_tables.shape[1], nb, DTYPE_CODE[k_cache.dtype],
          _addr(err_word))


# ---------------------------------------------------------------------------
# Verification of drafted tokens, block-scaled 8-bit caches, page tables on the
# device


def _prob_rows(t: torch.Tensor, name: str, n: int, rows: int) -> int:
    """The row stride, in elements, of [n, rows, vocab] probabilities whose rows are
    a fixed distance apart (a padded vocabulary cut to size, for instance)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n or shape[1] != rows:
        raise ValueError(f"{name} must be [{n}, {rows}, vocab]")
    if t.is_contiguous():
        return shape[2]
    a, b, c = t.stride()
    v = t.shape[2]
    if rows == 1:
        b = a if n > 1 else v
    if t.numel() and ((c != 1 and v > 1) or (n > 1 and a != rows * b) or b < v):
        raise ValueError(f"{name}: entries must be dense and rows a fixed distance apart")
    return b


def pa_verify_drafts(accept_lens: torch.Tensor, accepted: torch.Tensor, tokens: torch.Tensor,
                     target_probs: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                     draft_probs: torch.Tensor | None = None, draft_lens: torch.Tensor | None = None,
                     parents: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Which drafted tokens [N, T] are kept, and the token after them, given the
    target's probabilities [N, T + 1, V] (row i + 1: after drafted token i), the
    draft's [N, T, V] (row i: behind drafted token i - 1; None: the drafted tokens
    were chosen, not drawn) and random numbers [N, T + 1].  accepted [N, T] is a
    keep list of pa_compact_kv, tokens [N, T + 1] the accepted tokens and the
    next one, -1 behind them.  parents None: a chain (see include/pa.h)."""
    dev = _dense(accept_lens, accepted, tokens, draft_tokens, uniforms, draft_lens, parents, err_word)
    if target_probs.get_device() != dev or (draft_probs is not None and draft_probs.get_device() != dev):
        raise ValueError("every tensor must be a CUDA tensor on one device")
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be [N, T]")
    n, t = draft_tokens.shape
    target_stride = _prob_rows(target_probs, "target_probs", n, t + 1)
    v = target_probs.shape[2]
    draft_stride = 0
    if draft_probs is not None:
        draft_stride = _prob_rows(draft_probs, "draft_probs", n, t)
        if draft_probs.shape[2] != v or draft_probs.dtype is not target_probs.dtype:
            raise ValueError("target_probs and draft_probs must share vocabulary and dtype")
    _shapes(accept_lens, (n,), "accept_lens", accepted, (n, t), "accepted", tokens, (n, t + 1), "tokens", uniforms,
            (n, t + 1), "uniforms", draft_lens, (n,), "draft_lens", parents, (n, t), "parents")
    _int32(accept_lens, "accept_lens", accepted, "accepted", tokens, "tokens", draft_tokens, "draft_tokens", draft_lens,
           "draft_lens", parents, "parents")
    if uniforms.dtype is not torch.float32 or target_probs.dtype not in DTYPE_CODE:
        raise TypeError("uniforms must be float32, the probabilities float32, float16 or bfloat16")
    _call(_lib.pa_verify_drafts, dev, stream, accept_lens.data_ptr(), accepted.data_ptr(), tokens.data_ptr(),
          target_probs.data_ptr(), _addr(draft_probs), draft_tokens.data_ptr(), _addr(draft_lens), _addr(parents),
          uniforms.data_ptr(), n, t, v, target_stride, draft_stride, DTYPE_CODE[target_probs.dtype], _addr(err_word))
    return tokens


def _block_quant_pool(k_cache, v_cache, k_scales, v_scales) -> tuple:
    """(blocks, kv heads, block size, head_dim, code) of a block-scaled cache."""
    shape, code = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or code not in CODE_DTYPE or v_cache.dtype is not code:
        raise TypeError("the caches must be int8 / float8_e4m3fn codes [blocks, H_kv, block_size, head_dim]")
    per_head = shape[:2]
    _shapes(v_cache, shape, "v_cache", k_scales, per_head, "k_scales", v_scales, per_head, "v_scales")
    if k_scales.dtype is not torch.float32 or v_scales.dtype is not torch.float32:
        raise TypeError("k_scales and v_scales must be float32")
    return *shape, CODE_DTYPE[code]


def append_block_quant_workspace_for(slot_mapping: torch.Tensor, k_cache: torch.Tensor) -> torch.Tensor | None:
    """A workspace tensor for pa_append_kv_block_quant (None if 0 bytes)."""
    return _ws(int(_lib.pa_append_kv_block_quant_workspace_size(slot_mapping.numel(), k_cache.shape[2],
                                                                k_cache.shape[0])), k_cache.device)


def pa_append_kv_block_quant(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                             workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                             stream=None) -> None:
    """Store token i's K/V rows (fp32/fp16/bf16) as 8-bit codes at slot_mapping[i];
    a block's scale for each kv head ([blocks, H_kv]) grows with its rows, and
    what it held is coded again (see include/pa.h)."""
    dev = _dense(k, v, slot_mapping, k_cache, v_cache, k_scales, v_scales, workspace, err_word)
    nb, hkv, bs, d, code = _block_quant_pool(k_cache, v_cache, k_scales, v_scales)
    n = slot_mapping.numel()
    rows = (n, hkv, d)
    _shapes(k, rows, "k", v, rows, "v")
    if slot_mapping.dtype is not torch.int64:
        raise TypeError("slot_mapping must be int64")
    dtype = k.dtype
    if v.dtype is not dtype or dtype not in DTYPE_CODE:
        raise TypeError("k and v must share one of float32, float16, bfloat16")
    if workspace is None:
        workspace = _own_workspace(stream, append_block_quant_workspace_for, slot_mapping, k_cache)
    _call(_lib.pa_append_kv_block_quant, dev, stream, k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), n, hkv, d, bs, nb,
          DTYPE_CODE[dtype], code, _addr(workspace), _ws_bytes(workspace), _addr(err_word))


def block_quant_workspace_for(q: torch.Tensor, k_cache: torch.Tensor, max_blocks_per_seq: int) -> torch.Tensor | None:
    """A workspace tensor for pa_decode_block_quant (None if 0 bytes)."""
    n, h, d = q.shape
    return _ws(int(_lib.pa_decode_block_quant_workspace_size(n, h, k_cache.shape[1], d, k_cache.shape[2],
                                                             max_blocks_per_seq)), q.device)


def pa_decode_block_quant(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                          context_lens: torch.Tensor, scale: float | None = None, window: int = 0,
                          workspace: torch.Tensor | None = None, err_word: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """pa_decode over 8-bit codes [blocks, H_kv, block_size, d] with one scale for
    each block and kv head (see include/pa.h)."""
    dev = _dense(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, workspace, err_word)
    shape, table = q.shape, block_tables.shape
    n, h, d = shape
    nb, hkv, bs, d2, code = _block_quant_pool(k_cache, v_cache, k_scales, v_scales)
    if d2 != d:
        raise ValueError(f"k_cache has head_dim {d2}, expected {d}")
    _shapes(out, shape, "out", context_lens, (n,), "context_lens")
    if len(table) != 2 or table[0] != n:
        raise ValueError("block_tables must be [N, max_blocks_per_seq]")
    _int32(block_tables, "block_tables", context_lens, "context_lens")
    dtype, out_dtype = DTYPE_CODE.get(q.dtype), DTYPE_CODE.get(out.dtype)
    if dtype is None or out_dtype is None:
        raise TypeError("q and out must be float32, float16 or bfloat16")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = _own_workspace(stream, block_quant_workspace_for, q, k_cache, table[1])
    _call(_lib.pa_decode_block_quant, dev, stream, out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
          context_lens.data_ptr(), n, h, hkv, d, bs, float(scale), int(window), dtype, code, out_dtype, table[1], nb,
          _addr(workspace), _ws_bytes(workspace), _addr(err_word))
    return out


def pages_workspace_for(tables: torch.Tensor, ref_counts: torch.Tensor, num_rows: int = 0) -> torch.Tensor:
    """A workspace tensor for pa_pages_update (to num_rows rows, if more than
    tables has) and pa_pages_compact."""
    return _ws(int(_lib.pa_pages_workspace_size(max(num_rows, tables.shape[0]), ref_counts.numel())), tables.device)


def _check_pages(new_tables, new_ref_counts, pairs, status, tables, ref_counts, lens) -> tuple:
    """(old rows, max_blocks_per_seq, new rows, blocks, pairs)."""
    old, new, blocks, moves = tables.shape, new_tables.shape, ref_counts.shape, pairs.shape
    if len(old) != 2 or len(new) != 2 or new[1] != old[1]:
        raise ValueError("tables and new_tables must be [rows, max_blocks_per_seq]")
    if len(blocks) != 1 or len(moves) != 2 or moves[1] != 2:
        raise ValueError("ref_counts must be [blocks] and pairs [n, 2]")
    _shapes(new_ref_counts, blocks, "new_ref_counts", status, (4,), "status", lens, old[:1], "lens")
    _int32(new_tables, "new_tables", new_ref_counts, "new_ref_counts", status, "status", tables, "tables", ref_counts,
           "ref_counts", lens, "lens")
    if pairs.dtype is not torch.int64:
        raise TypeError("pairs must be int64")
    return *old, new[0], blocks[0], moves[0]


def pa_pages_update(new_tables: torch.Tensor, new_ref_counts: torch.Tensor, pairs: torch.Tensor,
                    status: torch.Tensor, tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor,
                    keep_lens: torch.Tensor, grow_lens: torch.Tensor, block_size: int,
                    parents: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The next step's block tables: row i keeps the first keep_lens[i] tokens of
    row parents[i] (None: i; negative: nothing) and gets blocks for grow_lens[i];
    pairs [rows, 2] are the copies of shared last blocks, for pa_copy_pages.
    status[0] is 0, and nothing else changed, if the free blocks do not suffice
    (see include/pa.h)."""
    dev = _dense(new_tables, new_ref_counts, pairs, status, tables, ref_counts, lens, keep_lens, grow_lens, parents,
                 workspace, err_word)
    old, m, n, nb, moves = _check_pages(new_tables, new_ref_counts, pairs, status, tables, ref_counts, lens)
    if moves != n:
        raise ValueError(f"pairs has shape {tuple(pairs.shape)}, expected {(n, 2)}")
    rows = (n,)
    _shapes(keep_lens, rows, "keep_lens", grow_lens, rows, "grow_lens", parents, rows, "parents")
    _int32(keep_lens, "keep_lens", grow_lens, "grow_lens", parents, "parents")
    if workspace is None:
        workspace = _own_workspace(stream, pages_workspace_for, tables, ref_counts, n)
    _call(_lib.pa_pages_update, dev, stream, new_tables.data_ptr(), new_ref_counts.data_ptr(), pairs.data_ptr(),
          status.data_ptr(), tables.data_ptr(), ref_counts.data_ptr(), lens.data_ptr(), _addr(parents),
          keep_lens.data_ptr(), grow_lens.data_ptr(), n, old, m, int(block_size), nb, _addr(workspace),
          _ws_bytes(workspace), _addr(err_word))
    return new_tables


def pa_pages_compact(new_tables: torch.Tensor, new_ref_counts: torch.Tensor, remap: torch.Tensor,
                     pairs: torch.Tensor, status: torch.Tensor, tables: torch.Tensor, ref_counts: torch.Tensor,
                     lens: torch.Tensor, block_size: int, workspace: torch.Tensor | None = None,
                     err_word: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Move a pool's used blocks to its front, by at most len(pairs) moves:
    pairs are the copies, for pa_copy_pages, remap every block's place now (see
    include/pa.h)."""
    dev = _dense(new_tables, new_ref_counts, remap, pairs, status, tables, ref_counts, lens, workspace, err_word)
    n, m, new_rows, nb, moves = _check_pages(new_tables, new_ref_counts, pairs, status, tables, ref_counts, lens)
    if new_rows != n:
        raise ValueError(f"new_tables has shape {tuple(new_tables.shape)}, expected {(n, m)}")
    _shapes(remap, (nb,), "remap")
    _int32(remap, "remap")
    if workspace is None:
        workspace = _own_workspace(stream, pages_workspace_for, tables, ref_counts)
    _call(_lib.pa_pages_compact, dev, stream, new_tables.data_ptr(), new_ref_counts.data_ptr(), remap.data_ptr(),
          pairs.data_ptr(), status.data_ptr(), tables.data_ptr(), ref_counts.data_ptr(), lens.data_ptr(),
          n, m, int(block_size), nb, moves, _addr(workspace), _ws_bytes(workspace), _addr(err_word))
    return new_tables


def pa_copy_pages(src_dst_pairs: torch.Tensor, pools, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Copy block src onto block dst, in each of up to 8 pools ([blocks, ...],
    of any types), for every pair with src >= 0."""
    dev = _dense(src_dst_pairs, err_word, *pools)
    n = src_dst_pairs.shape
    if src_dst_pairs.dtype is not torch.int64 or len(n) != 2 or n[1] != 2:
        raise TypeError("src_dst_pairs must be int64 [n, 2]")
    k = len(pools)
    if not k:
        raise ValueError("no pool")
    nb = pools[0].shape[0]
    at, size = [], []
    for t in pools:
        if t.shape[0] != nb:
            raise ValueError("the pools must have the same number of blocks")
        at.append(t.data_ptr())
        size.append(t.nbytes // (nb or 1))
    _call(_lib.pa_copy_pages, dev, stream, src_dst_pairs.data_ptr(), n[0], _array(ctypes.c_void_p, k)(*at),
          _array(ctypes.c_longlong, k)(*size), k, nb, _addr(err_word))


@functools.cache
def _array(kind, n: int):
    return kind * n


def version() -> tuple[int, int, int]:
    v = _lib.pa_version()
    return (v >> 16) & 0xFF, (v >> 8) & 0xFF, v & 0xFF
