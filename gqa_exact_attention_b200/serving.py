"""Serving operators: attention over packed prompts, attention of drafted-token trees over a
cache, and the pages of a paged cache.

Argument marshalling only, as in the package's ``__init__``: the work runs in the CUDA kernels
of ``libgqa_serve.so`` (built in-tree from ``csrc_serve/``), on the current stream, without a
fallback.  The C contract is ``include/gqa_serve.h``; the names here are the same.
"""
from __future__ import annotations

import ctypes
import math
import os

from . import GQA_OUT_BF16, GQA_OUT_F32, _check, _have_nvcc, _nvtx_enabled, _range

__all__ = [
    "gqa_attn_fwd_varlen", "gqa_attn_fwd_tree", "gqa_cache_resize", "gqa_cache_fork",
    "gqa_cache_compact", "gqa_serve_device_status", "serve_lib_path", "load_serve",
    "GQA_CACHE_DONE", "GQA_CACHE_NO_PAGES", "GQA_CACHE_INVALID", "GQA_CACHE_SHARED",
    "GQA_CACHE_MAX_REQUESTS",
]

serve_lib_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgqa_serve.so")

# outcomes of the cache calls' requests (the header's gqa_cache_status)
GQA_CACHE_DONE = 0
GQA_CACHE_NO_PAGES = 1
GQA_CACHE_INVALID = 2
GQA_CACHE_SHARED = 3
GQA_CACHE_MAX_REQUESTS = 4096

_lib = None
torch = None  # imported with the library


def load_serve():
    """Load ``libgqa_serve.so`` (building it in-tree first if it is absent or stale and nvcc
    is available).  Raises if it cannot be loaded."""
    global _lib, torch
    if _lib is not None:
        return _lib
    import torch
    try:
        from . import _build
        if _build.serve_stale() and _have_nvcc():
            _build.build_serve()
    except Exception as e:  # a failed build must not hide behind an old library
        if not os.path.exists(serve_lib_path):
            raise RuntimeError(f"libgqa_serve.so is missing and could not be built: {e}") from e
    if not os.path.exists(serve_lib_path):
        raise RuntimeError(f"libgqa_serve.so not found at {serve_lib_path}; run the package build")
    L = ctypes.CDLL(serve_lib_path)
    i, f, p, ll = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong
    L.gqa_attn_fwd_varlen.argtypes = [p, ll, p, ll, p, ll, p, p, p, i, p, i, i, i, i, i, i, f, i, p]
    L.gqa_attn_fwd_tree.argtypes = [p, p, p, p, i, i, i, p, p, i, p, p, i, p, i, i, i, i, i, i, f, p]
    L.gqa_cache_resize.argtypes = [p, p, p, i, i, i, i, p, p, i, p, p]
    L.gqa_cache_fork.argtypes = [p, p, i, ll, p, p, p, i, i, i, i, p, p, i, p, p]
    L.gqa_cache_compact.argtypes = [p, p, i, ll, p, p, p, i, i, i, i, p, p, p, i, p, p]
    L.gqa_serve_device_status.argtypes = [i]
    for name in ("gqa_attn_fwd_varlen", "gqa_attn_fwd_tree", "gqa_cache_resize", "gqa_cache_fork",
                 "gqa_cache_compact", "gqa_serve_device_status"):
        getattr(L, name).restype = i
    _lib = L
    return L


def gqa_serve_device_status(reset: bool = False) -> int:
    """gqa_attn_device_status of the serving kernels; synchronous."""
    return int(load_serve().gqa_serve_device_status(int(bool(reset))))


# The calls below may take a few microseconds on the GPU, so the checks are kept to a few Python
# operations each: device numbers are compared instead of device objects, and nothing is built
# that a valid call does not need.

def _ints(name, t, shape, index):
    """The address of a contiguous int32 tensor of this shape on CUDA device `index`."""
    if t.dtype is torch.int32 and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {list(shape)} on the same device")


def _rows(name, t, H, d, index):
    """The row stride of a bf16 tensor [n, H, d] on CUDA device `index` whose heads are contiguous
    (0: contiguous rows, or fewer than two)."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.get_device() != index or index < 0 \
            or t.shape[1] != H or t.shape[2] != d:
        raise ValueError(f"{name} must be a bf16 CUDA tensor [rows, {H}, {d}] on one device")
    if t.is_contiguous():
        return 0
    if t.numel() and (t.stride(2) != 1 or (H > 1 and t.stride(1) != d)):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if t.shape[0] <= 1 or t.numel() == 0:
        return 0
    if t.stride(0) < H * d or t.stride(0) % 8:
        raise ValueError(f"{name}'s rows must not overlap, and start a multiple of 8 elements apart")
    return t.stride(0)


def _outputs(out, lse, out_dtype, out_shape, lse_shape, q):
    index = q.get_device()
    if out is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        if dt is not torch.float32 and dt is not torch.bfloat16:
            raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
        out = torch.empty(out_shape, dtype=dt, device=q.device)
    elif out.dtype not in (torch.float32, torch.bfloat16) or not out.is_contiguous() \
            or out.get_device() != index or out.shape != out_shape:
        raise ValueError(f"out must be a contiguous fp32 or bf16 tensor {list(out_shape)} on q's device")
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    elif lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != index \
            or lse.shape != lse_shape:
        raise ValueError(f"lse must be a contiguous fp32 tensor {list(lse_shape)} on q's device")
    return out, lse, GQA_OUT_BF16 if out.dtype is torch.bfloat16 else GQA_OUT_F32


def _call(f, name, index, stream, *args):
    """The library's function, with the stream last, where device `index` is current."""
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index and not _nvtx_enabled():
        status = f(*args, raw)
    else:
        with torch.cuda.device(index), _range(name):
            status = f(*args, raw)
    if status:
        _check(status)


def gqa_attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k=None, out=None, lse=None,
                        out_dtype=None, scale=None, causal=False, stream=None):
    """out, lse = gqa_attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, ...).

    q: bf16 [total_q, Hq, d]; k, v: bf16 [total_k, Hk, d]: sequences one behind the other, rows
    contiguous or a multiple of 8 elements apart (columns of one projection).  cu_seqlens_q,
    cu_seqlens_k: int32 CUDA tensors [B + 1], where each sequence starts and the last ends
    (cu_seqlens_k None: the same as the queries').  Causal masks are bottom-right aligned in
    each sequence.  out is fp32 or bf16 [total_q, Hq, d]; lse fp32 [Hq, total_q]; rows outside
    every sequence are not written.
    """
    L = _lib or load_serve()
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [rows, heads, d]")
    total_q, Hq, d = q.shape
    total_k, Hk = k.shape[0], k.shape[1]
    dev = q.get_device()
    qs, ks, vs = _rows("q", q, Hq, d, dev), _rows("k", k, Hk, d, dev), _rows("v", v, Hk, d, dev)
    if v.shape[0] != total_k:
        raise ValueError("k and v must have the same shape")
    B = cu_seqlens_q.numel() - 1
    if B < 1:
        raise ValueError("cu_seqlens_q must hold at least two bounds")
    cq = _ints("cu_seqlens_q", cu_seqlens_q, (B + 1,), dev)
    if cu_seqlens_k is None:
        if total_k != total_q:
            raise ValueError("without cu_seqlens_k, k has as many rows as q")
        ck = cq
    else:
        ck = _ints("cu_seqlens_k", cu_seqlens_k, (B + 1,), dev)
    out, lse, code = _outputs(out, lse, out_dtype, (total_q, Hq, d), (Hq, total_q), q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _call(L.gqa_attn_fwd_varlen, "gqa_attn_fwd_varlen", dev, stream, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cq, ck,
          out.data_ptr(), code, lse.data_ptr(), B, total_q, total_k, Hq, Hk, d, float(scale), int(bool(causal)))
    return out, lse


def gqa_attn_fwd_tree(q, k_cache, v_cache, tree_mask, cache_seqlens, block_table=None,
                      tree_lens=None, out=None, lse=None, out_dtype=None, scale=None, stream=None):
    """out, lse = gqa_attn_fwd_tree(q, k_cache, v_cache, tree_mask, cache_seqlens, ...).

    q: bf16 [B, T, Hq, d], the drafted nodes' queries; their keys are the last of each
    sequence's.  k_cache, v_cache: bf16 [B, Sk, Hk, d], or with block_table (int32 [B,
    max_pages_per_seq]) page pools [num_pages, page_size, Hk, d].  cache_seqlens: int32 [B],
    the nodes included; tree_lens: int32 [B] nodes of each sequence (None: T).  tree_mask:
    int32 [B, T, ceil(T/32)], or [T, ceil(T/32)] for every sequence: bit j % 32 of word j // 32
    of row i is set where node i sees node j.  out is fp32 or bf16 [B, T, Hq, d]; lse fp32 [B,
    Hq, T]; rows past tree_lens get 0 and -inf.
    """
    L = _lib or load_serve()
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d], the cache [B, Sk, Hk, d] or [num_pages, page_size, Hk, d]")
    B, T, Hq, d = q.shape
    Hk = k_cache.shape[2]
    dev = q.get_device()
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not torch.bfloat16 or not t.is_contiguous() or t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor on q's device")
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != d:
        raise ValueError("k_cache and v_cache must have one shape, with q's d")
    words = (T + 31) // 32
    shared = tree_mask.dim() == 2
    mk = _ints("tree_mask", tree_mask, (T, words) if shared else (B, T, words), dev)
    ls = _ints("cache_seqlens", cache_seqlens, (B,), dev)
    tl = None if tree_lens is None else _ints("tree_lens", tree_lens, (B,), dev)
    if block_table is None:
        if k_cache.shape[0] != B:
            raise ValueError("without a block_table the cache is [B, Sk, Hk, d]")
        tb, M, P, page, Sk = None, 0, 0, 0, k_cache.shape[1]
    else:
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages_per_seq]")
        M, P, page, Sk = block_table.shape[1], k_cache.shape[0], k_cache.shape[1], 0
        tb = _ints("block_table", block_table, (B, M), dev)
    out, lse, code = _outputs(out, lse, out_dtype, (B, T, Hq, d), (B, Hq, T), q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _call(L.gqa_attn_fwd_tree, "gqa_attn_fwd_tree", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), tb, M, P,
          page, ls, mk, int(shared), tl, out.data_ptr(), code, lse.data_ptr(), B, T, Sk, Hq, Hk, d, float(scale))
    return out, lse


def _state(block_table, cache_seqlens, page_refs):
    """Device number, table, lengths and counts pointers, S, M and P of a cache's pages."""
    dev = block_table.get_device()
    if dev < 0 or block_table.dim() != 2 or page_refs.dim() != 1:
        raise ValueError("block_table must be a CUDA tensor [S, max_pages_per_seq], page_refs [num_pages]")
    S, M = shape = block_table.shape
    P, = pages = page_refs.shape
    return (dev, _ints("block_table", block_table, shape, dev), _ints("cache_seqlens", cache_seqlens, (S,), dev),
            _ints("page_refs", page_refs, pages, dev), S, M, P)


def _pools(k_pages, v_pages, P, index):
    """(K pointer, V pointer, layers, bytes of a row, page size) of a cache's pools."""
    shape = k_pages.shape
    if shape != v_pages.shape or k_pages.dtype is not v_pages.dtype or len(shape) not in (4, 5):
        raise ValueError("k_pages and v_pages must have one shape and type, [num_pages, page_size, Hk, d] or [layers, ...]")
    if k_pages.get_device() != index or v_pages.get_device() != index or not k_pages.is_contiguous() \
            or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages must be contiguous, on block_table's device")
    if shape[-4] != P:
        raise ValueError("page_refs must count as many pages as the pools have")
    k, v = k_pages.data_ptr(), v_pages.data_ptr()
    if k == v:
        raise ValueError("k_pages and v_pages must be different tensors")
    return k, v, shape[0] if len(shape) == 5 else 1, shape[-1] * shape[-2] * k_pages.element_size(), shape[-3]


def gqa_cache_resize(block_table, cache_seqlens, page_refs, page_size, new_lens, slots=None,
                     status=None, stream=None):
    """status = gqa_cache_resize(block_table, cache_seqlens, page_refs, page_size, new_lens, slots).

    Gives slot slots[i] (None: slot i) the pages for new_lens[i] keys: more, fewer, or none for
    0.  block_table int32 [S, max_pages_per_seq], cache_seqlens [S] and page_refs [num_pages]
    are updated in place; status int32 [n] holds each request's outcome (GQA_CACHE_*).
    """
    L = _lib or load_serve()
    dev, tb, ln, rf, S, M, P = _state(block_table, cache_seqlens, page_refs)
    n, = shape = new_lens.shape
    if slots is None and n > S:
        raise ValueError("without slots there are at most as many lengths as slots")
    nl = _ints("new_lens", new_lens, shape, dev)
    sl = None if slots is None else _ints("slots", slots, shape, dev)
    if status is None:
        status = torch.empty_like(new_lens)
    _call(L.gqa_cache_resize, "gqa_cache_resize", dev, stream, tb, ln, rf, S, M, P, int(page_size), sl, nl, n,
          _ints("status", status, shape, dev))
    return status


def gqa_cache_fork(k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children,
                   status=None, stream=None):
    """status = gqa_cache_fork(k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children).

    Makes slot children[i] a copy of slot parents[i]: whole pages are shared, the last partly
    filled one is copied in every layer.  k_pages, v_pages: [num_pages, page_size, Hk, d] or
    [layers, num_pages, page_size, Hk, d], of any type.  status int32 [n] as gqa_cache_resize.
    """
    L = _lib or load_serve()
    dev, tb, ln, rf, S, M, P = _state(block_table, cache_seqlens, page_refs)
    k, v, layers, row, page = _pools(k_pages, v_pages, P, dev)
    n, = shape = parents.shape
    pa, ch = _ints("parents", parents, shape, dev), _ints("children", children, shape, dev)
    if status is None:
        status = torch.empty_like(parents)
    _call(L.gqa_cache_fork, "gqa_cache_fork", dev, stream, k, v, layers, row, tb, ln, rf, S, M, P, page, pa, ch, n,
          _ints("status", status, shape, dev))
    return status


def gqa_cache_compact(k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens,
                      tree_lens=None, status=None, stream=None):
    """status = gqa_cache_compact(k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens, tree_lens).

    Of the tree_lens[s] (None: T) drafted nodes at the end of each slot, those in keep[s,
    :keep_lens[s]] (int32 [S, T], increasing) stay, moved together behind the context in every
    layer; the sequence ends behind them and its unused pages are given up.  status int32 [S].
    """
    L = _lib or load_serve()
    dev, tb, ln, rf, S, M, P = _state(block_table, cache_seqlens, page_refs)
    k, v, layers, row, page = _pools(k_pages, v_pages, P, dev)
    if keep.dim() != 2:
        raise ValueError("keep must be [S, T]")
    T = keep.shape[1]
    kp, kl = _ints("keep", keep, (S, T), dev), _ints("keep_lens", keep_lens, (S,), dev)
    tl = None if tree_lens is None else _ints("tree_lens", tree_lens, (S,), dev)
    if status is None:
        status = torch.empty_like(keep_lens)
    _call(L.gqa_cache_compact, "gqa_cache_compact", dev, stream, k, v, layers, row, tb, ln, rf, S, M, P, page, kp, kl,
          tl, T, _ints("status", status, (S,), dev))
    return status
