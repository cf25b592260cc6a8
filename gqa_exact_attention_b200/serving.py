"""Serving operators: attention over packed prompts, attention of drafted-token trees over a
cache, and the pages of a paged cache.

The work runs in the CUDA kernels of ``libgqa_serve.so`` (built in-tree from ``csrc_serve/``), on
the current stream, without a fallback.  The C contract is ``include/gqa_serve.h``; the names here
are the same.  Tensors are checked, outputs allocated and the library called by a small module
(``bind/serve_bind.cpp``): a call may take a few microseconds on the GPU, less than the same
checks do as Python operations (resizing 8 slots: 11 us a call with ctypes, 6 us so).
"""
from __future__ import annotations

import ctypes
import os
from shutil import which

from . import _check, _have_nvcc, _range, _rebuild

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
_bind = None


def load_serve():
    """Load ``libgqa_serve.so`` (building it in-tree first if it is absent or stale and nvcc
    is available).  Raises if it cannot be loaded."""
    global _lib
    if _lib is not None:
        return _lib
    from . import _build
    _rebuild("libgqa_serve.so", serve_lib_path, _build.serve_stale, _build.build_serve, _have_nvcc())
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


def _load_bind():
    global _bind
    load_serve()
    import torch  # noqa: F401  (the module's own libraries)

    from . import _build
    _rebuild("_serve_bind.so", _build.SERVE_BIND, _build.bind_stale, _build.build_bind, which("g++") is not None)
    from . import _serve_bind
    _serve_bind.on_error(_check)
    _bind = _serve_bind
    return _bind


def _call(name, *args):
    """The binding's function of this name, inside an NVTX range when GQA_NVTX is set."""
    b = _bind or _load_bind()
    f = getattr(b, name)
    if b.nvtx():
        with _range(("gqa_attn_fwd_" if name in ("varlen", "tree") else "gqa_cache_") + name):
            return f(*args)
    return f(*args)


def _bf16(out_dtype):
    if out_dtype is None:
        return False
    import torch
    if out_dtype is torch.bfloat16 or out_dtype is torch.float32:
        return out_dtype is torch.bfloat16
    raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")


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
    return _call("varlen", q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, _bf16(out_dtype), scale, causal, stream)


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
    return _call("tree", q, k_cache, v_cache, tree_mask, cache_seqlens, block_table, tree_lens, out, lse,
                 _bf16(out_dtype), scale, stream)


def gqa_cache_resize(block_table, cache_seqlens, page_refs, page_size, new_lens, slots=None,
                     status=None, stream=None):
    """status = gqa_cache_resize(block_table, cache_seqlens, page_refs, page_size, new_lens, slots).

    Gives slot slots[i] (None: slot i) the pages for new_lens[i] keys: more, fewer, or none for
    0.  block_table int32 [S, max_pages_per_seq], cache_seqlens [S] and page_refs [num_pages]
    are updated in place; status int32 [n] holds each request's outcome (GQA_CACHE_*).
    """
    return _call("resize", block_table, cache_seqlens, page_refs, page_size, new_lens, slots, status, stream)


def gqa_cache_fork(k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children,
                   status=None, stream=None):
    """status = gqa_cache_fork(k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children).

    Makes slot children[i] a copy of slot parents[i]: whole pages are shared, the last partly
    filled one is copied in every layer.  k_pages, v_pages: [num_pages, page_size, Hk, d] or
    [layers, num_pages, page_size, Hk, d], of any type.  status int32 [n] as gqa_cache_resize.
    """
    return _call("fork", k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children, status, stream)


def gqa_cache_compact(k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens,
                      tree_lens=None, status=None, stream=None):
    """status = gqa_cache_compact(k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens, tree_lens).

    Of the tree_lens[s] (None: T) drafted nodes at the end of each slot, those in keep[s,
    :keep_lens[s]] (int32 [S, T], increasing) stay, moved together behind the context in every
    layer; the sequence ends behind them and its unused pages are given up.  status int32 [S].
    """
    return _call("compact", k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens, tree_lens,
                 status, stream)
