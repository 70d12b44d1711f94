"""ctypes binding of libpagedmoe.so (include/pagedmoe.h): argument marshalling only.

Every function keeps the C name. Tensors are passed as raw device pointers
(``tensor.data_ptr()``) with the current torch CUDA stream; every step of the
layer runs in the library's own CUDA kernels. If the library is missing, loading
fails with an error (there is no fallback path).
"""

import ctypes
import os
from typing import NamedTuple

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpagedmoe.so")

PMOE_OK, PMOE_EINVAL, PMOE_ENOMEM, PMOE_EHOSTALLOC, PMOE_ECUDA, PMOE_EUNSUPPORTED, PMOE_ETIMEOUT, PMOE_EDEVICE = \
    0, -1, -2, -3, -4, -5, -6, -7
PMOE_BF16, PMOE_FP8_BLOCK128, PMOE_INT4_GPTQ_G128, PMOE_MXFP4, PMOE_NVFP4 = 0, 1, 2, 3, 4
PMOE_PAGEIN_COPY_ENGINE, PMOE_PAGEIN_SM_PULL = 0, 1
PMOE_KV_BF16, PMOE_KV_E4M3 = 0, 1
PMOE_SCORE_SOFTMAX, PMOE_SCORE_SIGMOID = 0, 1


class PmoeError(RuntimeError):
    def __init__(self, status, what):
        lib = _LIB
        text = lib.pmoe_status_string(status).decode() if lib else str(status)
        detail = lib.pmoe_last_error().decode() if lib else ""
        super().__init__(f"{what}: {text} ({status}) {detail}".strip())
        self.status = status


class pmoe_cache_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_experts", "top_k", "hidden", "intermediate", "num_slots", "num_layers", "format",
        "max_tokens", "pagein_mode", "device")]


class pmoe_kv_desc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)] + \
        [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "kv_heads", "head_dim", "dtype")]


class pmoe_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("steps", "hits", "misses", "waves", "bytes_paged")]


class pmoe_kernel_times(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 12), ("launches", ctypes.c_uint64 * 12), ("copies", ctypes.c_uint64)]


KERNEL_CLASSES = ("residency", "group", "gather", "gateup", "down", "combine", "pull", "pagein_copy", "decode")

_LIB = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SIGS = {
    "pmoe_version": ([], _I),
    "pmoe_status_string": ([_I], ctypes.c_char_p),
    "pmoe_last_error": ([], ctypes.c_char_p),
    "pmoe_expert_bytes": ([_I, _I, _I], ctypes.c_size_t),
    "moe_router_topk": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_router_gemm_topk": ([_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_group_by_expert": ([_P, _I, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P], _I),
    "moe_group_scratch_ints": ([_I, _I], ctypes.c_size_t),
    "expert_cache_create": ([ctypes.POINTER(pmoe_cache_desc), ctypes.POINTER(_P)], _I),
    "expert_cache_destroy": ([_P], None),
    "expert_cache_host_store": ([_P, _I, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_size_t)], _I),
    "expert_cache_load_expert": ([_P, _I, _I, _P, ctypes.c_size_t], _I),
    "expert_cache_reset": ([_P, _I], _I),
    "expert_cache_ensure_resident": ([_P, _I, _P, _I, _P, ctypes.POINTER(_I)], _I),
    "expert_cache_prefetch": ([_P, _I, _P, _I, _P], _I),
    "moe_paged_forward": ([_P, _I, _P, _I, _P, _P, _P, _P, _P], _I),
    "expert_cache_stats": ([_P, _I, ctypes.POINTER(pmoe_stats)], _I),
    "expert_cache_slot_table": ([_P, _I, _P, _P], _I),
    "expert_cache_read_slot": ([_P, _I, _I, _P, ctypes.c_size_t], _I),
    "expert_cache_set_timing": ([_P, _I], _I),
    "expert_cache_kernel_times": ([_P, ctypes.POINTER(pmoe_kernel_times)], _I),
    "moe_decode_forward_noalloc": ([_P, ctypes.c_size_t, _I, _P, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P,
                                    _P], _I),
    "moe_kv_append": ([ctypes.POINTER(pmoe_kv_desc), _P, _L, _P, _L, _P, _L, _I, _I, _P, _I, _P, _P, _I, _I, _P, _P,
                       ctypes.c_float, _P, _P, _P, _P], _I),
    "moe_prefix_attention": ([ctypes.POINTER(pmoe_kv_desc), _P, _L, _I, _I, ctypes.c_float, _P, _I, _P, _I, _I, _P, _P,
                              _I, _P, _P, _P, ctypes.c_size_t, _P, _P], _I),
    "moe_prefix_attention_scratch_bytes": ([ctypes.POINTER(pmoe_kv_desc), _I, _I, _I, _I], ctypes.c_size_t),
    "moe_sample_tokens": ([_P, _I, _I, _I, _L, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "moe_batch_tables": ([_P, _I, _I, _I, _P, _I, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "moe_chunk_attention": ([ctypes.POINTER(pmoe_kv_desc), _P, _L, _I, _I, ctypes.c_float, _P, _P, _I, _P, _I, _I, _I, _P,
                             _P, _P, ctypes.c_size_t, _P, _P], _I),
    "moe_chunk_attention_scratch_bytes": ([ctypes.POINTER(pmoe_kv_desc), _I, _I, _I], ctypes.c_size_t),
    "moe_router_select": ([_P, _I, _I, _I, _L, _I, _I, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P], _I),
    "moe_adjust_logits": ([_P, _I, _I, _I, _L, _P, _L, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _L, _P, _I, _L, _P, _P], _I),
    "moe_paged_stack_forward": ([_P, _P, _I, _P, _P, _P, _P, _P], _I),
}
EXPORTED = tuple(_SIGS)


def load(path=LIB_PATH):
    """Load the library (building it first if sources are newer)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    from . import build as _build
    if _build.needs_build():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"libpagedmoe.so not found at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = lib
    return lib


def _check(status, what):
    if status != PMOE_OK:
        raise PmoeError(status, what)


def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def pmoe_expert_bytes(fmt, H, I):
    return int(load().pmoe_expert_bytes(fmt, H, I))


def moe_router_topk(logits, top_k, renormalize=True, ids_out=None, w_out=None, stream=None):
    """logits: CUDA fp32 [T, E] -> (ids int32 [T, top_k], w fp32 [T, top_k])."""
    import torch
    lib = load()
    T, E = logits.shape
    assert logits.dtype == torch.float32 and logits.is_cuda and logits.is_contiguous()
    if ids_out is None:
        ids_out = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    if w_out is None:
        w_out = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _check(lib.moe_router_topk(_ptr(logits), T, E, top_k, 1 if renormalize else 0, _ptr(ids_out), _ptr(w_out),
                               _stream_handle(stream)), "moe_router_topk")
    return ids_out, w_out


def moe_group_by_expert(ids, E, err_out=None, stream=None):
    """ids: CUDA int32 (any shape, flattened to P pairs) -> (counts [E], offs [E + 1],
    perm [P], pos [P]) int32; perm entries from offs[E] on (ids outside [0, E)) are
    undefined. err_out (CUDA int32 [1]) gets 1 ORed in for such an id."""
    import torch
    lib = load()
    assert ids.dtype == torch.int32 and ids.is_cuda and ids.is_contiguous()
    P = ids.numel()
    dev = ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offs = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(P, 1), dtype=torch.int32, device=dev)[:P]
    pos = torch.empty(max(P, 1), dtype=torch.int32, device=dev)[:P]
    n_scratch = int(lib.moe_group_scratch_ints(P, E))
    scratch = torch.empty(n_scratch, dtype=torch.int32, device=dev) if n_scratch > 0 else None
    _check(lib.moe_group_by_expert(_ptr(ids), P, E, _ptr(counts), _ptr(offs), _ptr(perm), _ptr(pos), _ptr(scratch),
                                   n_scratch, _ptr(err_out), _stream_handle(stream)), "moe_group_by_expert")
    return counts, offs, perm, pos


def moe_router_gemm_topk(x, router_weight, top_k, renormalize=True, ids_out=None, w_out=None, logits_out=None,
                         stream=None):
    """x: CUDA bf16 [T, H], router_weight: CUDA bf16 [E, H] -> (ids int32 [T, top_k],
    w fp32 [T, top_k]); logits_out (fp32 [T, E]) is filled when given."""
    import torch
    lib = load()
    T, H = x.shape
    E = router_weight.shape[0]
    assert x.dtype == torch.bfloat16 and router_weight.dtype == torch.bfloat16 and router_weight.shape[1] == H
    assert x.is_cuda and x.is_contiguous() and router_weight.is_contiguous()
    if ids_out is None:
        ids_out = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
    if w_out is None:
        w_out = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
    _check(lib.moe_router_gemm_topk(_ptr(x), _ptr(router_weight), T, H, E, top_k, 1 if renormalize else 0,
                                    _ptr(logits_out), _ptr(ids_out), _ptr(w_out), _stream_handle(stream)),
           "moe_router_gemm_topk")
    return ids_out, w_out


def moe_decode_forward_noalloc(experts, stride, E, top_k, H, I, fmt, x, ids, w, y=None, slot_of=None,
                               residual=None, err_out=None, n_slots=None, stream=None):
    """Decode MoE over experts already in device memory; allocates no device memory
    (the library uses a fixed static scratch). experts: CUDA uint8 tensor holding the
    expert slots `stride` bytes apart (n_slots defaults to all of them); x: bf16 [T, H];
    ids int32 / w fp32 [T, top_k]; slot_of: int32 [E] or None; err_out: int32 [1] that
    receives the call's device error bits, or None. Returns y."""
    import torch
    T = x.shape[0]
    assert experts.is_cuda and experts.dtype == torch.uint8 and experts.is_contiguous()
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape == (T, H)
    assert ids.is_cuda and ids.dtype == torch.int32 and ids.is_contiguous() and tuple(ids.shape) == (T, top_k)
    assert w.is_cuda and w.dtype == torch.float32 and w.is_contiguous() and tuple(w.shape) == (T, top_k)
    if slot_of is not None:
        assert slot_of.is_cuda and slot_of.dtype == torch.int32 and slot_of.is_contiguous() and slot_of.numel() == E
    if residual is not None:
        assert residual.is_cuda and residual.dtype == torch.bfloat16 and residual.is_contiguous()
        assert residual.shape == x.shape
    if err_out is not None:
        assert err_out.is_cuda and err_out.dtype == torch.int32 and err_out.numel() >= 1
    if n_slots is None:
        n_slots = experts.numel() // stride
    if y is None:
        y = torch.empty_like(x)
    assert y.is_cuda and y.dtype == torch.bfloat16 and y.is_contiguous() and y.shape == x.shape
    _check(load().moe_decode_forward_noalloc(_ptr(experts), stride, n_slots, _ptr(slot_of), E, top_k, H, I, fmt,
                                             _ptr(x), T, _ptr(ids), _ptr(w), _ptr(residual), _ptr(y), _ptr(err_out),
                                             _stream_handle(stream)), "moe_decode_forward_noalloc")
    return y


# The calls of a serving step (below) go through _binding, which checks their tensors and calls
# the library in C++: their kernels take a few microseconds, less than the checks in Python.

_BINDING = None


def _binding():
    global _BINDING
    if _BINDING is None:
        import torch  # noqa: F401  (the binding links to its libraries)
        lib = load()
        from . import _binding as b
        b.setup(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
            "moe_kv_append", "moe_prefix_attention", "pmoe_attention_plan", "moe_sample_tokens", "moe_batch_tables",
            "moe_chunk_attention", "moe_chunk_attention_scratch_bytes", "moe_router_select", "moe_adjust_logits")))
        _BINDING = b
    return _BINDING


def _empty(shape, dtype, like, stream):
    """A new tensor on the device of `like`, owned by `stream` (None: the current one)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def moe_kv_append(k_cache, v_cache, q, k, v, positions, slots, inv_freq, pair_axis=None, interleaved=False, q_norm=None,
                  k_norm=None, eps=1e-6, k_scale=None, v_scale=None, q_out=None, err_out=None, stream=None):
    """Head norm, rotation and append of T tokens' keys and values to a paged cache.
    k_cache, v_cache: bf16 or float8_e4m3fn [num_pages, kv_heads, page_size, head_dim], of one
    page stride; q: bf16 [T, q_heads, head_dim], k, v: bf16 [T, kv_heads, head_dim] (views of
    one projection will do); positions: int32 [axes, T] or [T]; slots: int32 [T], page *
    page_size + row, -1 = not stored; inv_freq: fp32 [rotary_dim / 2] or None; pair_axis:
    int32 [rotary_dim / 2]; q_norm, k_norm: bf16 [head_dim]. Returns the rotated q (q_out)."""
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q, stream)
    status = (_BINDING or _binding()).kv_append(
        k_cache, v_cache, q, k, v, positions, slots, inv_freq, pair_axis, interleaved, q_norm, k_norm, eps, k_scale,
        v_scale, q_out, err_out, stream)
    if status:
        raise PmoeError(status, "moe_kv_append")
    return q_out


def _desc(k_cache, v_cache):
    """A cache's descriptor, for the sizes of scratch."""
    import torch
    pages, heads, page, dim = k_cache.shape
    kind = PMOE_KV_E4M3 if k_cache.dtype == torch.float8_e4m3fn else PMOE_KV_BF16
    # the scales' values do not matter for the size, but that there are some does
    stride = k_cache.stride(0) if pages > 1 else heads * page * dim  # a single page has no stride
    return pmoe_kv_desc(k_cache.data_ptr(), v_cache.data_ptr(), stride, k_cache.data_ptr(), k_cache.data_ptr(),
                        pages, page, heads, dim, kind)


def moe_prefix_attention_scratch_bytes(k_cache, v_cache, T, q_heads, prefix_len, max_suffix):
    """Bytes of scratch that are enough for a moe_prefix_attention call of these sizes, and for
    every one with fewer rows, a shorter prefix or a smaller max_suffix."""
    import torch
    with torch.cuda.device(k_cache.device):
        return int(load().moe_prefix_attention_scratch_bytes(_desc(k_cache, v_cache), T, q_heads, prefix_len, max_suffix))


def moe_prefix_attention(k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, scale=None,
                         row_seq=None, k_scale=None, v_scale=None, out=None, lse_out=None, scratch=None, err_out=None,
                         stream=None):
    """Attention of q (bf16 [T, q_heads, head_dim]) over a paged cache (as moe_kv_append's).
    Row t sees the first prefix_len keys of prefix_pages (int32), which all rows share, then
    the first suffix_len[t] (int32 [T], at most max_suffix) of page_table[row_seq[t]] (int32
    [sequences, pages]; row_seq int32 [T], default t). scale defaults to head_dim ** -0.5.
    lse_out: fp32 [T, q_heads] or None; scratch: uint8, of the size that
    moe_prefix_attention_scratch_bytes gives for the largest of the calls it serves, taken from torch's allocator for the
    call when not given. Returns out (bf16 [T, q_heads, head_dim])."""
    if out is None:
        out = _empty(q.shape, q.dtype, q, stream)
    status = (_BINDING or _binding()).prefix_attention(
        k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix,
        scale, row_seq, k_scale, v_scale, out, lse_out, scratch, err_out, stream)
    if status:
        raise PmoeError(status, "moe_prefix_attention")
    return out


def moe_sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ids_out=None, logprob_out=None,
                      stream=None):
    """Draw one token id per row of logits (CUDA fp32 or bf16 [T, V], rows contiguous) from
    u (fp32 [T], in [0, 1)). temperature, top_p, min_p: fp32 [T], top_k: int32 [T], or None
    (1, 1, 0 and 0: no cut); temperature 0 takes the largest logit. logprob_out: fp32 [T],
    the drawn token's log probability among the kept ones. Returns ids (int32 [T])."""
    if ids_out is None:
        import torch
        ids_out = _empty(logits.shape[0], torch.int32, logits, stream)
    status = (_BINDING or _binding()).sample_tokens(logits, u, temperature, top_k, top_p, min_p, ids_out, logprob_out, stream)
    if status:
        raise PmoeError(status, "moe_sample_tokens")
    return ids_out


class BatchTables(NamedTuple):
    """What moe_batch_tables gives: int32 tensors."""
    lens: object        # [R] keys of each request after the step
    free_count: object  # [1] free pages after it
    q_start: object     # [R + 1] first row of each request
    positions: object   # [T]
    slots: object       # [T], -1: not stored
    row_seq: object     # [T] request of each row, -1: none
    row_len: object     # [T] keys up to each row's token, 0: not stored


def moe_batch_tables(page_table, free_pages, free_count, lens, new_len, T, page_size, num_pages, lens_out=None,
                     free_count_out=None, q_start=None, positions=None, slots=None, row_seq=None, row_len=None, err_out=None,
                     stream=None):
    """Pages, slots, positions and row ranges of a step of T rows, from the requests' lengths.
    page_table: int32 [R, pages], new pages are written to it; free_pages: int32 [n], a stack of
    which the lowest free_count (int32 [1]) are free; lens, new_len: int32 [R], keys in the cache and
    new tokens (0: rests, -1: ended, its pages are given back). lens_out may be lens, free_count_out
    may be free_count. Returns BatchTables."""
    def out(x, n):
        import torch
        return _empty(n, torch.int32, page_table, stream) if x is None else x

    R = page_table.shape[0]
    r = BatchTables(out(lens_out, R), out(free_count_out, 1), out(q_start, R + 1), out(positions, T), out(slots, T),
                    out(row_seq, T), out(row_len, T))
    status = (_BINDING or _binding()).batch_tables(
        page_table, free_pages, free_count, lens, new_len, T, page_size, num_pages, r.lens, r.free_count, r.q_start,
        r.positions, r.slots, r.row_seq, r.row_len, err_out, stream)
    if status:
        raise PmoeError(status, "moe_batch_tables")
    return r


def moe_chunk_attention_scratch_bytes(k_cache, v_cache, T, q_heads, requests):
    """Bytes of scratch that are enough for a moe_chunk_attention call of these sizes, and for every
    one with fewer rows or requests."""
    import torch
    with torch.cuda.device(k_cache.device):
        return int(load().moe_chunk_attention_scratch_bytes(_desc(k_cache, v_cache), T, q_heads, requests))


def moe_chunk_attention(k_cache, v_cache, q, q_start, kv_len, page_table, window=0, sinks=0, scale=None, k_scale=None,
                        v_scale=None, out=None, lse_out=None, scratch=None, err_out=None, stream=None):
    """Attention of each request's new tokens over its own pages of a paged cache (as
    moe_kv_append's). q: bf16 [T, q_heads, head_dim]; rows q_start[r] .. q_start[r + 1] - 1 (int32
    [R + 1]) are the last of request r's kv_len[r] keys (int32 [R]), in the pages page_table[r] (int32
    [R, pages]). A row sees the keys up to its own; with a window only the last `window` of these, and
    the first `sinks`. scale defaults to head_dim ** -0.5. lse_out: fp32 [T, q_heads] or None;
    scratch: uint8, of the size that moe_chunk_attention_scratch_bytes gives, taken from torch's
    allocator for the call when not given. Returns out (bf16 [T, q_heads, head_dim]); rows of no
    request are left as they were there."""
    if out is None:
        out = _empty(q.shape, q.dtype, q, stream)
    status = (_BINDING or _binding()).chunk_attention(
        k_cache, v_cache, q, q_start, kv_len, page_table, window, sinks, scale, k_scale, v_scale, out, lse_out, scratch,
        err_out, stream)
    if status:
        raise PmoeError(status, "moe_chunk_attention")
    return out


def moe_router_select(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True,
                      scale=1.0, ids_out=None, w_out=None, stream=None):
    """Experts by scores: logits (CUDA fp32 or bf16 [T, E], rows contiguous) -> (ids int32 [T, top_k],
    w fp32 [T, top_k]). scoring: "softmax" or "sigmoid"; bias (fp32 [E]) is added for the choice
    alone; of `groups` groups of neighbouring experts the top_groups with the largest sums of their
    group_top (1 or 2) best are kept; w is renormalised and multiplied by scale."""
    import torch
    if scoring not in ("softmax", "sigmoid"):
        raise AssertionError(f"scoring: {scoring!r}")
    T = logits.shape[0]
    if ids_out is None:
        ids_out = _empty((T, max(top_k, 0)), torch.int32, logits, stream)
    if w_out is None:
        w_out = _empty((T, max(top_k, 0)), torch.float32, logits, stream)
    status = (_BINDING or _binding()).router_select(
        logits, bias, top_k, PMOE_SCORE_SIGMOID if scoring == "sigmoid" else PMOE_SCORE_SOFTMAX, groups, top_groups,
        group_top, renormalize, scale, ids_out, w_out, stream)
    if status:
        raise PmoeError(status, "moe_router_select")
    return ids_out, w_out


def moe_adjust_logits(logits, history=None, prompt_len=None, history_len=None, repetition=None, frequency=None,
                      presence=None, bias_ids=None, bias=None, mask=None, out=None, err_out=None, stream=None):
    """Penalties, biases and masks on logits (CUDA fp32 or bf16 [T, V], rows contiguous). history: int32
    [T, n], of which the first history_len[t] ids count (int32 [T]), the first prompt_len[t] of these
    as the prompt; repetition (of prompt and output), frequency and presence (of the output): fp32
    [T]; bias_ids: int32 [T, B], -1 = none, with bias fp32 [T, B]; mask: int32 [T, words], bit v % 32 of
    word v // 32 set where v is allowed. out: fp32 or bf16 [T, V], default fp32; logits itself for a
    change in place. Returns out."""
    if out is None:
        import torch
        out = _empty(logits.shape, torch.float32, logits, stream)
    status = (_BINDING or _binding()).adjust_logits(
        logits, history, prompt_len, history_len, repetition, frequency, presence, bias_ids, bias, mask, out, err_out, stream)
    if status:
        raise PmoeError(status, "moe_adjust_logits")
    return out


class ExpertCache:
    """Owns one pmoe_cache (expert_cache_create ... expert_cache_destroy)."""

    def __init__(self, num_experts, top_k, hidden, intermediate, num_slots, num_layers=1, fmt=PMOE_BF16,
                 max_tokens=8, pagein_mode=PMOE_PAGEIN_COPY_ENGINE, device=0):
        lib = load()
        self.desc = pmoe_cache_desc(num_experts, top_k, hidden, intermediate, num_slots, num_layers, fmt,
                                    max_tokens, pagein_mode, device)
        h = ctypes.c_void_p()
        _check(lib.expert_cache_create(ctypes.byref(self.desc), ctypes.byref(h)), "expert_cache_create")
        self.handle = h
        self.E, self.top_k, self.H, self.I, self.K = num_experts, top_k, hidden, intermediate, num_slots
        self.layers, self.fmt, self.max_tokens = num_layers, fmt, max_tokens
        self.expert_bytes = pmoe_expert_bytes(fmt, hidden, intermediate)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            load().expert_cache_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- host store
    def host_store(self, layer):
        """numpy uint8 view [E, stride] of the layer's pinned store."""
        p = ctypes.c_void_p()
        stride = ctypes.c_size_t()
        _check(load().expert_cache_host_store(self.handle, layer, ctypes.byref(p), ctypes.byref(stride)),
               "expert_cache_host_store")
        buf = (ctypes.c_uint8 * (self.E * stride.value)).from_address(p.value)
        return np.frombuffer(buf, dtype=np.uint8).reshape(self.E, stride.value)

    def load_layer(self, layer, experts):
        """experts: uint8 [E, expert_bytes] -> copied into the store."""
        view = self.host_store(layer)
        view[:, :self.expert_bytes] = experts

    def expert_cache_load_expert(self, layer, expert, data):
        data = np.ascontiguousarray(data, dtype=np.uint8)
        _check(load().expert_cache_load_expert(self.handle, layer, expert, data.ctypes.data_as(ctypes.c_void_p),
                                               data.size), "expert_cache_load_expert")

    def expert_cache_reset(self, layer=-1):
        _check(load().expert_cache_reset(self.handle, layer), "expert_cache_reset")

    def expert_cache_ensure_resident(self, layer, ids, stream=None):
        waves = ctypes.c_int(0)
        _check(load().expert_cache_ensure_resident(self.handle, layer, _ptr(ids), ids.numel(),
                                                   _stream_handle(stream), ctypes.byref(waves)),
               "expert_cache_ensure_resident")
        return waves.value

    def expert_cache_prefetch(self, layer, ids, stream=None):
        _check(load().expert_cache_prefetch(self.handle, layer, _ptr(ids), ids.numel(), _stream_handle(stream)),
               "expert_cache_prefetch")

    def moe_paged_forward(self, layer, x, ids, w, y=None, residual=None, stream=None):
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        assert x.dtype == torch.bfloat16 and ids.dtype == torch.int32 and w.dtype == torch.float32
        _check(load().moe_paged_forward(self.handle, layer, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(residual), _ptr(y),
                                        _stream_handle(stream)), "moe_paged_forward")
        return y

    def moe_paged_stack_forward(self, x, ids_all, w_all, y=None, work=None, stream=None):
        """All layers: h_{l+1} = h_l + moe_l(h_l). ids_all/w_all: [L, T, top_k] device."""
        import torch
        if y is None:
            y = torch.empty_like(x)
        if work is None and self.layers > 1:
            work = torch.empty_like(x)
        _check(load().moe_paged_stack_forward(self.handle, _ptr(x), x.shape[0], _ptr(ids_all), _ptr(w_all), _ptr(y),
                                              _ptr(work), _stream_handle(stream)), "moe_paged_stack_forward")
        return y

    def expert_cache_stats(self, layer=-1):
        s = pmoe_stats()
        _check(load().expert_cache_stats(self.handle, layer, ctypes.byref(s)), "expert_cache_stats")
        return {n: int(getattr(s, n)) for n, _ in pmoe_stats._fields_}

    def expert_cache_slot_table(self, layer):
        exp = np.empty(self.K, np.int32)
        lu = np.empty(self.K, np.int32)
        _check(load().expert_cache_slot_table(self.handle, layer, exp.ctypes.data_as(ctypes.c_void_p),
                                              lu.ctypes.data_as(ctypes.c_void_p)), "expert_cache_slot_table")
        return exp, lu

    def expert_cache_read_slot(self, layer, slot):
        out = np.empty(self.expert_bytes, np.uint8)
        _check(load().expert_cache_read_slot(self.handle, layer, slot, out.ctypes.data_as(ctypes.c_void_p),
                                             out.size), "expert_cache_read_slot")
        return out

    def expert_cache_set_timing(self, enable=True):
        _check(load().expert_cache_set_timing(self.handle, 1 if enable else 0), "expert_cache_set_timing")

    def expert_cache_kernel_times(self):
        kt = pmoe_kernel_times()
        _check(load().expert_cache_kernel_times(self.handle, ctypes.byref(kt)), "expert_cache_kernel_times")
        return {name: {"ms": kt.ms[i], "launches": int(kt.launches[i])} for i, name in enumerate(KERNEL_CLASSES)} | \
            {"copies": int(kt.copies)}
