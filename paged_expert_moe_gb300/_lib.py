"""ctypes binding of libpagedmoe.so (include/pagedmoe.h): argument marshalling only.

Every function keeps the C name. Tensors are passed as raw device pointers
(``tensor.data_ptr()``) with the current torch CUDA stream; every step of the
layer runs in the library's own CUDA kernels. If the library is missing, loading
fails with an error (there is no fallback path).
"""

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpagedmoe.so")

PMOE_OK, PMOE_EINVAL, PMOE_ENOMEM, PMOE_EHOSTALLOC, PMOE_ECUDA, PMOE_EUNSUPPORTED, PMOE_ETIMEOUT, PMOE_EDEVICE = \
    0, -1, -2, -3, -4, -5, -6, -7
PMOE_BF16, PMOE_FP8_BLOCK128, PMOE_INT4_GPTQ_G128, PMOE_MXFP4, PMOE_NVFP4 = 0, 1, 2, 3, 4
PMOE_PAGEIN_COPY_ENGINE, PMOE_PAGEIN_SM_PULL = 0, 1
PMOE_KV_BF16, PMOE_KV_E4M3 = 0, 1


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


# The calls of a decode step take a few microseconds on the GPU, so their binding is kept
# lean: pointers go to ctypes as plain integers and the stream as its raw handle.

def _raw_stream(stream, like):
    import torch
    return torch._C._cuda_getCurrentRawStream(like.get_device()) if stream is None else stream.cuda_stream


def _opt(x, dtype, n):
    """The address of a contiguous CUDA tensor of n elements, None for None."""
    if x is None:
        return None
    assert x.dtype is dtype and x.is_cuda and x.numel() == n and x.is_contiguous(), (x.dtype, x.shape, dtype, n)
    return x.data_ptr()


def _empty(shape, dtype, like, stream):
    """A new tensor on the device of `like`, owned by `stream` (None: the current one)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(nbytes, stream):
    """The address of nbytes of device memory from torch's caching allocator, for `stream` (a
    raw handle). Given back with _release right after the launches: whatever reuses the block
    on this stream runs after them. (A tensor for it costs 8 us a call more.)"""
    import torch
    return torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, stream)


def _release(address):
    import torch
    torch._C._cuda_cudaCachingAllocator_raw_delete(address)


def _kv_desc(k_cache, v_cache, k_scale, v_scale):
    """pmoe_kv_desc of a paged cache: CUDA bf16 or float8_e4m3fn [num_pages, kv_heads,
    page_size, head_dim] tensors of the same strides, contiguous but for the page stride."""
    import torch
    pages, heads, page, dim = shape = k_cache.shape
    stride = k_cache.stride()
    dt = k_cache.dtype
    assert k_cache.is_cuda and v_cache.is_cuda and v_cache.dtype is dt and v_cache.shape == shape
    assert v_cache.stride() == stride and stride[1:] == (page * dim, dim, 1)
    if dt is torch.bfloat16:
        return pmoe_kv_desc(k_cache.data_ptr(), v_cache.data_ptr(), stride[0], None, None, pages, page, heads, dim,
                            PMOE_KV_BF16)
    assert dt is torch.float8_e4m3fn
    return pmoe_kv_desc(k_cache.data_ptr(), v_cache.data_ptr(), stride[0], _opt(k_scale, torch.float32, heads),
                        _opt(v_scale, torch.float32, heads), pages, page, heads, dim, PMOE_KV_E4M3)


def _heads(x, T, heads, dim):
    """(address, elements from token to token) of bf16 x [T, heads, dim] whose heads are
    contiguous; one token or head has no stride of its own."""
    import torch
    st, sh, sd = x.stride()
    assert x.dtype is torch.bfloat16 and x.is_cuda and x.shape == (T, heads, dim)
    assert sd == 1 and (sh == dim or heads == 1)
    return x.data_ptr(), st if T > 1 else heads * dim


def moe_kv_append(k_cache, v_cache, q, k, v, positions, slots, inv_freq, pair_axis=None, interleaved=False, q_norm=None,
                  k_norm=None, eps=1e-6, k_scale=None, v_scale=None, q_out=None, err_out=None, stream=None):
    """Head norm, rotation and append of T tokens' keys and values to a paged cache.
    k_cache, v_cache: bf16 or float8_e4m3fn [num_pages, kv_heads, page_size, head_dim];
    q: bf16 [T, q_heads, head_dim], k, v: bf16 [T, kv_heads, head_dim] (views of one
    projection will do); positions: int32 [axes, T] or [T]; slots: int32 [T], page *
    page_size + row, -1 = not stored; inv_freq: fp32 [rotary_dim / 2] or None; pair_axis:
    int32 [rotary_dim / 2]; q_norm, k_norm: bf16 [head_dim]. Returns the rotated q (q_out)."""
    import torch
    T, q_heads, dim = q.shape
    desc = _kv_desc(k_cache, v_cache, k_scale, v_scale)
    hk = desc.kv_heads
    assert dim == desc.head_dim
    i32, bf16 = torch.int32, torch.bfloat16
    axes = positions.shape[0] if positions is not None and positions.dim() == 2 else 1
    pairs = 0 if inv_freq is None else inv_freq.numel()
    if q_out is None:
        q_out = _empty((T, q_heads, dim), bf16, q, stream)
    _check(load().moe_kv_append(desc, *_heads(q, T, q_heads, dim), *_heads(k, T, hk, dim), *_heads(v, T, hk, dim), T,
                                q_heads, _opt(positions, i32, axes * T), axes, _opt(pair_axis, i32, pairs),
                                _opt(inv_freq, torch.float32, pairs), 2 * pairs, 1 if interleaved else 0,
                                _opt(q_norm, bf16, dim), _opt(k_norm, bf16, dim), eps, _opt(slots, i32, T),
                                _opt(q_out, bf16, T * q_heads * dim), _opt(err_out, i32, 1), _raw_stream(stream, q)),
           "moe_kv_append")
    return q_out


def moe_prefix_attention_scratch_bytes(k_cache, v_cache, T, q_heads, prefix_len, max_suffix, k_scale=None, v_scale=None):
    """Bytes of scratch a moe_prefix_attention call of these sizes needs."""
    return int(load().moe_prefix_attention_scratch_bytes(_kv_desc(k_cache, v_cache, k_scale, v_scale), T, q_heads,
                                                         prefix_len, max_suffix))


def moe_prefix_attention(k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, scale=None,
                         row_seq=None, k_scale=None, v_scale=None, out=None, lse_out=None, scratch=None, err_out=None,
                         stream=None):
    """Attention of q (bf16 [T, q_heads, head_dim]) over a paged cache (as moe_kv_append's).
    Row t sees the first prefix_len keys of prefix_pages (int32), which all rows share, then
    the first suffix_len[t] (int32 [T], at most max_suffix) of page_table[row_seq[t]] (int32
    [sequences, pages]; row_seq int32 [T], default t). scale defaults to head_dim ** -0.5.
    lse_out: fp32 [T, q_heads] or None; scratch: uint8, allocated here when not given.
    Returns out (bf16 [T, q_heads, head_dim])."""
    import torch
    T, q_heads, dim = q.shape
    desc = _kv_desc(k_cache, v_cache, k_scale, v_scale)
    i32 = torch.int32
    assert dim == desc.head_dim
    pages = None
    if prefix_len > 0:
        n = prefix_pages.numel()
        assert n * desc.page_size >= prefix_len
        pages = _opt(prefix_pages, i32, n)
    table = lens = None
    sequences = width = 0
    if max_suffix > 0:
        sequences, width = page_table.shape
        table, lens = _opt(page_table, i32, sequences * width), _opt(suffix_len, i32, T)
    lib = load()
    if out is None:
        out = _empty((T, q_heads, dim), torch.bfloat16, q, stream)
    raw = _raw_stream(stream, q)
    own = None
    if scratch is not None:
        nbytes = scratch.numel()
        work = _opt(scratch, torch.uint8, nbytes)
    else:
        nbytes = lib.moe_prefix_attention_scratch_bytes(desc, T, q_heads, prefix_len, max_suffix)
        work = own = _scratch(nbytes, raw) if nbytes else None
    try:
        _check(lib.moe_prefix_attention(desc, *_heads(q, T, q_heads, dim), T, q_heads,
                                        dim ** -0.5 if scale is None else scale, pages, prefix_len, table, width, sequences,
                                        _opt(row_seq, i32, T), lens, max_suffix, _opt(out, torch.bfloat16, T * q_heads * dim),
                                        _opt(lse_out, torch.float32, T * q_heads), work, nbytes, _opt(err_out, i32, 1), raw),
               "moe_prefix_attention")
    finally:
        if own is not None:
            _release(own)
    return out


def moe_sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ids_out=None, logprob_out=None,
                      stream=None):
    """Draw one token id per row of logits (CUDA fp32 or bf16 [T, V], rows contiguous) from
    u (fp32 [T], in [0, 1)). temperature, top_p, min_p: fp32 [T], top_k: int32 [T], or None
    (1, 1, 0 and 0: no cut); temperature 0 takes the largest logit. logprob_out: fp32 [T],
    the drawn token's log probability among the kept ones. Returns ids (int32 [T])."""
    import torch
    T, V = logits.shape
    dt, f32 = logits.dtype, torch.float32
    st, sv = logits.stride()
    assert logits.is_cuda and (dt is f32 or dt is torch.bfloat16) and (V == 1 or sv == 1)
    if ids_out is None:
        ids_out = _empty(T, torch.int32, logits, stream)
    _check(load().moe_sample_tokens(logits.data_ptr(), 0 if dt is f32 else 1, T, V, st if T > 1 else V,
                                    _opt(temperature, f32, T), _opt(top_k, torch.int32, T), _opt(top_p, f32, T),
                                    _opt(min_p, f32, T), _opt(u, f32, T), _opt(ids_out, torch.int32, T),
                                    _opt(logprob_out, f32, T), _raw_stream(stream, logits)), "moe_sample_tokens")
    return ids_out


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
