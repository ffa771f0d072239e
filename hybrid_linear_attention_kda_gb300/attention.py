"""Python binding of the softmax-attention side (``include/kda_attention.h``): the paged
key/value cache's plan and append, prompt attention and decode attention.

Argument marshalling only, as in the package itself; the header states layouts, masks and
errors.  q, k and v may be views of a fused projection's output: the heads of one token are
dense, the tokens evenly spaced.
"""
import collections
import ctypes

import torch

import hybrid_linear_attention_kda_gb300 as _kda

KDA_DEV_NO_BLOCKS, KDA_DEV_BAD_GROUP = 0x40, 0x80


class CachePlanArgs(ctypes.Structure):
    """Mirror of ``kda_cache_plan_args``."""
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("block_size", ctypes.c_int32), ("table_stride", ctypes.c_int32),
        ("n_free", ctypes.c_int32), ("n_blocks", ctypes.c_int64), ("max_tokens", ctypes.c_int64),
        ("cached_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("free_blocks", ctypes.c_void_p),
        ("free_begin", ctypes.c_void_p), ("free_end", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("slot_map", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


class AttnPrefillArgs(ctypes.Structure):
    """Mirror of ``kda_attn_prefill_args``."""
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("total_tokens", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
        ("n_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32), ("table_stride", ctypes.c_int32),
    ]


class AttnDecodeArgs(ctypes.Structure):
    """Mirror of ``kda_attn_decode_args``."""
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("q_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64), ("q", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("n_blocks", ctypes.c_int64),
        ("block_size", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("n_groups", ctypes.c_int32),
        ("reserved0", ctypes.c_int32), ("group_start", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


#: What ``cache_plan`` returns: device tensors, as ``kda_cache_plan`` describes them.
CachePlan = collections.namedtuple("CachePlan", "cu_seqlens kv_lens slot_map positions")


def declare(lib):
    """Set the ctypes signatures of the entry points."""
    vp, i32, i64, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER
    lib.kda_cache_plan.restype = ctypes.c_int
    lib.kda_cache_plan.argtypes = [P(CachePlanArgs), vp]
    lib.kda_cache_append.restype = ctypes.c_int
    lib.kda_cache_append.argtypes = [i64, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, i64, i32, vp]
    lib.kda_attn_prefill.restype = ctypes.c_int
    lib.kda_attn_prefill.argtypes = [P(AttnPrefillArgs), vp]
    lib.kda_attn_decode_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_decode_workspace_size.argtypes = [P(AttnDecodeArgs)]
    lib.kda_attn_decode.restype = ctypes.c_int
    lib.kda_attn_decode.argtypes = [P(AttnDecodeArgs), vp]


_FLOATS = (torch.bfloat16, torch.float32)
_I32, _F32, _Tensor = torch.int32, torch.float32, torch.Tensor


def _shape(x, name, ndim):
    """``_kda._dims``, without a copy where the rank is right."""
    if type(x) is _Tensor and x.dim() == ndim:
        return x.shape
    return _kda._dims(x, name, ndim)


def _dev(x, name, dtype, shape, dev, index):
    """``_kda._dev`` of a tensor that must have this dtype, shape and device (of index
    ``index``).  A serving step makes these calls for every layer, so what passes is
    settled in one expression; what does not goes through the checks that name the fault."""
    if type(x) is _Tensor and x.dtype is dtype and x.shape == shape and x.get_device() == index and x.is_contiguous():
        return x.data_ptr()
    return _kda._dev(x, name, dtype, shape, dev)


def _tokens(x, name, dtype, shape, dev=None):
    """(address, elements between tokens) of a [T, heads, d] tensor whose tokens are
    evenly spaced and whose heads are dense."""
    T, heads, d = shape
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor (got {type(x).__name__})")
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {x.dtype})")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(x.shape)})")
    stride, inner, last = x.stride()
    if (last != 1 and d > 1) or (inner != d and heads > 1):
        raise ValueError(f"{name}'s heads must be dense within a token (strides {x.stride()})")
    if T <= 1:
        stride = heads * d
    elif stride < heads * d:
        raise ValueError(f"{name}'s tokens overlap (strides {x.stride()})")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (got {x.device})")
    if dev is not None and x.device != dev:
        raise ValueError(f"{name} is on {x.device}, the other operands on {dev}")
    return x.data_ptr(), stride


def _first(x, name):
    """(shape, address, stride, device, device index, dtype code) of the tensor that the others
    have to match."""
    shape = _shape(x, name, 3)
    if x.dtype not in _FLOATS:
        raise TypeError(f"{name} must be {_FLOATS[0]} or {_FLOATS[1]} (got {x.dtype})")
    ptr, stride = _tokens(x, name, x.dtype, shape)
    return shape, ptr, stride, x.device, x.get_device(), _kda._dtype_code(x)


def _on_stream(stream, dev, call):
    """``call(handle)`` with ``stream`` current, so that what is allocated inside belongs to it."""
    if stream is None:
        return call(_current_stream(dev))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _current_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):          # the handle without a Stream object around it
    def _current_stream(dev):                                # noqa: F811
        return torch._C._cuda_getCurrentRawStream(dev.index)


def _cache(k_cache, v_cache, dtype, heads, d, dev, index):
    """(addresses, n_blocks, block_size) of the paged cache."""
    n_blocks, _, bs, _ = _shape(k_cache, "k_cache", 4)
    shape = (n_blocks, heads, bs, d)
    return (_dev(k_cache, "k_cache", dtype, shape, dev, index), _dev(v_cache, "v_cache", dtype, shape, dev, index),
            n_blocks, bs)


def kda_cache_plan(args: CachePlanArgs, stream=None):
    _kda._check(_kda.load().kda_cache_plan(ctypes.byref(args), _kda._stream_handle(stream)))


def cache_plan(cached_lens, new_lens, block_table, free_blocks, free_begin, free_end, *, block_size, n_blocks,
               max_tokens, cu_seqlens=None, kv_lens=None, slot_map=None, positions=None, stream=None):
    """The cache metadata of one step (``kda_cache_plan``).  cached_lens, new_lens int32 [n];
    block_table int32 [n, stride], completed in place; free_blocks int32 [n_free]; free_begin,
    free_end int32 [1], two different tensors.  The outputs are allocated unless given.
    Returns a ``CachePlan`` of cu_seqlens [n + 1], kv_lens [n], slot_map and positions
    [max_tokens]."""
    n, = _shape(cached_lens, "cached_lens", 1)
    _, stride = _shape(block_table, "block_table", 2)
    n_free, = _shape(free_blocks, "free_blocks", 1)
    T = int(max_tokens)
    if T < 0:
        raise ValueError(f"max_tokens must be >= 0 (got {T})")
    dev, ix = cached_lens.device, cached_lens.get_device()
    ptrs = (_dev(cached_lens, "cached_lens", _I32, (n,), None, ix if ix >= 0 else None),
            _dev(new_lens, "new_lens", _I32, (n,), dev, ix),
            _dev(free_blocks, "free_blocks", _I32, (n_free,), dev, ix),
            _dev(free_begin, "free_begin", _I32, (1,), dev, ix), _dev(free_end, "free_end", _I32, (1,), dev, ix),
            _dev(block_table, "block_table", _I32, (n, stride), dev, ix))

    def call(handle):
        def out(x, name, size):
            if x is None:
                x = torch.empty(size, dtype=_I32, device=dev)
                return x, x.data_ptr()
            return x, _dev(x, name, _I32, (size,), dev, ix)
        kv, kv_p = out(kv_lens, "kv_lens", n)
        cu, cu_p = out(cu_seqlens, "cu_seqlens", n + 1)
        slots, slots_p = out(slot_map, "slot_map", T)
        pos, pos_p = out(positions, "positions", T)
        a = CachePlanArgs(n, int(block_size), stride, n_free, int(n_blocks), T, *ptrs, kv_p, cu_p, slots_p, pos_p)
        _kda._check(_kda.load().kda_cache_plan(ctypes.byref(a), handle))
        return CachePlan(cu, kv, slots, pos)
    return _on_stream(stream, dev, call)


def kda_cache_append(k, v, slot_map, k_cache, v_cache, stream=None):
    """k_cache[slot] = k[t], v_cache[slot] = v[t] with slot = slot_map[t] (-1 skips the token).
    k, v [T, H_kv, d]; slot_map int32 [T]; caches [n_blocks, H_kv, block_size, d]."""
    shape, kp, ks, dev, ix, code = _first(k, "k")
    T, H, d = shape
    vp, vs = _tokens(v, "v", k.dtype, shape, dev)
    sp = _dev(slot_map, "slot_map", _I32, (T,), dev, ix)
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, k.dtype, H, d, dev, ix)
    handle = _current_stream(dev) if stream is None else _kda._stream_handle(stream)
    _kda._check(_kda.load().kda_cache_append(T, H, d, code, kp, ks, vp, vs, sp, kc, vc, n_blocks, bs, handle))


def kda_attn_prefill(args: AttnPrefillArgs, stream=None):
    _kda._check(_kda.load().kda_attn_prefill(ctypes.byref(args), _kda._stream_handle(stream)))


def _outputs(q, shape, dev, ix, o, lse, want_lse):
    """(o, its address and stride, lse, its address), allocated where they are not given."""
    T, H, d = shape
    if o is None:
        o = torch.empty(shape, dtype=q.dtype, device=dev)
        op, os_ = o.data_ptr(), H * d
    else:
        op, os_ = _tokens(o, "o", q.dtype, shape, dev)
    if lse is not None:
        return o, op, os_, lse, _dev(lse, "lse", _F32, (T, H), dev, ix)
    if not want_lse:
        return o, op, os_, None, None
    lse = torch.empty((T, H), dtype=_F32, device=dev)
    return o, op, os_, lse, lse.data_ptr()


def _scale(scale, d):
    return d ** -0.5 if scale is None else float(scale)


def attn_prefill(q, k, v, cu_seqlens, *, scale=None, o=None, lse=None, want_lse=False, stream=None):
    """Causal attention over packed prompts (``kda_attn_prefill``): q [T, H, d]; k, v
    [T, H_kv, d]; cu_seqlens int32 [n + 1].  scale defaults to d^-0.5; o and lse are allocated
    unless given (tokens past cu_seqlens[n] are left unwritten).  Returns (o, lse or None)."""
    shape, qp, qs, dev, ix, code = _first(q, "q")
    T, H, d = shape
    H_kv = _shape(k, "k", 3)[1]
    kp, ks = _tokens(k, "k", q.dtype, (T, H_kv, d), dev)
    vp, vs = _tokens(v, "v", q.dtype, (T, H_kv, d), dev)
    entries, = _shape(cu_seqlens, "cu_seqlens", 1)
    cu = _dev(cu_seqlens, "cu_seqlens", _I32, (entries,), dev, ix)

    def call(handle):
        out, op, os_, z, zp = _outputs(q, shape, dev, ix, o, lse, want_lse)
        a = AttnPrefillArgs(entries - 1, H, H_kv, d, code, _scale(scale, d), T, qs, ks, vs, os_, qp, kp, vp, op, zp, cu)
        _kda._check(_kda.load().kda_attn_prefill(ctypes.byref(a), handle))
        return out, z
    return _on_stream(stream, dev, call)


def attn_prefill_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, *, scale=None, o=None, lse=None,
                       want_lse=False, stream=None):
    """``attn_prefill`` with all keys and values in the paged cache: sequence s holds kv_lens[s]
    positions, the last of which are its queries.  caches [n_blocks, H_kv, block_size, d];
    block_table int32 [n, stride]; kv_lens int32 [n]; cu_seqlens int32 [n + 1].  Returns (o, lse
    or None)."""
    shape, qp, qs, dev, ix, code = _first(q, "q")
    T, H, d = shape
    H_kv = _shape(k_cache, "k_cache", 4)[1]
    n, stride = _shape(block_table, "block_table", 2)
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, q.dtype, H_kv, d, dev, ix)
    table = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    cu = _dev(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev, ix)
    if n and not stride:
        raise ValueError("block_table must have at least one column")

    def call(handle):
        out, op, os_, z, zp = _outputs(q, shape, dev, ix, o, lse, want_lse)
        if n and T:
            a = AttnPrefillArgs(n, H, H_kv, d, code, _scale(scale, d), T, qs, 0, 0, os_, qp, None, None, op, zp, cu, kc, vc,
                                table, kv, n_blocks, bs, stride)
            _kda._check(_kda.load().kda_attn_prefill(ctypes.byref(a), handle))
        return out, z
    return _on_stream(stream, dev, call)


def kda_attn_decode_workspace_size(args: AttnDecodeArgs) -> int:
    return int(_kda.load().kda_attn_decode_workspace_size(ctypes.byref(args)))


def kda_attn_decode(args: AttnDecodeArgs, stream=None):
    _kda._check(_kda.load().kda_attn_decode(ctypes.byref(args), _kda._stream_handle(stream)))


def attn_decode(q, k_cache, v_cache, block_table, kv_lens, *, group_start=None, prefix_lens=None, scale=None, o=None,
                lse=None, want_lse=False, workspace=None, stream=None):
    """Decode attention over the paged cache (``kda_attn_decode``): one query per sequence,
    q [n, H, d], over its kv_lens[s] positions.  group_start int32 [g + 1] and prefix_lens
    int32 [g] name the groups of consecutive sequences that share their first blocks; those
    are read once per group.  workspace: uint8, allocated unless a large enough one is given.
    Returns (o, lse or None)."""
    if (group_start is None) != (prefix_lens is None):
        raise ValueError("group_start and prefix_lens come together")
    shape, qp, qs, dev, ix, code = _first(q, "q")
    n, H, d = shape
    H_kv = _shape(k_cache, "k_cache", 4)[1]
    stride = _shape(block_table, "block_table", 2)[1]
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, q.dtype, H_kv, d, dev, ix)
    table = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    groups, start, prefix = 0, None, None
    if group_start is not None:
        groups, = _shape(prefix_lens, "prefix_lens", 1)
        start = _dev(group_start, "group_start", _I32, (groups + 1,), dev, ix)
        prefix = _dev(prefix_lens, "prefix_lens", _I32, (groups,), dev, ix)

    def call(handle):
        out, op, os_, z, zp = _outputs(q, shape, dev, ix, o, lse, want_lse)
        a = AttnDecodeArgs(n, H, H_kv, d, code, _scale(scale, d), qs, os_, qp, op, zp, kc, vc, table, kv, n_blocks, bs,
                           stride, groups, 0, start, prefix)
        lib = _kda.load()
        need, ws = lib.kda_attn_decode_workspace_size(ctypes.byref(a)), workspace
        if need:
            if ws is None or ws.numel() * ws.element_size() < need:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
            a.workspace = _kda._dev(ws, "workspace", device=dev)
            a.workspace_bytes = ws.numel() * ws.element_size()
        _kda._check(lib.kda_attn_decode(ctypes.byref(a), handle))
        return out, z
    return _on_stream(stream, dev, call)
