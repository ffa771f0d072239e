"""Python binding of the softmax-attention side (``include/kda_attention.h``): the paged
key/value cache's plan and append, prompt attention and decode attention.

Argument marshalling only, as in the package itself; the header states layouts, masks and
errors.  q, k and v may be views of a fused projection's output: the heads of one token are
dense, the tokens evenly spaced.  All tensors are on the current device: the library launches there.
"""
import collections
import ctypes

import torch

import hybrid_linear_attention_kda_gb300 as _kda
from .attention_abi import KDA_DEV_BAD_GROUP, KDA_DEV_NO_BLOCKS, AttnDecodeArgs, AttnPrefillArgs, CachePlanArgs  # noqa: F401

#: What ``cache_plan`` returns: device tensors, as ``kda_cache_plan`` describes them.
CachePlan = collections.namedtuple("CachePlan", "cu_seqlens kv_lens slot_map positions")

_FLOATS = (torch.bfloat16, torch.float32)
_CODES = {torch.bfloat16: _kda.KDA_BF16, torch.float32: _kda.KDA_FP32}
_I32, _F32, _U8, _Tensor, _empty, _byref = torch.int32, torch.float32, torch.uint8, torch.Tensor, torch.empty, ctypes.byref

# A serving step makes these calls for every layer, so each tensor that passes is settled
# in one expression; what does not goes through the checks that name the fault.


def _shape(x, name, ndim):
    """``_kda._dims``, without a copy where the rank is right."""
    if type(x) is _Tensor and x.dim() == ndim:
        return x.shape
    return _kda._dims(x, name, ndim)


def _dev(x, name, dtype, shape, dev, index):
    """``_kda._dev`` of a tensor that must have this dtype, shape and device (of index ``index``)."""
    if type(x) is _Tensor and x.dtype is dtype and x.shape == shape and x.get_device() == index and x.is_contiguous():
        return x.data_ptr()
    return _kda._dev(x, name, dtype, shape, dev)


def _tokens(x, name, dtype, shape, dev, index):
    """(address, elements between tokens) of a [T, heads, d] tensor whose tokens are evenly
    spaced and whose heads are dense."""
    T, heads, d = shape
    if type(x) is _Tensor and x.dtype is dtype and x.shape == shape and x.get_device() == index and index >= 0:
        stride, inner, last = x.stride()
        if last == 1 and inner == d and stride >= heads * d:
            return x.data_ptr(), stride if T > 1 else heads * d         # between tokens: of one, of no account
    if not isinstance(x, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor (got {type(x).__name__})")
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {x.dtype})")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(x.shape)})")
    stride, inner, last = x.stride()
    if last != 1 or (inner != d and heads > 1):
        raise ValueError(f"{name}'s heads must be dense within a token (strides {x.stride()})")
    if T <= 1:
        stride = heads * d
    elif stride < heads * d:
        raise ValueError(f"{name}'s tokens overlap (strides {x.stride()})")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (got {x.device})")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, the other operands on {dev}")
    return x.data_ptr(), stride


def _current_device():
    return torch.cuda.current_device()


if hasattr(torch._C, "_cuda_getDevice"):                    # without the check that CUDA is up: a tensor is on it
    _current_device = torch._C._cuda_getDevice


def _not_current(index, name):
    """The library launches on the current device and sets that one's status word."""
    raise ValueError(f"{name} is on cuda:{index}, which is not the current device (cuda:{_current_device()})")


def _first(x, name):
    """(shape, dtype, its code, device, device index, address, stride) of the tensor that the
    others have to match."""
    shape = _shape(x, name, 3)
    dtype = x.dtype
    if dtype not in _CODES:
        raise TypeError(f"{name} must be {_FLOATS[0]} or {_FLOATS[1]} (got {dtype})")
    dev, index = x.device, x.get_device()
    ptr, stride = _tokens(x, name, dtype, shape, dev, index)
    if index != _current_device():
        _not_current(index, name)
    return shape, dtype, _CODES[dtype], dev, index, ptr, stride


def _on(stream, x):
    """A context in which ``stream`` is current, so that what is allocated belongs to it."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    return torch.cuda.stream(stream)


def _elsewhere(stream, x):
    """Whether a call has to be repeated under ``_on(stream, x)``; a tensor that is not on a GPU
    is left to the checks."""
    return stream is not None and isinstance(x, _Tensor) and x.is_cuda


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):          # the handle without a Stream object around it
    _current_stream = torch._C._cuda_getCurrentRawStream


def _cache(k_cache, v_cache, dtype, heads, d, dev, index):
    """(addresses, n_blocks, block_size) of the paged cache."""
    shape = _shape(k_cache, "k_cache", 4)
    n_blocks, bs = shape[0], shape[2]
    want = (n_blocks, heads, bs, d)
    return (_dev(k_cache, "k_cache", dtype, want, dev, index), _dev(v_cache, "v_cache", dtype, want, dev, index),
            n_blocks, bs)


def kda_cache_plan(args: CachePlanArgs, stream=None):
    _kda._check(_kda.load().kda_cache_plan(ctypes.byref(args), _kda._stream_handle(stream)))


def cache_plan(cached_lens, new_lens, block_table, free_blocks, free_begin, free_end, *, block_size, n_blocks,
               max_tokens, cu_seqlens=None, kv_lens=None, slot_map=None, positions=None, stream=None):
    """The cache metadata of one step (``kda_cache_plan``).  cached_lens, new_lens int32 [n];
    block_table int32 [n, stride], completed in place; free_blocks int32 [n_free]; free_begin,
    free_end int32 [1], two different tensors.  The outputs are allocated unless given, and may
    not overlap the inputs (kv_lens is not cached_lens).  Returns a ``CachePlan`` of cu_seqlens [n + 1], kv_lens [n], slot_map and positions
    [max_tokens]."""
    if _elsewhere(stream, cached_lens):
        with _on(stream, cached_lens):
            return cache_plan(cached_lens, new_lens, block_table, free_blocks, free_begin, free_end,
                              block_size=block_size, n_blocks=n_blocks, max_tokens=max_tokens, cu_seqlens=cu_seqlens,
                              kv_lens=kv_lens, slot_map=slot_map, positions=positions)
    n, = _shape(cached_lens, "cached_lens", 1)
    stride = _shape(block_table, "block_table", 2)[1]
    n_free, = _shape(free_blocks, "free_blocks", 1)
    T = int(max_tokens)
    if T < 0:
        raise ValueError(f"max_tokens must be >= 0 (got {T})")
    dev, ix = cached_lens.device, cached_lens.get_device()
    a0 = _dev(cached_lens, "cached_lens", _I32, (n,), None, ix if ix >= 0 else None)
    if ix != _current_device():
        _not_current(ix, "cached_lens")
    a1 = _dev(new_lens, "new_lens", _I32, (n,), dev, ix)
    a2 = _dev(free_blocks, "free_blocks", _I32, (n_free,), dev, ix)
    a3 = _dev(free_begin, "free_begin", _I32, (1,), dev, ix)
    a4 = _dev(free_end, "free_end", _I32, (1,), dev, ix)
    a5 = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv_lens = _empty(n, dtype=_I32, device=dev) if kv_lens is None else kv_lens
    cu_seqlens = _empty(n + 1, dtype=_I32, device=dev) if cu_seqlens is None else cu_seqlens
    slot_map = _empty(T, dtype=_I32, device=dev) if slot_map is None else slot_map
    positions = _empty(T, dtype=_I32, device=dev) if positions is None else positions
    a = CachePlanArgs(n, int(block_size), stride, n_free, int(n_blocks), T, a0, a1, a2, a3, a4, a5,
                      _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix), _dev(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev, ix),
                      _dev(slot_map, "slot_map", _I32, (T,), dev, ix), _dev(positions, "positions", _I32, (T,), dev, ix))
    status = _kda.load().kda_cache_plan(_byref(a), _current_stream(ix))
    if status:
        _kda._check(status)
    return CachePlan(cu_seqlens, kv_lens, slot_map, positions)


def kda_cache_append(k, v, slot_map, k_cache, v_cache, stream=None):
    """k_cache[slot] = k[t], v_cache[slot] = v[t] with slot = slot_map[t] (-1 skips the token).
    k, v [T, H_kv, d]; slot_map int32 [T]; caches [n_blocks, H_kv, block_size, d]."""
    shape, dtype, code, dev, ix, kp, ks = _first(k, "k")
    T, H, d = shape
    vp, vs = _tokens(v, "v", dtype, shape, dev, ix)
    sp = _dev(slot_map, "slot_map", _I32, (T,), dev, ix)
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, dtype, H, d, dev, ix)
    handle = _current_stream(ix) if stream is None else _kda._stream_handle(stream)
    status = _kda.load().kda_cache_append(T, H, d, code, kp, ks, vp, vs, sp, kc, vc, n_blocks, bs, handle)
    if status:
        _kda._check(status)


def kda_attn_prefill(args: AttnPrefillArgs, stream=None):
    _kda._check(_kda.load().kda_attn_prefill(ctypes.byref(args), _kda._stream_handle(stream)))


def _workspace(a, workspace, need, dev):
    """Give ``a`` the workspace, or a new one where it is missing or too small; the caller's
    frame keeps it until the launch."""
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        a._held = workspace = _empty(need, dtype=_U8, device=dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need
    else:
        a.workspace = _kda._dev(workspace, "workspace", device=dev)
        a.workspace_bytes = workspace.numel() * workspace.element_size()


def _outputs(dtype, shape, dev, ix, o, lse, want_lse):
    """(o, its address and stride, lse, its address), allocated where they are not given."""
    T, H, d = shape
    if o is None:
        o = _empty(shape, dtype=dtype, device=dev)
        op, os_ = o.data_ptr(), H * d
    else:
        op, os_ = _tokens(o, "o", dtype, shape, dev, ix)
    if lse is not None:
        return o, op, os_, lse, _dev(lse, "lse", _F32, (T, H), dev, ix)
    if not want_lse:
        return o, op, os_, None, None
    lse = _empty((T, H), dtype=_F32, device=dev)
    return o, op, os_, lse, lse.data_ptr()


def kda_attn_prefill_workspace_size(args: AttnPrefillArgs) -> int:
    return int(_kda.load().kda_attn_prefill_workspace_size(_byref(args)))


def _prefill(a, workspace, dev, ix):
    lib = _kda.load()
    need = lib.kda_attn_prefill_workspace_size(_byref(a))
    if need:
        _workspace(a, workspace, need, dev)
    status = lib.kda_attn_prefill(_byref(a), _current_stream(ix))
    if status:
        _kda._check(status)


def attn_prefill(q, k, v, cu_seqlens, *, scale=None, o=None, lse=None, want_lse=False, workspace=None, stream=None):
    """Causal attention over packed prompts (``kda_attn_prefill``): q [T, H, d]; k, v
    [T, H_kv, d]; cu_seqlens int32 [n + 1].  scale defaults to d^-0.5; o and lse are allocated
    unless given (tokens past cu_seqlens[n] are left unwritten), and so is the workspace
    (uint8), where one is of use.  Returns (o, lse or None)."""
    if _elsewhere(stream, q):
        with _on(stream, q):
            return attn_prefill(q, k, v, cu_seqlens, scale=scale, o=o, lse=lse, want_lse=want_lse, workspace=workspace)
    shape, dtype, code, dev, ix, qp, qs = _first(q, "q")
    T, H, d = shape
    kv = (T, _shape(k, "k", 3)[1], d)
    kp, ks = _tokens(k, "k", dtype, kv, dev, ix)
    vp, vs = _tokens(v, "v", dtype, kv, dev, ix)
    entries, = _shape(cu_seqlens, "cu_seqlens", 1)
    cu = _dev(cu_seqlens, "cu_seqlens", _I32, (entries,), dev, ix)
    o, op, os_, lse, zp = _outputs(dtype, shape, dev, ix, o, lse, want_lse)
    a = AttnPrefillArgs(entries - 1, H, kv[1], d, code, d ** -0.5 if scale is None else scale, T, qs, ks, vs, os_, qp, kp, vp,
                        op, zp, cu)
    _prefill(a, workspace, dev, ix)
    return o, lse


def attn_prefill_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, *, scale=None, o=None, lse=None,
                       want_lse=False, workspace=None, stream=None):
    """``attn_prefill`` with all keys and values in the paged cache: sequence s holds kv_lens[s]
    positions, the last of which are its queries.  caches [n_blocks, H_kv, block_size, d];
    block_table int32 [n, stride]; kv_lens int32 [n]; cu_seqlens int32 [n + 1].  Returns (o, lse
    or None)."""
    if _elsewhere(stream, q):
        with _on(stream, q):
            return attn_prefill_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, scale=scale, o=o, lse=lse,
                                      want_lse=want_lse, workspace=workspace)
    shape, dtype, code, dev, ix, qp, qs = _first(q, "q")
    T, H, d = shape
    H_kv = _shape(k_cache, "k_cache", 4)[1]
    n, stride = _shape(block_table, "block_table", 2)
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, dtype, H_kv, d, dev, ix)
    table = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    cu = _dev(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev, ix)
    if n and not stride:
        raise ValueError("block_table must have at least one column")
    o, op, os_, lse, zp = _outputs(dtype, shape, dev, ix, o, lse, want_lse)
    if n and T:
        a = AttnPrefillArgs(n, H, H_kv, d, code, d ** -0.5 if scale is None else scale, T, qs, 0, 0, os_, qp, None, None, op,
                            zp, cu, kc, vc, table, kv, n_blocks, bs, stride)
        _prefill(a, workspace, dev, ix)
    return o, lse


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
    if _elsewhere(stream, q):
        with _on(stream, q):
            return attn_decode(q, k_cache, v_cache, block_table, kv_lens, group_start=group_start,
                               prefix_lens=prefix_lens, scale=scale, o=o, lse=lse, want_lse=want_lse,
                               workspace=workspace)
    shape, dtype, code, dev, ix, qp, qs = _first(q, "q")
    n, H, d = shape
    H_kv = _shape(k_cache, "k_cache", 4)[1]
    stride = _shape(block_table, "block_table", 2)[1]
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, dtype, H_kv, d, dev, ix)
    table = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    groups, start, prefix = 0, None, None
    if group_start is not None:
        groups, = _shape(prefix_lens, "prefix_lens", 1)
        start = _dev(group_start, "group_start", _I32, (groups + 1,), dev, ix)
        prefix = _dev(prefix_lens, "prefix_lens", _I32, (groups,), dev, ix)
    o, op, os_, lse, zp = _outputs(dtype, shape, dev, ix, o, lse, want_lse)
    a = AttnDecodeArgs(n, H, H_kv, d, code, d ** -0.5 if scale is None else scale, qs, os_, qp, op, zp, kc, vc, table, kv,
                       n_blocks, bs, stride, groups, 0, start, prefix)
    lib = _kda.load()
    need = lib.kda_attn_decode_workspace_size(_byref(a))
    if need:
        _workspace(a, workspace, need, dev)
    status = lib.kda_attn_decode(_byref(a), _current_stream(ix))
    if status:
        _kda._check(status)
    return o, lse
