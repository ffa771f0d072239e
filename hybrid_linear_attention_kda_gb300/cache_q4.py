"""Python binding of the paged key/value cache in 4 bits (``include/kda_cache_q4.h``): its append, its read-back into a
full-width cache, and decode attention over it.

Argument marshalling only, as in the package itself; the header states format, layouts and errors.  k and v may be views of
a fused projection's output.  All tensors are on the current device: the library launches there.
"""
import collections
import ctypes
import struct

import torch

import hybrid_linear_attention_kda_gb300 as _kda
from . import attention as _attention
from .attention import (_cache, _current_stream, _dev, _elsewhere, _empty, _first, _FLOATS, _I32, _on, _outputs, _shape, _tokens,
                        _U8)
from .attention_abi import PACK, AttnDecodeQ4Args, CacheAppendQ4Args, CacheUnpackQ4Args

_BF, _byref = torch.bfloat16, ctypes.byref
_pack_append, _pack_unpack, _pack_decode = (struct.Struct(PACK[block]).pack for block in (CacheAppendQ4Args, CacheUnpackQ4Args, AttnDecodeQ4Args))
GROUP = 64          # channels that share a scale

#: The cache's tensors: codes uint8 [n_blocks, H_kv, block_size, d / 2], scales bf16 [n_blocks, H_kv, block_size, d / 64, 2].
Q4Cache = collections.namedtuple("Q4Cache", "k_codes k_scales v_codes v_scales")


def q4_cache(n_blocks, n_kv_heads, block_size, d, device=None):
    """A new ``Q4Cache``, uninitialised."""
    if d % GROUP:
        raise ValueError(f"d must be a multiple of {GROUP} (got {d})")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    shape = (n_blocks, n_kv_heads, block_size)
    return Q4Cache(*(t for _ in range(2) for t in (torch.empty((*shape, d // 2), dtype=_U8, device=device),
                                                   torch.empty((*shape, d // GROUP, 2), dtype=_BF, device=device))))


def _q4(cache, heads, d, dev, index):
    """The cache's argument block, as values to pack: four addresses, n_blocks, block_size, 0."""
    k_codes, k_scales, v_codes, v_scales = cache
    n_blocks, _, bs, _ = _shape(k_codes, "k_codes", 4)
    codes, scales = (n_blocks, heads, bs, d // 2), (n_blocks, heads, bs, d // GROUP, 2)
    return (_dev(k_codes, "k_codes", _U8, codes, dev, index), _dev(k_scales, "k_scales", _BF, scales, dev, index),
            _dev(v_codes, "v_codes", _U8, codes, dev, index), _dev(v_scales, "v_scales", _BF, scales, dev, index), n_blocks, bs, 0)


def kda_cache_append_q4(args: CacheAppendQ4Args, stream=None):
    _kda._check(_kda.load().kda_cache_append_q4(_byref(args), _kda._stream_handle(stream)))


def cache_append_q4(k, v, slot_map, cache, *, k_out=None, v_out=None, want_values=False, stream=None):
    """The tokens' keys and values into the 4-bit cache (``kda_cache_append_q4``): k, v [T, H_kv, d]; slot_map int32 [T], -1
    skips the token; cache a ``Q4Cache``.  k_out and v_out receive the values that the cache now stands for, in k's type
    (skipped tokens' rows are left as they are); they may be k and v, and are allocated with want_values.  Returns (k_out,
    v_out)."""
    if _elsewhere(stream, k):
        with _on(stream, k):
            return cache_append_q4(k, v, slot_map, cache, k_out=k_out, v_out=v_out, want_values=want_values)
    shape, dtype, code, dev, ix, kp, ks = _first(k, "k")
    T, H_kv, d = shape
    vp, vs = _tokens(v, "v", dtype, shape, dev, ix)
    slots = _dev(slot_map, "slot_map", _I32, (T,), dev, ix)
    block = _q4(cache, H_kv, d, dev, ix)
    if want_values:
        k_out = _empty(shape, dtype=dtype, device=dev) if k_out is None else k_out
        v_out = _empty(shape, dtype=dtype, device=dev) if v_out is None else v_out
    ko, kos = (0, 0) if k_out is None else _tokens(k_out, "k_out", dtype, shape, dev, ix)
    vo, vos = (0, 0) if v_out is None else _tokens(v_out, "v_out", dtype, shape, dev, ix)
    a = _pack_append(T, H_kv, d, code, 0, ks, vs, kos, vos, kp, vp, ko, vo, slots, *block)
    status = _kda.load().kda_cache_append_q4(a, _current_stream(ix))
    if status:
        _kda._check(status)
    return k_out, v_out


def kda_cache_unpack_q4(args: CacheUnpackQ4Args, stream=None):
    _kda._check(_kda.load().kda_cache_unpack_q4(_byref(args), _kda._stream_handle(stream)))


def cache_unpack_q4(cache, block_table, kv_lens, k_cache, v_cache, to_table, *, first=None, stream=None):
    """Positions first[s] (None: 0) .. kv_lens[s] - 1 of each sequence out of the 4-bit cache, by block_table int32 [n,
    stride], into the full-width caches [n_blocks, H_kv, block_size, d], by to_table int32 [n, stride 2]
    (``kda_cache_unpack_q4``)."""
    if _elsewhere(stream, k_cache):
        with _on(stream, k_cache):
            return cache_unpack_q4(cache, block_table, kv_lens, k_cache, v_cache, to_table, first=first)
    wide, H_kv, bs, d = _shape(k_cache, "k_cache", 4)
    dtype = k_cache.dtype
    if dtype not in _FLOATS:
        raise TypeError(f"k_cache must be {_FLOATS[0]} or {_FLOATS[1]} (got {dtype})")
    dev, ix = k_cache.device, k_cache.get_device()
    kc = _dev(k_cache, "k_cache", dtype, (wide, H_kv, bs, d), None, ix if ix >= 0 else None)
    if ix != _attention._current_device():
        _attention._not_current(ix, "k_cache")
    vc = _dev(v_cache, "v_cache", dtype, (wide, H_kv, bs, d), dev, ix)
    block = _q4(cache, H_kv, d, dev, ix)
    if block[5] != bs:
        raise ValueError(f"the caches' block sizes differ ({block[5]} and {bs})")
    n, stride = _shape(block_table, "block_table", 2)
    to_stride = _shape(to_table, "to_table", 2)[1]
    table, to = _dev(block_table, "block_table", _I32, (n, stride), dev, ix), _dev(to_table, "to_table", _I32, (n, to_stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    at = 0 if first is None else _dev(first, "first", _I32, (n,), dev, ix)
    a = _pack_unpack(n, H_kv, d, _kda.KDA_BF16 if dtype == _BF else _kda.KDA_FP32, *block, table, to, stride, to_stride, at,
                     kv, kc, vc, wide)
    status = _kda.load().kda_cache_unpack_q4(a, _current_stream(ix))
    if status:
        _kda._check(status)


def kda_attn_decode_q4_workspace_size(args: AttnDecodeQ4Args) -> int:
    return int(_kda.load().kda_attn_decode_q4_workspace_size(_byref(args)))


def kda_attn_decode_q4(args: AttnDecodeQ4Args, stream=None):
    _kda._check(_kda.load().kda_attn_decode_q4(_byref(args), _kda._stream_handle(stream)))


def attn_decode_q4(q, cache, block_table, kv_lens, *, k_prefix=None, v_prefix=None, group_start=None, prefix_lens=None,
                   scale=None, o=None, lse=None, want_lse=False, workspace=None, stream=None):
    """Decode attention over the 4-bit cache (``kda_attn_decode_q4``): one query per sequence, q [n, H, d], over its
    kv_lens[s] positions.  group_start int32 [g + 1], prefix_lens int32 [g] and the full-width caches k_prefix, v_prefix
    [n_blocks, H_kv, block_size, d] come together: the groups of consecutive sequences whose first positions are shared, and
    where those positions are (their entries of block_table are blocks of k_prefix).  The rest as for ``attn_decode``.
    Returns (o, lse or None)."""
    if group_start is None:
        apart = k_prefix is not None or v_prefix is not None or prefix_lens is not None
    else:
        apart = k_prefix is None or v_prefix is None or prefix_lens is None
    if apart:
        raise ValueError("k_prefix, v_prefix, group_start and prefix_lens come together")
    if _elsewhere(stream, q):
        with _on(stream, q):
            return attn_decode_q4(q, cache, block_table, kv_lens, k_prefix=k_prefix, v_prefix=v_prefix,
                                  group_start=group_start, prefix_lens=prefix_lens, scale=scale, o=o, lse=lse,
                                  want_lse=want_lse, workspace=workspace)
    shape, dtype, code, dev, ix, qp, qs = _first(q, "q")
    n, H, d = shape
    H_kv = _shape(cache[0], "k_codes", 4)[1]
    stride = _shape(block_table, "block_table", 2)[1]
    block = _q4(cache, H_kv, d, dev, ix)
    bs = block[5]
    table = _dev(block_table, "block_table", _I32, (n, stride), dev, ix)
    kv = _dev(kv_lens, "kv_lens", _I32, (n,), dev, ix)
    groups = start = prefix = kc = vc = wide = 0
    if group_start is not None:
        groups, = _shape(prefix_lens, "prefix_lens", 1)
        start = _dev(group_start, "group_start", _I32, (groups + 1,), dev, ix)
        prefix = _dev(prefix_lens, "prefix_lens", _I32, (groups,), dev, ix)
        kc, vc, wide, prefix_bs = _cache(k_prefix, v_prefix, dtype, H_kv, d, dev, ix)
        if prefix_bs != bs:
            raise ValueError(f"the caches' block sizes differ ({prefix_bs} and {bs})")
    o, op, os_, lse, zp = _outputs(dtype, shape, dev, ix, o, lse, want_lse)
    before = (n, H, H_kv, d, code, d ** -0.5 if scale is None else scale, qs, os_, qp, op, zp or 0, kc, vc, table, kv, wide, bs,
              stride, groups, 0, start, prefix)
    lib = _kda.load()
    need = lib.kda_attn_decode_q4_workspace_size(_pack_decode(*before, 0, 0, *block))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = _empty(need, dtype=_U8, device=dev)
        at = workspace.data_ptr()
    else:
        at, need = _kda._dev(workspace, "workspace", device=dev), workspace.numel() * workspace.element_size()
    status = lib.kda_attn_decode_q4(_pack_decode(*before, at, need, *block), _current_stream(ix))
    if status:
        _kda._check(status)
    return o, lse
