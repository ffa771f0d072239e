"""Python binding of the softmax-attention side (``include/kda_attention.h``): the paged
key/value cache's plan and append, prompt attention and decode attention.

Argument marshalling only, as in the package itself; the header states layouts, masks and
errors.  q, k and v may be views of a fused projection's output: the heads of one token are
dense, the tokens evenly spaced.
"""
import collections
import contextlib
import ctypes

import torch

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


def _base():
    import hybrid_linear_attention_kda_gb300 as kda
    return kda


_FLOATS = (torch.bfloat16, torch.float32)


def _tokens(x, name, dtype, heads, d, device, rows=None):
    """(address, elements between tokens) of a [T, heads, d] tensor whose tokens are
    evenly spaced and whose heads are dense."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor (got {type(x).__name__})")
    allowed = dtype if isinstance(dtype, tuple) else (dtype,)
    if x.dtype not in allowed:
        raise TypeError(f"{name} must be {' or '.join(str(t) for t in allowed)} (got {x.dtype})")
    want = (x.shape[0] if rows is None and x.dim() else rows, heads, d)
    if tuple(x.shape) != want:
        raise ValueError(f"{name} must have shape {want} (got {tuple(x.shape)})")
    stride, inner, last = x.stride()
    if (last != 1 and d > 1) or (inner != d and heads > 1):
        raise ValueError(f"{name}'s heads must be dense within a token (strides {x.stride()})")
    if x.shape[0] <= 1:
        stride = heads * d
    if stride < heads * d:
        raise ValueError(f"{name}'s tokens overlap (strides {x.stride()})")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (got {x.device})")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, the other operands on {device}")
    return x.data_ptr(), stride


@contextlib.contextmanager
def _on(stream, device):
    """Make ``stream`` current, so that what is allocated inside belongs to it."""
    if stream is None:
        yield
        return
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        yield


def _cache(kda, k_cache, v_cache, dtype, heads, d, dev):
    """(addresses, n_blocks, block_size) of the paged cache."""
    n_blocks, _, bs, _ = kda._dims(k_cache, "k_cache", 4)
    shape = (n_blocks, heads, bs, d)
    return (kda._dev(k_cache, "k_cache", dtype, shape, dev), kda._dev(v_cache, "v_cache", dtype, shape, dev),
            n_blocks, bs)


def kda_cache_plan(args: CachePlanArgs, stream=None):
    kda = _base()
    kda._check(kda.load().kda_cache_plan(ctypes.byref(args), kda._stream_handle(stream)))


def cache_plan(cached_lens, new_lens, block_table, free_blocks, free_begin, free_end, *, block_size, n_blocks,
               max_tokens, cu_seqlens=None, kv_lens=None, slot_map=None, positions=None, stream=None):
    """The cache metadata of one step (``kda_cache_plan``).  cached_lens, new_lens int32 [n];
    block_table int32 [n, stride], completed in place; free_blocks int32 [n_free]; free_begin,
    free_end int32 [1], two different tensors.  The outputs are allocated unless given.
    Returns a ``CachePlan`` of cu_seqlens [n + 1], kv_lens [n], slot_map and positions
    [max_tokens]."""
    kda = _base()
    n = kda._dims(cached_lens, "cached_lens", 1)[0]
    rows, stride = kda._dims(block_table, "block_table", 2)
    n_free = kda._dims(free_blocks, "free_blocks", 1)[0]
    i32, T = torch.int32, int(max_tokens)
    if T < 0:
        raise ValueError(f"max_tokens must be >= 0 (got {T})")
    a = CachePlanArgs()
    a.cached_lens = kda._dev(cached_lens, "cached_lens", i32, (n,))
    dev = cached_lens.device
    a.new_lens = kda._dev(new_lens, "new_lens", i32, (n,), dev)
    a.block_table = kda._dev(block_table, "block_table", i32, (n, stride), dev)
    a.free_blocks = kda._dev(free_blocks, "free_blocks", i32, (n_free,), dev)
    a.free_begin = kda._dev(free_begin, "free_begin", i32, (1,), dev)
    a.free_end = kda._dev(free_end, "free_end", i32, (1,), dev)
    with _on(stream, dev):
        def out(x, size):
            return torch.empty(size, dtype=i32, device=dev) if x is None else x
        plan = CachePlan(out(cu_seqlens, n + 1), out(kv_lens, n), out(slot_map, T), out(positions, T))
        a.cu_seqlens = kda._dev(plan.cu_seqlens, "cu_seqlens", i32, (n + 1,), dev)
        a.kv_lens = kda._dev(plan.kv_lens, "kv_lens", i32, (n,), dev)
        a.slot_map = kda._dev(plan.slot_map, "slot_map", i32, (T,), dev)
        a.positions = kda._dev(plan.positions, "positions", i32, (T,), dev)
        a.n_seqs, a.block_size, a.table_stride, a.n_free = n, int(block_size), stride, n_free
        a.n_blocks, a.max_tokens = int(n_blocks), T
        kda_cache_plan(a, stream)
    return plan


def kda_cache_append(k, v, slot_map, k_cache, v_cache, stream=None):
    """k_cache[slot] = k[t], v_cache[slot] = v[t] with slot = slot_map[t] (-1 skips the token).
    k, v [T, H_kv, d]; slot_map int32 [T]; caches [n_blocks, H_kv, block_size, d]."""
    kda = _base()
    T, H, d = kda._dims(k, "k", 3)
    kp, ks = _tokens(k, "k", _FLOATS, H, d, None)
    dev = k.device
    vp, vs = _tokens(v, "v", k.dtype, H, d, dev, T)
    sp = kda._dev(slot_map, "slot_map", torch.int32, (T,), dev)
    kc, vc, n_blocks, bs = _cache(kda, k_cache, v_cache, k.dtype, H, d, dev)
    kda._check(kda.load().kda_cache_append(T, H, d, kda._dtype_code(k), kp, ks, vp, vs, sp, kc, vc, n_blocks, bs,
                                           kda._stream_handle(stream)))


def kda_attn_prefill(args: AttnPrefillArgs, stream=None):
    kda = _base()
    kda._check(kda.load().kda_attn_prefill(ctypes.byref(args), kda._stream_handle(stream)))


def _outputs(kda, a, q, o, lse, want_lse, dev):
    T, H, d = q.shape
    if o is None:
        o = torch.empty((T, H, d), dtype=q.dtype, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    a.o, a.o_stride = _tokens(o, "o", q.dtype, H, d, dev, T)
    a.lse = kda._opt_dev(lse, "lse", dtype=torch.float32, shape=(T, H), device=dev)
    return o, lse


def _prefill(kda, a, q, cu_seqlens, H_kv, scale, o, lse, want_lse, stream, dev):
    T, H, d = q.shape
    n = kda._dims(cu_seqlens, "cu_seqlens", 1)[0] - 1
    a.cu_seqlens = kda._dev(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    a.n_seqs, a.n_heads, a.n_kv_heads, a.d = n, H, H_kv, d
    a.dtype, a.total_tokens = kda._dtype_code(q), T
    a.scale = float(d ** -0.5 if scale is None else scale)
    with _on(stream, dev):
        o, lse = _outputs(kda, a, q, o, lse, want_lse, dev)
        kda_attn_prefill(a, stream)
    return o, lse


def attn_prefill(q, k, v, cu_seqlens, *, scale=None, o=None, lse=None, want_lse=False, stream=None):
    """Causal attention over packed prompts (``kda_attn_prefill``): q [T, H, d]; k, v
    [T, H_kv, d]; cu_seqlens int32 [n + 1].  scale defaults to d^-0.5; o and lse are allocated
    unless given (tokens past cu_seqlens[n] are left unwritten).  Returns (o, lse or None)."""
    kda = _base()
    T, H, d = kda._dims(q, "q", 3)
    H_kv = kda._dims(k, "k", 3)[1]
    a = AttnPrefillArgs()
    a.q, a.q_stride = _tokens(q, "q", _FLOATS, H, d, None)
    dev = q.device
    a.k, a.k_stride = _tokens(k, "k", q.dtype, H_kv, d, dev, T)
    a.v, a.v_stride = _tokens(v, "v", q.dtype, H_kv, d, dev, T)
    return _prefill(kda, a, q, cu_seqlens, H_kv, scale, o, lse, want_lse, stream, dev)


def attn_prefill_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, *, scale=None, o=None, lse=None,
                       want_lse=False, stream=None):
    """``attn_prefill`` with all keys and values in the paged cache: sequence s holds kv_lens[s]
    positions, the last of which are its queries.  caches [n_blocks, H_kv, block_size, d];
    block_table int32 [n, stride]; kv_lens int32 [n].  Returns (o, lse or None)."""
    kda = _base()
    T, H, d = kda._dims(q, "q", 3)
    H_kv = kda._dims(k_cache, "k_cache", 4)[1]
    n, stride = kda._dims(block_table, "block_table", 2)
    a = AttnPrefillArgs()
    a.q, a.q_stride = _tokens(q, "q", _FLOATS, H, d, None)
    dev = q.device
    a.k_cache, a.v_cache, a.n_blocks, a.block_size = _cache(kda, k_cache, v_cache, q.dtype, H_kv, d, dev)
    a.block_table = kda._dev(block_table, "block_table", torch.int32, (n, stride), dev)
    a.kv_lens = kda._dev(kv_lens, "kv_lens", torch.int32, (n,), dev)
    if kda._dims(cu_seqlens, "cu_seqlens", 1)[0] != n + 1:
        raise ValueError(f"cu_seqlens must have {n + 1} entries (got {cu_seqlens.shape[0]})")
    a.table_stride = stride
    if n == 0:
        a.block_table = a.kv_lens = None
        a.k_stride = a.v_stride = H_kv * d
    return _prefill(kda, a, q, cu_seqlens, H_kv, scale, o, lse, want_lse, stream, dev)


def kda_attn_decode_workspace_size(args: AttnDecodeArgs) -> int:
    return int(_base().load().kda_attn_decode_workspace_size(ctypes.byref(args)))


def kda_attn_decode(args: AttnDecodeArgs, stream=None):
    kda = _base()
    kda._check(kda.load().kda_attn_decode(ctypes.byref(args), kda._stream_handle(stream)))


def attn_decode(q, k_cache, v_cache, block_table, kv_lens, *, group_start=None, prefix_lens=None, scale=None, o=None,
                lse=None, want_lse=False, workspace=None, stream=None):
    """Decode attention over the paged cache (``kda_attn_decode``): one query per sequence,
    q [n, H, d], over its kv_lens[s] positions.  group_start int32 [g + 1] and prefix_lens
    int32 [g] name the groups of consecutive sequences that share their first blocks; those
    are read once per group.  workspace: uint8, allocated unless a large enough one is given.
    Returns (o, lse or None)."""
    kda = _base()
    n, H, d = kda._dims(q, "q", 3)
    H_kv = kda._dims(k_cache, "k_cache", 4)[1]
    stride = kda._dims(block_table, "block_table", 2)[1]
    if (group_start is None) != (prefix_lens is None):
        raise ValueError("group_start and prefix_lens come together")
    a = AttnDecodeArgs()
    a.q, a.q_stride = _tokens(q, "q", _FLOATS, H, d, None)
    dev = q.device
    a.k_cache, a.v_cache, a.n_blocks, a.block_size = _cache(kda, k_cache, v_cache, q.dtype, H_kv, d, dev)
    a.block_table = kda._dev(block_table, "block_table", torch.int32, (n, stride), dev)
    a.kv_lens = kda._dev(kv_lens, "kv_lens", torch.int32, (n,), dev)
    a.n_groups = 0
    if group_start is not None:
        a.n_groups = kda._dims(prefix_lens, "prefix_lens", 1)[0]
        a.group_start = kda._dev(group_start, "group_start", torch.int32, (a.n_groups + 1,), dev)
        a.prefix_lens = kda._dev(prefix_lens, "prefix_lens", torch.int32, (a.n_groups,), dev)
    a.n_seqs, a.n_heads, a.n_kv_heads, a.d = n, H, H_kv, d
    a.dtype, a.table_stride = kda._dtype_code(q), stride
    a.scale = float(d ** -0.5 if scale is None else scale)
    with _on(stream, dev):
        o, lse = _outputs(kda, a, q, o, lse, want_lse, dev)
        need = kda_attn_decode_workspace_size(a)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None:
            a.workspace = kda._dev(workspace, "workspace", device=dev)
            a.workspace_bytes = workspace.numel() * workspace.element_size()
        kda_attn_decode(a, stream)
    return o, lse
