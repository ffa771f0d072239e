"""The C interface of the softmax-attention side (``include/kda_attention.h``, ``kda_rope.h``,
``kda_cache_q4.h``): its argument blocks, status bits and signatures.  Without torch, so that loading the library needs none.
"""
import ctypes

KDA_DEV_NO_BLOCKS, KDA_DEV_BAD_GROUP, KDA_DEV_BAD_POSITION = 0x40, 0x80, 0x100


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
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
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


class QkRopeArgs(ctypes.Structure):
    """Mirror of ``kda_qk_rope_args``."""
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("eps", ctypes.c_float), ("reserved0", ctypes.c_int32), ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("turns", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


class CacheAppendRopeArgs(ctypes.Structure):
    """Mirror of ``kda_cache_append_rope_args``."""
    _fields_ = [
        ("qk", QkRopeArgs), ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64), ("slot_map", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("n_blocks", ctypes.c_int64),
        ("block_size", ctypes.c_int32), ("reserved0", ctypes.c_int32),
    ]


class CacheQ4(ctypes.Structure):
    """Mirror of ``kda_cache_q4``."""
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p), ("n_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
    ]


class CacheAppendQ4Args(ctypes.Structure):
    """Mirror of ``kda_cache_append_q4_args``."""
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("n_kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("reserved0", ctypes.c_int32), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("k_out_stride", ctypes.c_int64), ("v_out_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p), ("slot_map", ctypes.c_void_p),
        ("cache", CacheQ4),
    ]


class CacheUnpackQ4Args(ctypes.Structure):
    """Mirror of ``kda_cache_unpack_q4_args``."""
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("cache", CacheQ4), ("block_table", ctypes.c_void_p), ("to_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int32), ("to_stride", ctypes.c_int32), ("first", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("n_blocks", ctypes.c_int64),
    ]


class AttnDecodeQ4Args(ctypes.Structure):
    """Mirror of ``kda_attn_decode_q4_args``."""
    _fields_ = [("base", AttnDecodeArgs), ("cache", CacheQ4)]


#: The blocks' layouts for ``struct``, which fills one in a fifth of the time that ctypes takes.
PACK = {QkRopeArgs: "@q6ifi12q", CacheAppendRopeArgs: "@q6ifi12q6q2i", CacheAppendQ4Args: "@q4i4q5q5q2i",
        CacheUnpackQ4Args: "@4i5q2i2q2i5q", AttnDecodeQ4Args: "@5if2q7qq4i4q5q2i"}


def declare(lib):
    """Set the ctypes signatures of the entry points."""
    vp, i32, i64, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER
    lib.kda_cache_plan.restype = ctypes.c_int
    lib.kda_cache_plan.argtypes = [P(CachePlanArgs), vp]
    lib.kda_cache_append.restype = ctypes.c_int
    lib.kda_cache_append.argtypes = [i64, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, i64, i32, vp]
    lib.kda_attn_prefill.restype = ctypes.c_int
    lib.kda_attn_prefill.argtypes = [P(AttnPrefillArgs), vp]
    lib.kda_attn_prefill_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_prefill_workspace_size.argtypes = [P(AttnPrefillArgs)]
    lib.kda_attn_decode_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_decode_workspace_size.argtypes = [P(AttnDecodeArgs)]
    lib.kda_attn_decode.restype = ctypes.c_int
    lib.kda_attn_decode.argtypes = [P(AttnDecodeArgs), vp]
    # These take a ctypes block (byref) or the same bytes packed (``PACK``), whichever the caller has made.
    lib.kda_attn_decode_q4_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_decode_q4_workspace_size.argtypes = [vp]
    for name in ("kda_qk_norm_rope", "kda_cache_append_rope", "kda_cache_append_q4", "kda_cache_unpack_q4", "kda_attn_decode_q4"):
        entry = getattr(lib, name)
        entry.restype = ctypes.c_int
        entry.argtypes = [vp, vp]
