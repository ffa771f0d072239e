"""The C interface of the softmax-attention side (``include/kda_attention.h``): its argument blocks,
status bits and signatures.  Without torch, so that loading the library needs none.
"""
import ctypes

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
