"""What the attention side refuses, without a GPU: the C entry points' host checks and the binding's."""
import ctypes

import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import build as kbuild

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _fill(a, over, pointers):
    for p in pointers:
        setattr(a, p, P)
    for key, x in over.items():
        setattr(a, key, x)
    return a


def _plan(**over):
    a = kda.CachePlanArgs()
    a.n_seqs, a.block_size, a.table_stride, a.n_free, a.n_blocks, a.max_tokens = 2, 16, 4, 3, 8, 10
    a = _fill(a, over, ("cached_lens", "new_lens", "free_blocks", "free_begin", "block_table", "kv_lens", "cu_seqlens",
                        "slot_map", "positions"))
    if "free_end" not in over:
        a.free_end = P + 64
    return a


def _prefill(paged=False, **over):
    a = kda.AttnPrefillArgs()
    a.n_seqs, a.n_heads, a.n_kv_heads, a.d, a.dtype, a.scale = 1, 4, 2, 128, kda.KDA_BF16, 0.1
    a.total_tokens, a.q_stride, a.k_stride, a.v_stride, a.o_stride = 8, 512, 256, 256, 512
    a.n_blocks, a.block_size, a.table_stride = 8, 16, 4
    ptrs = ["q", "o", "cu_seqlens"] + (["k_cache", "v_cache", "block_table", "kv_lens"] if paged else ["k", "v"])
    return _fill(a, over, ptrs)


def _decode(**over):
    a = kda.AttnDecodeArgs()
    a.n_seqs, a.n_heads, a.n_kv_heads, a.d, a.dtype, a.scale = 3, 4, 2, 64, kda.KDA_FP32, 0.1
    a.q_stride, a.o_stride, a.n_blocks, a.block_size, a.table_stride, a.n_groups = 256, 256, 8, 16, 4, 1
    a = _fill(a, {}, ("q", "o", "k_cache", "v_cache", "block_table", "kv_lens", "group_start", "prefix_lens", "workspace"))
    a.workspace_bytes = kda.kda_attn_decode_workspace_size(a)
    return _fill(a, over, ())


INV, UNS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


def test_struct_sizes(lib):
    assert ctypes.sizeof(kda.CachePlanArgs) == 4 * 4 + 8 * 2 + 8 * 10
    assert ctypes.sizeof(kda.AttnPrefillArgs) == 4 * 6 + 8 * 5 + 8 * 10 + 8 + 4 * 2 + 8 * 2
    assert ctypes.sizeof(kda.AttnDecodeArgs) == 4 * 6 + 8 * 2 + 8 * 7 + 8 + 4 * 4 + 8 * 3 + 8


@pytest.mark.parametrize("over,status", [
    (dict(n_seqs=-1), INV), (dict(block_size=8), UNS), (dict(block_size=48), UNS), (dict(table_stride=0), INV),
    (dict(table_stride=1 << 28), INV), (dict(n_free=-1), INV), (dict(n_blocks=0), INV), (dict(n_blocks=1 << 28), INV),
    (dict(max_tokens=-1), INV), (dict(max_tokens=1 << 31), INV), (dict(free_begin=0), INV), (dict(free_end=P), INV),
    (dict(block_table=P + 2), INV), (dict(slot_map=0), INV), (dict(cu_seqlens=0), INV), (dict(cached_lens=0), INV),
])
def test_plan_refuses(lib, over, status):
    assert lib.kda_cache_plan(ctypes.byref(_plan(**over)), None) == status
    assert lib.kda_last_error()


def test_null_argument_blocks(lib):
    for fn in (lib.kda_cache_plan, lib.kda_attn_prefill, lib.kda_attn_decode):
        assert fn(None, None) == INV
    assert lib.kda_attn_decode_workspace_size(None) == 0


@pytest.mark.parametrize("args,status", [
    ((4, 0, 128, 0, P, 256, P, 256, P, P, P, 8, 16), INV), ((4, 2, 96, 0, P, 256, P, 256, P, P, P, 8, 16), UNS),
    ((4, 2, 128, 9, P, 256, P, 256, P, P, P, 8, 16), UNS), ((4, 2, 128, 0, P, 252, P, 256, P, P, P, 8, 16), INV),
    ((4, 2, 128, 0, P, 128, P, 256, P, P, P, 8, 16), INV), ((4, 2, 128, 0, P + 2, 256, P, 256, P, P, P, 8, 16), INV),
    ((4, 2, 128, 0, P, 256, P, 256, P, P, P, 8, 24), UNS), ((4, 2, 128, 0, P, 256, P, 256, P, P, P, 0, 16), INV),
    ((-1, 2, 128, 0, P, 256, P, 256, P, P, P, 8, 16), INV), ((4, 2, 128, 0, P, 256, None, 256, P, P, P, 8, 16), INV),
    ((0, 2, 128, 0, None, 256, None, 256, None, None, None, 8, 16), kda.KDA_OK),
    ((4, 2, 128, 0, P, 260, P, 256, P, P, P, 8, 16), INV),
])
def test_append_refuses(lib, args, status):
    assert lib.kda_cache_append(*args, None) == status


@pytest.mark.parametrize("paged,over,status", [
    (False, dict(n_heads=5), INV), (False, dict(n_kv_heads=0), INV), (False, dict(n_heads=258), UNS),
    (False, dict(d=96), UNS), (False, dict(dtype=3), UNS), (False, dict(scale=float("nan")), INV),
    (False, dict(scale=float("inf")), INV), (False, dict(total_tokens=-1), INV), (False, dict(total_tokens=1 << 31), INV),
    (False, dict(q_stride=508), INV), (False, dict(q_stride=516), INV), (False, dict(k_stride=128), INV),
    (False, dict(o_stride=504), INV), (False, dict(q=0), INV), (False, dict(o=P + 8), INV), (False, dict(v=0), INV),
    (False, dict(cu_seqlens=0), INV), (False, dict(lse=P + 1), INV), (False, dict(n_seqs=-1), INV),
    (True, dict(block_size=20), UNS), (True, dict(table_stride=0), INV), (True, dict(n_blocks=0), INV),
    (True, dict(n_blocks=1 << 26), INV), (True, dict(k_cache=0), INV), (True, dict(kv_lens=0), INV),
    (False, dict(n_seqs=0), kda.KDA_OK), (True, dict(total_tokens=0), kda.KDA_OK),
])
def test_prefill_refuses(lib, paged, over, status):
    assert lib.kda_attn_prefill(ctypes.byref(_prefill(paged, **over)), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(n_heads=3), INV), (dict(d=32), UNS), (dict(dtype=-1), UNS), (dict(scale=float("nan")), INV), (dict(n_seqs=-3), INV),
    (dict(n_groups=-1), INV), (dict(reserved0=1), INV), (dict(block_size=0), UNS), (dict(table_stride=-1), INV),
    (dict(n_blocks=-1), INV), (dict(q_stride=255), INV), (dict(q=0), INV), (dict(group_start=0), INV),
    (dict(prefix_lens=0), INV), (dict(workspace=0), INV), (dict(workspace=P + 16), INV), (dict(workspace_bytes=100), INV),
    (dict(n_seqs=0), kda.KDA_OK),
])
def test_decode_refuses(lib, over, status):
    assert lib.kda_attn_decode(ctypes.byref(_decode(**over)), None) == status


def test_decode_workspace(lib):
    size = kda.kda_attn_decode_workspace_size
    assert size(_decode()) > 0 and size(_decode(n_seqs=0)) == 0 and size(_decode(d=96)) == 0
    assert size(_decode(n_seqs=600)) > size(_decode(n_groups=0, n_seqs=600))


@pytest.fixture
def no_library(monkeypatch):
    def refuse():
        raise AssertionError("the binding reached the library with an unchecked tensor")
    monkeypatch.setattr(kda, "load", refuse)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_before_the_library(no_library):
    q, k = torch.zeros((6, 4, 64)), torch.zeros((6, 2, 64))
    cache = torch.zeros((3, 2, 16, 64))
    for call, msg in [
        (lambda: kda.attn_prefill(q, k, k, _i(2)), "q must be on a CUDA device"),
        (lambda: kda.attn_prefill(q[0], k, k, _i(2)), "q must have 3 dimensions"),
        (lambda: kda.attn_prefill(q.half(), k, k, _i(2)), "q must be torch.bfloat16"),
        (lambda: kda.attn_prefill(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, _i(2)), "dense within a token"),
        (lambda: kda.attn_prefill(q[:1].expand(6, 4, 64), k, k, _i(2)), "tokens overlap"),
        (lambda: kda.attn_prefill_paged(q, cache, cache, _i(1, 2), _i(1), _i(2)), "q must be on a CUDA device"),
        (lambda: kda.attn_decode(q, cache, cache, _i(6, 2), _i(6)), "q must be on a CUDA device"),
        (lambda: kda.attn_decode(q, cache, cache, _i(6, 2), _i(6), group_start=_i(2)), "come together"),
        (lambda: kda.kda_cache_append(k, k, _i(6), cache, cache), "k must be on a CUDA device"),
        (lambda: kda.cache_plan(_i(2).long(), _i(2), _i(2, 3), _i(4), _i(1), _i(1), block_size=16, n_blocks=9, max_tokens=4),
         "cached_lens must be torch.int32"),
        (lambda: kda.cache_plan(_i(2), _i(2), _i(2, 3), _i(4), _i(1), _i(1), block_size=16, n_blocks=9, max_tokens=-4),
         "max_tokens"),
        (lambda: kda.cache_plan(_i(2), _i(2), _i(2, 3), _i(4), _i(1), _i(1), block_size=16, n_blocks=9, max_tokens=4),
         "CUDA device"),
    ]:
        with pytest.raises((TypeError, ValueError), match=msg):
            call()
