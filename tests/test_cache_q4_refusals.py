"""What the 4-bit cache's calls refuse, without a GPU, and their oracle."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import build as kbuild
from oracle import cache_q4 as oq

P = 0x10000000
M = 1 << 20
INV, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _cache(c):
    c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.n_blocks, c.block_size = P + 20 * M, P + 21 * M, P + 22 * M, P + 23 * M, 8, 16


def _set(a, over):
    for key, x in over.items():
        setattr(a.cache if key in dict(kda.CacheQ4._fields_) and not hasattr(type(a), key) else a, key, x)
    return a


def _append(**over):
    a = kda.CacheAppendQ4Args()
    a.n_tokens, a.n_kv_heads, a.d, a.dtype = 4, 2, 128, kda.KDA_BF16
    a.k_stride = a.v_stride = a.k_out_stride = a.v_out_stride = 256
    a.k, a.v, a.k_out, a.v_out, a.slot_map = (P + i * M for i in range(5))
    _cache(a.cache)
    return _set(a, over)


def _unpack(**over):
    a = kda.CacheUnpackQ4Args()
    a.n_seqs, a.n_kv_heads, a.d, a.dtype, a.table_stride, a.to_stride = 3, 2, 128, kda.KDA_BF16, 4, 5
    a.block_table, a.to_table, a.first, a.kv_lens, a.k_cache, a.v_cache = (P + i * M for i in range(6))
    _cache(a.cache)
    a.n_blocks = 8
    return _set(a, over)


def _decode(groups=0, cache=(), **over):
    a = kda.AttnDecodeQ4Args()
    b = a.base
    b.n_seqs, b.n_heads, b.n_kv_heads, b.d, b.dtype, b.scale = 3, 4, 2, 64, kda.KDA_FP32, 0.1
    b.q_stride, b.o_stride, b.block_size, b.table_stride, b.n_groups = 256, 256, 16, 4, groups
    names = ["q", "o", "block_table", "kv_lens", "workspace"] + (["k_cache", "v_cache", "group_start", "prefix_lens"] if groups else [])
    for name in names:
        setattr(b, name, P)
    b.n_blocks = 8 if groups else 0
    _cache(a.cache)
    b.workspace_bytes = kda.kda_attn_decode_q4_workspace_size(a)
    for key, x in over.items():
        setattr(b, key, x)
    for key, x in dict(cache).items():
        setattr(a.cache, key, x)
    return a


def test_struct_sizes(lib):
    assert ctypes.sizeof(kda.CacheQ4) == 8 * 5 + 4 * 2
    assert ctypes.sizeof(kda.CacheAppendQ4Args) == 8 + 4 * 4 + 8 * 9 + 48
    assert ctypes.sizeof(kda.CacheUnpackQ4Args) == 4 * 4 + 48 + 8 * 2 + 4 * 2 + 8 * 5
    assert ctypes.sizeof(kda.AttnDecodeQ4Args) == ctypes.sizeof(kda.AttnDecodeArgs) + 48


def test_null_argument_blocks(lib):
    for fn in (lib.kda_cache_append_q4, lib.kda_cache_unpack_q4, lib.kda_attn_decode_q4):
        assert fn(None, None) == INV
    assert lib.kda_attn_decode_q4_workspace_size(None) == 0


CACHE = [(dict(block_size=24), UNS), (dict(reserved0=0, k_codes=0), INV), (dict(k_scales=P + 8), INV), (dict(v_codes=P + 20 * M + 4), INV),
         (dict(v_scales=0), INV)]


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(n_tokens=-1), INV), (dict(n_tokens=1 << 31), INV), (dict(n_kv_heads=0), INV), (dict(d=96), UNS), (dict(dtype=5), UNS),
    (dict(k_stride=128), INV), (dict(v_stride=260), INV), (dict(k_out_stride=252), INV), (dict(v_out_stride=128), INV), (dict(k=0), INV),
    (dict(v=P + 8), INV), (dict(slot_map=0), INV), (dict(slot_map=P + 2), INV), (dict(k_out=P + 3), INV), (dict(n_blocks=0), INV),
    (dict(n_blocks=1 << 27), INV), (dict(k_out=P + 256), INV), (dict(k_out=P + M), INV), (dict(v_out=P), INV), (dict(v_out=P + 2 * M), INV),
    (dict(k_out=P + 4 * M - 256), INV), (dict(k=P + 20 * M), INV), (dict(v_out=P + 23 * M), INV), (dict(slot_map=P + 22 * M), INV),
    (dict(k_codes=P + 22 * M), INV), (dict(k_scales=P + 20 * M), INV), (dict(n_tokens=0, k=0, v=0, k_codes=0), OK),
])
def test_append_refuses(lib, over, status):
    assert lib.kda_cache_append_q4(ctypes.byref(_append(**over)), None) == status


def test_append_refuses_reserved(lib):
    a = _append()
    a.reserved0 = 1
    assert lib.kda_cache_append_q4(ctypes.byref(a), None) == INV
    a = _append()
    a.cache.reserved0 = 1
    assert lib.kda_cache_append_q4(ctypes.byref(a), None) == INV


@pytest.mark.parametrize("over,status", [
    (dict(block_size=24), UNS), (dict(k_codes=0), INV), (dict(v_scales=P + 4), INV), (dict(n_seqs=-1), INV), (dict(n_kv_heads=0), INV),
    (dict(d=32), UNS), (dict(dtype=2), UNS), (dict(table_stride=0), INV), (dict(to_stride=1 << 28), INV), (dict(n_blocks=0), INV),
    (dict(block_table=0), INV), (dict(to_table=P + 2), INV), (dict(first=P + 1), INV), (dict(kv_lens=0), INV), (dict(k_cache=P + 8), INV),
    (dict(v_cache=0), INV), (dict(k_cache=P + 5 * M), INV), (dict(k_cache=P), INV), (dict(v_cache=P + M), INV), (dict(k_cache=P + 21 * M), INV),
    (dict(v_cache=P + 2 * M), INV), (dict(k_cache=P + 3 * M), INV), (dict(n_seqs=0, k_cache=0, block_table=0, k_codes=0), OK),
])
def test_unpack_refuses(lib, over, status):
    assert lib.kda_cache_unpack_q4(ctypes.byref(_unpack(**over)), None) == status


@pytest.mark.parametrize("groups,over,cache,status", [
    (0, dict(n_heads=3), (), INV), (0, dict(d=32), (), UNS), (0, dict(dtype=-1), (), UNS), (0, dict(scale=float("inf")), (), INV),
    (0, dict(q=0), (), INV), (0, dict(o=P + 8), (), INV), (0, dict(block_table=0), (), INV), (0, dict(kv_lens=P + 1), (), INV),
    (0, dict(q_stride=128), (), INV), (0, dict(workspace=0), (), INV), (0, dict(workspace=P + 128), (), INV), (0, dict(workspace_bytes=64), (), INV),
    (0, dict(reserved0=1), (), INV), (0, dict(block_size=32), (), INV), (0, {}, dict(block_size=32), INV), (0, {}, dict(k_codes=0), INV),
    (0, {}, dict(n_blocks=0), INV), (0, {}, dict(v_scales=P + 8), INV), (0, {}, dict(reserved0=2), INV),
    (1, dict(k_cache=0), (), INV), (1, dict(v_cache=P + 8), (), INV), (1, dict(n_blocks=0), (), INV), (1, dict(group_start=0), (), INV),
    (1, dict(prefix_lens=0), (), INV), (1, dict(n_groups=-1), (), INV), (0, dict(n_seqs=0, q=0), dict(k_codes=0), OK),
])
def test_decode_refuses(lib, groups, over, cache, status):
    assert lib.kda_attn_decode_q4(ctypes.byref(_decode(groups, cache, **over)), None) == status


def test_workspace_sizes(lib):
    assert kda.kda_attn_decode_q4_workspace_size(_decode(n_seqs=0)) == 0 and kda.kda_attn_decode_q4_workspace_size(_decode(d=96)) == 0
    some = kda.kda_attn_decode_q4_workspace_size(_decode())
    assert 0 < some < kda.kda_attn_decode_q4_workspace_size(_decode(1)) and some % 256 == 0


def test_binding_refuses(lib):
    k, i = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    c = kda.q4_cache(2, 2, 16, 64, "cpu")
    assert [tuple(t.shape) for t in c] == [(2, 2, 16, 32), (2, 2, 16, 1, 2)] * 2
    with pytest.raises(ValueError, match="multiple of 64"):
        kda.q4_cache(2, 2, 16, 96, "cpu")
    with pytest.raises(ValueError, match="CUDA device"):
        kda.cache_append_q4(k, k, i, c)
    wide = torch.zeros(2, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.cache_unpack_q4(c, i[None], i[:1], wide, wide, i[None])
    with pytest.raises(TypeError, match="k_cache must be"):
        kda.cache_unpack_q4(c, i[None], i[:1], wide.half(), wide.half(), i[None])
    with pytest.raises(ValueError, match="come together"):
        kda.attn_decode_q4(torch.zeros(1, 2, 64), c, i[None], i[:1], group_start=i[:2], prefix_lens=i[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        kda.attn_decode_q4(torch.zeros(1, 2, 64), c, i[None], i[:1])


def test_oracle_quantizes():
    """Values are within half a step; the ends of a group's range are met as nearly as bf16 bounds allow; corners."""
    rng = np.random.RandomState(0)
    x = (rng.randn(50, 128) * np.exp(rng.randn(50, 1) * 4)).astype(np.float32)
    codes, s, m = oq.quantize(x)
    v = oq.values(codes, s, m)
    wide = np.repeat(s.astype(np.float64), 64, -1)
    assert (np.abs(v - x) <= 0.5 * wide * (1 + 2.0 ** -20)).all()
    y = x.reshape(50, 2, 64)
    assert (m <= y.min(-1)).all() and (m.astype(np.float64) + 15 * s.astype(np.float64) >= y.max(-1) * (1 - 2.0 ** -20) - 1e-30).all()
    assert np.array_equal(oq.unpacked(oq.packed(codes)), codes)
    codes, s, m = oq.quantize(np.array([[1.5] * 64, [0.0] * 64, [1.0] * 63 + [np.inf]], np.float32))
    assert (codes == 0).all() and (s == 0).all() and m[0] == 1.5 and m[1] == 0 and np.isnan(m[2])
    ties = np.array([[0.0, 15.0] + [i % 15 + 0.5 for i in range(62)]], np.float32)
    codes, s, m = oq.quantize(ties)
    assert s == 1 and m == 0 and codes[0, 2:8].tolist() == [0, 2, 2, 4, 4, 6]      # to even


def test_oracle_rounds_bf16_outwards():
    x = np.array([1.0, 1.0000001, -1.0000001, -1.0, 0.0, 3.4e38, -3.4e38, 1e-40, -1e-40], np.float32)
    down, up = oq.bf16_toward(x, False), oq.bf16_toward(x, True)
    assert (down <= x).all() and (up >= x).all() and np.isinf(up[5]) and np.isinf(down[6])
    assert down[1] == 1 and up[1] == 1 + 2.0 ** -7 and down[2] == -1 - 2.0 ** -7 and up[2] == -1
