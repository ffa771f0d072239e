"""What the norm and rotation calls refuse, without a GPU, and their oracle and frequencies."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import build as kbuild
from hybrid_linear_attention_kda_gb300.attention_abi import PACK
from oracle import rope as orope

P = 0x10000000
INV, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _rope(a=None, **over):
    a = kda.QkRopeArgs() if a is None else a
    a.n_tokens, a.n_heads, a.n_kv_heads, a.d, a.dtype, a.rot_dim, a.eps = 4, 4, 2, 128, kda.KDA_BF16, 64, 1e-6
    a.q_stride, a.k_stride, a.q_out_stride, a.k_out_stride = 512, 256, 512, 256
    for i, name in enumerate(("q", "k", "q_out", "k_out", "q_weight", "k_weight", "turns", "positions")):
        setattr(a, name, P + (i << 20))
    for key, x in over.items():
        setattr(a, key, x)
    return a


def _append(qk=(), **over):
    a = kda.CacheAppendRopeArgs()
    _rope(a.qk, k_out=None, k_out_stride=0)
    a.v, a.v_stride, a.slot_map, a.k_cache, a.v_cache, a.n_blocks, a.block_size = P + (8 << 20), 256, P + (9 << 20), P + (10 << 20), P + (12 << 20), 8, 16
    for key, x in dict(qk).items():
        setattr(a.qk, key, x)
    for key, x in over.items():
        setattr(a, key, x)
    return a


def test_struct_sizes(lib):
    assert ctypes.sizeof(kda.QkRopeArgs) == 8 + 4 * 8 + 8 * 4 + 8 * 8
    assert ctypes.sizeof(kda.CacheAppendRopeArgs) == ctypes.sizeof(kda.QkRopeArgs) + 8 * 6 + 4 * 2


def _leaves(block):
    """(offset, ctypes type) of a block's fields, those of blocks within it too."""
    out = []
    for name, kind in block._fields_:
        at = getattr(block, name).offset
        out += [(at + o, k) for o, k in _leaves(kind)] if issubclass(kind, ctypes.Structure) else [(at, kind)]
    return out


@pytest.mark.parametrize("block", list(PACK), ids=lambda b: b.__name__)
def test_packed_blocks_are_the_ctypes_blocks(block):
    """The binding packs its argument blocks by format: field for field at the places of the ctypes mirror."""
    pack = struct.Struct(PACK[block])
    assert pack.size == ctypes.sizeof(block)
    fields = _leaves(block)
    data = pack.pack(*[float(i + 1) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(fields)])
    for i, (at, kind) in enumerate(fields):
        assert kind.from_buffer_copy(data, at).value == i + 1, (i, kind)


SHARED = [
    (dict(n_tokens=-1), INV), (dict(n_tokens=1 << 31), INV), (dict(n_heads=-1), INV), (dict(n_heads=5000, q_stride=640000, q_out_stride=640000), UNS),
    (dict(n_kv_heads=0), INV), (dict(d=96), UNS), (dict(dtype=2), UNS), (dict(rot_dim=-8), INV), (dict(rot_dim=136), INV),
    (dict(rot_dim=20), INV), (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(interleaved=2), INV), (dict(reserved0=1), INV), (dict(q_stride=504), INV), (dict(k_stride=128), INV),
    (dict(q_out_stride=516), INV), (dict(q=0), INV), (dict(k=P + 8), INV), (dict(q_out=0), INV), (dict(q_weight=P + 4), INV),
    (dict(turns=0), INV), (dict(turns=P + 8), INV), (dict(positions=0), INV), (dict(positions=P + 2), INV),
    (dict(q_out=P + 16), INV), (dict(q_out=P, q_out_stride=1024), INV),                     # q moved within itself
    (dict(q_out=P + (1 << 20)), INV),                                                       # over k
    (dict(q_out=P + (7 << 20)), INV), (dict(q_out=P + (6 << 20) - 256), INV),               # over positions, turns
    (dict(n_tokens=0, q=0, k=0), OK),
]


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(n_heads=0), INV), (dict(k_out=0), INV), (dict(k_out_stride=128), INV), (dict(k_out=P), INV),
    (dict(k_out=P + (2 << 20)), INV), (dict(k_out=P + (5 << 20)), INV),
    # views of one projection's output: beside each other, but one of them a head further on than it may be
    (dict(q_stride=1024, k_stride=1024, q_out_stride=1024, k_out_stride=1024, q_out=P, k=P + 1024, k_out=P + 512), INV),
])
def test_norm_rope_refuses(lib, over, status):
    assert lib.kda_qk_norm_rope(ctypes.byref(_rope(**over)), None) == status
    assert status == OK or lib.kda_last_error()


@pytest.mark.parametrize("over,status", SHARED)
def test_append_refuses_what_the_rotation_refuses(lib, over, status):
    assert lib.kda_cache_append_rope(ctypes.byref(_append(qk=over)), None) == status


@pytest.mark.parametrize("qk,over,status", [
    ((), dict(v=0), INV), ((), dict(v_stride=128), INV), ((), dict(slot_map=0), INV), ((), dict(k_cache=P + 8), INV),
    ((), dict(v_cache=0), INV), ((), dict(n_blocks=0), INV), ((), dict(block_size=24), UNS), ((), dict(reserved0=3), INV),
    ((), dict(k_cache=P + (12 << 20) + 256), INV), ((), dict(k_cache=P + (1 << 20)), INV), ((), dict(v_cache=P + (8 << 20)), INV),
    ((), dict(v_cache=P + (9 << 20)), INV), (dict(q_out=P + (8 << 20)), (), INV), (dict(q_out=P + (10 << 20)), (), INV),
    (dict(n_heads=0), (), INV), (dict(n_heads=0, q=0, q_out=0), (), INV),
])
def test_append_refuses(lib, qk, over, status):
    assert lib.kda_cache_append_rope(ctypes.byref(_append(qk, **dict(over))), None) == status


def test_null_argument_blocks(lib):
    assert lib.kda_qk_norm_rope(None, None) == INV and lib.kda_cache_append_rope(None, None) == INV


def test_binding_refuses(lib):
    q, k, pos = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.qk_norm_rope(q, k, pos)
    with pytest.raises(ValueError, match="dimensions"):
        kda.qk_norm_rope(q[0], k, pos)
    with pytest.raises(TypeError, match="bfloat16"):
        kda.qk_norm_rope(q.half(), k, pos)
    cache = torch.zeros(2, 2, 16, 64)
    with pytest.raises(ValueError, match="come with q"):
        kda.cache_append_rope(k, k, pos, None, pos, cache, cache, q_out=q)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.cache_append_rope(k, k, pos, None, pos, cache, cache)


def test_turns():
    """F = round(f / 2 pi 2^64) modulo 2^64, to the last bits, with negative and fast frequencies."""
    f = [1.0, 1e-4, 0.5, -1.0, 2 * math.pi, 100.0, 0.0]
    t = kda.rope_turns(f, device="cpu")
    assert t.dtype == torch.int64 and t[-1] == 0
    assert t[0] == 0x28BE60DB9391054A                       # the first bits of 1 / 2 pi
    assert int(t[0]) + int(t[3]) == 0
    assert abs(int(t[2]) * 2 - int(t[0])) <= 1
    got = orope.angles([1, 7, 1 << 20], t.tolist())
    want = np.array([1, 7, 1 << 20])[:, None] * np.array(f)
    assert np.abs(np.exp(1j * got) - np.exp(1j * want)).max() < 1e-7     # float64's own error at 100 * 2^20
    assert torch.equal(kda.rope_turns(torch.tensor(f, dtype=torch.float64)), t)
    with pytest.raises(ValueError, match="finite"):
        kda.rope_turns([float("nan")], device="cpu")


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotates(interleaved):
    """Scores of rotated vectors depend on the distance of their positions alone, and lengths stay."""
    rng = np.random.RandomState(0)
    x, y = rng.randn(1, 1, 64), rng.randn(1, 1, 64)
    turns = [int(t) for t in rng.randint(0, 1 << 60, 32)]
    score = [(orope.norm_rope(x, None, 0.0, [p], turns, interleaved)[0] * orope.norm_rope(y, None, 0.0, [p + 5], turns, interleaved)[0]).sum()
             for p in (0, 3, 1 << 20)]
    assert np.allclose(score, score[0], rtol=0, atol=1e-12)
    z = orope.norm_rope(x, np.ones(64), 0.0, [9], turns, interleaved)[0]
    assert abs((z * z).mean() - 1) < 1e-12
