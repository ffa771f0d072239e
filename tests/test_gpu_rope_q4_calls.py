"""Calls of the rotation and the 4-bit cache that their documentation allows, beside the ones that compute something: empty
batches, wrong tensors on the GPU, streams, replays, two calls at once, the largest and the smallest shapes."""
import numpy as np
import pytest
import torch

import _attention as A
import _q4
from oracle import rope as orope

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_batches(kda, cuda_device, dtype):
    dev, d = cuda_device, 64
    none, some, i0 = torch.empty((0, 4, d), dtype=dtype, device=dev), torch.empty((0, 2, d), dtype=dtype, device=dev), _i32([], dev)
    before = kda.kda_launch_count()
    q, k = kda.qk_norm_rope(none, some, i0)
    assert q.shape == none.shape and k.shape == some.shape
    cache = kda.q4_cache(2, 2, 16, d, dev)
    wide = torch.zeros((2, 2, 16, d), dtype=dtype, device=dev)
    assert kda.cache_append_rope(some, some, i0, None, i0, wide, wide.clone(), q=none).shape == none.shape
    assert kda.cache_append_q4(some, some, i0, cache) == (None, None)
    kda.cache_unpack_q4(cache, torch.empty((0, 3), dtype=torch.int32, device=dev), i0, wide, wide.clone(),
                        torch.empty((0, 2), dtype=torch.int32, device=dev))
    o, lse = kda.attn_decode_q4(none, cache, torch.empty((0, 3), dtype=torch.int32, device=dev), i0, want_lse=True)
    assert o.shape == none.shape and lse.shape == (0, 4) and kda.kda_launch_count() == before


def test_no_sequence_holds_anything(kda, cuda_device):
    dev, d = cuda_device, 128
    c = _q4.Paged(1, [0] * 300, 2, d, 16, BF, dev)
    o, lse = c.decode(kda, A.randn(2, (300, 8, d), BF, dev))
    assert kda.kda_check_status() == 0 and (o == 0).all() and (lse == float("-inf")).all()


def test_only_prefixes(kda, cuda_device):
    """Requests at the moment after their shared prompt: no own token yet."""
    for dtype in (BF, F32):
        c = _q4.Paged(3, [0] * 6, 2, 64, 32, dtype, cuda_device, [(0, 4), (4, 6)], [96, 32])
        q = A.randn(4, (6, 6, 64), dtype, cuda_device)
        o, lse = c.decode(kda, q)
        assert kda.kda_check_status() == 0
        _q4.check(o, lse, q, c, 64 ** -0.5, dtype)


def test_binding_refuses(kda, cuda_device):
    dev = cuda_device
    q, k, i = torch.zeros(3, 4, 64, device=dev), torch.zeros(3, 2, 64, device=dev), _i32([0, 1, 2], dev)
    c = kda.q4_cache(2, 2, 16, 64, dev)
    wide, table = torch.zeros(2, 2, 16, 64, device=dev), _i32([[0], [1], [0]], dev)
    turns = kda.rope_turns([1.0] * 32, dev)
    before = kda.kda_launch_count()
    for error, match, call in (
            (TypeError, "k must be", lambda: kda.qk_norm_rope(q, k.bfloat16(), i)),
            (ValueError, "k must have shape", lambda: kda.qk_norm_rope(q, k[:2], i)),
            (ValueError, "k must have shape", lambda: kda.qk_norm_rope(q, torch.zeros(3, 2, 128, device=dev), i)),
            (ValueError, "positions must have shape", lambda: kda.qk_norm_rope(q, k, i[:2])),
            (TypeError, "positions must be", lambda: kda.qk_norm_rope(q, k, i.long())),
            (TypeError, "turns must be", lambda: kda.qk_norm_rope(q, k, i, turns.int())),
            (ValueError, "33 frequencies", lambda: kda.qk_norm_rope(q, k, i, kda.rope_turns([1.0] * 33, dev))),
            (kda.KdaError, "multiple of 8", lambda: kda.qk_norm_rope(q, k, i, turns[:2])),
            (TypeError, "q_weight must be", lambda: kda.qk_norm_rope(q, k, i, q_weight=torch.ones(64, dtype=BF, device=dev))),
            (ValueError, "k_weight must have shape", lambda: kda.qk_norm_rope(q, k, i, k_weight=torch.ones(32, device=dev))),
            (kda.KdaError, "eps", lambda: kda.qk_norm_rope(q, k, i, eps=-1.0)),
            (kda.KdaError, "q_weight is not 16-byte", lambda: kda.qk_norm_rope(q, k, i, q_weight=torch.ones(66, device=dev)[1:65])),
            (kda.KdaError, "q_out overlaps k", lambda: kda.qk_norm_rope(k.clone(), k, i, q_out=k)),
            (ValueError, "heads must be dense", lambda: kda.qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, i)),
            (ValueError, "v must have shape", lambda: kda.cache_append_rope(k, k[:, :1], i, turns, i, wide, wide.clone())),
            (ValueError, "v_cache must have shape", lambda: kda.cache_append_rope(k, k, i, turns, i, wide, wide[:1])),
            (kda.KdaError, "overlaps", lambda: kda.cache_append_rope(k, k, i, turns, i, wide, wide)),
            (ValueError, "k_scales must have shape", lambda: kda.cache_append_q4(k, k, i, c._replace(k_scales=c.k_scales[:, :, :8]))),
            (TypeError, "v_codes must be", lambda: kda.cache_append_q4(k, k, i, c._replace(v_codes=c.v_codes.char()))),
            (ValueError, "k_codes must have shape", lambda: kda.cache_append_q4(torch.zeros(3, 3, 64, device=dev), torch.zeros(3, 3, 64, device=dev), i, c)),
            (kda.KdaError, "k_out overlaps v", lambda: kda.cache_append_q4(k, k, i, c, k_out=k)),
            (ValueError, "block sizes differ", lambda: kda.cache_unpack_q4(c, table, i, torch.zeros(2, 2, 32, 64, device=dev), torch.zeros(2, 2, 32, 64, device=dev), table)),
            (ValueError, "to_table must have shape", lambda: kda.cache_unpack_q4(c, table, i, wide, wide.clone(), table[:2])),
            (ValueError, "first must have shape", lambda: kda.cache_unpack_q4(c, table, i, wide, wide.clone(), table, first=i[:2])),
            (kda.KdaError, "overlaps", lambda: kda.cache_unpack_q4(c, table, i, wide, wide, table)),
            (ValueError, "kv_lens must have shape", lambda: kda.attn_decode_q4(q, c, table, i[:2])),
            (ValueError, "k_prefix|k_cache", lambda: kda.attn_decode_q4(q, c, table, i, k_prefix=wide[:, :1], v_prefix=wide, group_start=i[:2], prefix_lens=i[:1])),
            (ValueError, "block sizes differ", lambda: kda.attn_decode_q4(q, c, table, i, k_prefix=torch.zeros(2, 2, 32, 64, device=dev), v_prefix=torch.zeros(2, 2, 32, 64, device=dev), group_start=i[:2], prefix_lens=i[:1]))):
        with pytest.raises(error, match=match):
            call()
    assert kda.kda_launch_count() == before


def test_two_streams_at_once(kda, cuda_device):
    """Calls in flight on two streams, each with its own workspace, change nothing of each other."""
    dev, d, H, H_kv = cuda_device, 128, 8, 2
    cases = [_q4.Paged(10 + i, [3000 + 500 * i, 7, 900], H_kv, d, 32, BF, dev) for i in range(2)]
    q = [A.randn(20 + i, (3, H, d), BF, dev) for i in range(2)]
    alone = [c.decode(kda, x) for c, x in zip(cases, q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(10):
        for c, x, s in zip(cases, q, streams):
            s.wait_stream(torch.cuda.current_stream())
            outs.append(kda.attn_decode_q4(x, c.cache, c.table, c.kv_lens, want_lse=True, stream=s))
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(lse, alone[i % 2][1])


def test_replays_of_two_graphs(kda, cuda_device):
    """Two captured graphs of decode, append and read-back, replayed in turn."""
    dev, d, H, H_kv, bs = cuda_device, 64, 4, 2, 16
    c = _q4.Paged(30, [500, 33, 64], H_kv, d, bs, BF, dev)
    wide = [torch.zeros((c.n_blocks, H_kv, bs, d), dtype=BF, device=dev) for _ in range(2)]
    q = [A.randn(31 + i, (3, H, d), BF, dev) for i in range(2)]
    want = [c.decode(kda, x) for x in q]
    graphs, got = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(kda.attn_decode_q4(x, c.cache, c.table, c.kv_lens, want_lse=True))
            kda.cache_unpack_q4(c.cache, c.table, c.kv_lens, *wide, c.table)
        graphs.append(g)
    for _ in range(3):
        for i in (0, 1, 1, 0):
            for t in got[i]:
                t.fill_(7)
            graphs[i].replay()
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
    assert kda.kda_check_status() == 0
    keys, values, _, _ = c.sequence(0)
    at = [(c.table_np[0, j // bs], j % bs) for j in range(500)]
    for cache, ref in zip(wide, (keys, values)):
        got_rows = torch.stack([cache[b, :, o] for b, o in at]).cpu()
        assert torch.equal(got_rows, torch.from_numpy(ref).to(BF))


def test_many_sequences(kda, cuda_device):
    """More sequences than a thread block scans at once, most of them tiny: each unit's beginning and end on the line."""
    dev, d, n = cuda_device, 64, 3000
    kv = (np.random.RandomState(5).randint(0, 40, n) ** 2 // 20).tolist()
    c = _q4.Paged(6, kv, 1, d, 16, BF, dev)
    q = A.randn(7, (n, 3, d), BF, dev)
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, BF, only=range(0, n, 17))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_heads_than_a_unit(kda, cuda_device, dtype):
    """128 query heads of one key/value head, long enough to be cut into pieces that are joined."""
    dev, d = cuda_device, 128
    c = _q4.Paged(8, [2100, 5], 1, d, 128, dtype, dev)
    q = A.randn(9, (2, 128, d), dtype, dev)
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, dtype)


def test_one_token_of_one_head(kda, cuda_device):
    """A single row, whatever the stride of its token says."""
    dev = cuda_device
    x = A.randn(11, (1, 64), F32, dev)
    q = x.as_strided((1, 1, 64), (3, 64, 1))
    turns = [12345678901234567890 % (1 << 64)] + [7] * 31
    a, b = kda.qk_norm_rope(q, q.clone(), _i32([2 ** 31 - 1], dev), torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], device=dev))
    assert kda.kda_check_status() == 0
    ref, spread = orope.norm_rope(A.np64(x)[None], None, 0.0, [2 ** 31 - 1], turns, False)
    assert (np.abs(A.np64(a) - ref) <= 48 * A.U * spread).all() and torch.equal(a, b)
    c = kda.q4_cache(1, 1, 16, 64, dev)
    k, v = kda.cache_append_q4(q, q, _i32([15], dev), c, want_values=True)
    o, lse = kda.attn_decode_q4(q, kda.Q4Cache(*c), _i32([[0]], dev), _i32([0], dev), want_lse=True)
    assert kda.kda_check_status() == 0 and (o == 0).all() and lse.item() == float("-inf") and torch.equal(k, v)


def test_large_queries_and_keys(kda, cuda_device):
    """Scores up to 2^27 in magnitude: weights are then one key's, whatever the distance to the next."""
    dev, d = cuda_device, 64
    for dtype in (BF, F32):
        c = _q4.Paged(12, [50], 1, d, 16, dtype, dev, std=2.0 ** 10)
        q = A.randn(13, (1, 4, d), dtype, dev, 2.0 ** 10)
        for sign in (1.0, -1.0):
            o, lse = c.decode(kda, q, scale=sign)
            assert kda.kda_check_status() == 0
            _q4.check(o, lse, q, c, sign, dtype)
