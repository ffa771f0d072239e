"""Decode attention over the 4-bit cache, alone and behind full-width shared prefixes, against the float64 reference.  The
bounds are derived in ``_q4``."""
import numpy as np
import pytest
import torch

import _attention as A
import _q4

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 8, 2, 16), (64, 4, 4, 32), (64, 5, 1, 16), (128, 9, 1, 64), (128, 24, 1, 128),
                                         (64, 128, 1, 256), (64, 51, 3, 16), (128, 16, 2, 16)])
def test_plain_decode(kda, cuda_device, dtype, d, H, H_kv, bs):
    kv = [1, 15, 16, 17, 0, 63, 64, 65, 200, 333]
    c = _q4.Paged(1, kv, H_kv, d, bs, dtype, cuda_device)
    q = A.randn(2, (len(kv), H, d), dtype, cuda_device)
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 8, 2, 16), (64, 3, 3, 32), (128, 100, 1, 16), (64, 16, 8, 64)])
def test_shared_prefixes(kda, cuda_device, dtype, d, H, H_kv, bs):
    """Groups of many and of one, a prefix of zero, suffixes of zero and more."""
    groups, prefix = [(0, 40), (40, 42), (42, 43), (43, 50)], [2 * bs, 0, 5 * bs, bs]
    own = np.random.RandomState(3).randint(0, 70, 50).tolist()
    own[0] = own[45] = 0
    c = _q4.Paged(4, own, H_kv, d, bs, dtype, cuda_device, groups, prefix)
    q = A.randn(5, (50, H, d), dtype, cuda_device)
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_views_and_scales(kda, cuda_device, dtype, scale):
    """q and o as views, scales of both signs, more table columns than needed."""
    dev, d, H, H_kv = cuda_device, 64, 6, 2
    c = _q4.Paged(6, [70, 3, 129], H_kv, d, 32, dtype, dev, stride=9, std=2.0)
    x, y = A.randn(7, (3, 3 * H, d), dtype, dev), torch.zeros((3, H + 2, d), dtype=dtype, device=dev)
    q, o, lse = x[:, H:2 * H], y[:, 1:-1], torch.zeros((3, H), device=dev)
    got, got_lse = c.decode(kda, q, scale=scale, o=o, lse=lse)
    assert kda.kda_check_status() == 0 and got is o and got_lse is lse
    _q4.check(o, lse, q, c, scale, dtype)
    assert not y[:, 0].any() and not y[:, -1].any()
    again, none = c.decode(kda, q, scale=scale, want_lse=False)
    assert none is None and torch.equal(again, o)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,H_kv,d", [(8, 2, 128), (4, 1, 64), (16, 1, 128)])
def test_split_over_workers(kda, cuda_device, dtype, H, H_kv, d):
    """Sequences cut into many pieces and joined; results do not depend on the workspace's bytes or on the run."""
    dev, n = cuda_device, 3
    c = _q4.Paged(8, [5001, 1, 2300], H_kv, d, 64, dtype, dev)
    q = A.randn(9, (n, H, d), dtype, dev, 2.0)
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, dtype)
    for byte in (0, 0xFF):
        ws = torch.full((64 << 20,), byte, dtype=torch.uint8, device=dev)
        o2, lse2 = c.decode(kda, q, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_hidden_slots_hold_anything(kda, cuda_device, dtype):
    """Unowned slots have NaN scales throughout (the fixture's fill); infinities and other codes change nothing either."""
    kv, d = [5, 70, 129], 64
    c = _q4.Paged(10, kv, 2, d, 32, dtype, cuda_device)
    q = A.randn(11, (3, 4, d), dtype, cuda_device)
    a, la = c.decode(kda, q)
    for t in (c.cache.k_scales, c.cache.v_scales):
        t[torch.isnan(t)] = float("inf")
    b, lb = c.decode(kda, q)
    assert torch.equal(a, b) and torch.equal(la, lb)
    _q4.check(a, la, q, c, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_seen_nan_stays_where_it_is(kda, cuda_device, dtype):
    """A value group that is NaN makes its channels of its heads NaN, a key group the heads' whole rows; nothing else."""
    kv, d, H, H_kv = [40, 90], 128, 4, 2
    c = _q4.Paged(12, kv, H_kv, d, 16, dtype, cuda_device)
    q = A.randn(13, (2, H, d), dtype, cuda_device)
    a, la = c.decode(kda, q)
    c.m[1, c.table_np[1, 2], 1, 3, 1] = np.nan              # values of sequence 1, head 1, position 35, channels 64 ..
    c.upload()
    b, lb = c.decode(kda, q)
    hit = torch.zeros_like(a, dtype=torch.bool)
    hit[1, 2:, 64:] = True
    assert torch.isnan(b[hit]).all() and torch.equal(b[~hit], a[~hit]) and torch.equal(la, lb)
    c.m[0, c.table_np[0, 0], 0, 0, 0] = np.nan              # keys of sequence 0, head 0
    c.upload()
    b, lb = c.decode(kda, q)
    hit[0, :2] = True
    assert torch.isnan(b[hit]).all() and torch.equal(b[~hit], a[~hit]) and torch.isnan(lb[0, :2]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_of_very_different_sizes(kda, cuda_device, dtype):
    """Attention on one position with tiny values among others with huge ones, and heads of tiny and huge queries."""
    kv, d, H = [100], 64, 4
    c = _q4.Paged(14, kv, 1, d, 16, dtype, cuda_device)
    q = A.randn(15, (1, H, d), dtype, cuda_device)
    q[0, 1] *= 2.0 ** -70
    q[0, 2] *= 2.0 ** 20
    c.s[1], c.m[1] = c.s[1] * np.float32(2.0 ** 40), c.m[1] * np.float32(2.0 ** 40)
    best = int(np.argmax(c.sequence(0)[0][:, 0] @ A.np64(q)[0, 2]))
    at = (1, c.table_np[0, best // 16], 0, best % 16)
    c.s[at], c.m[at] = c.s[at] * np.float32(2.0 ** -80), c.m[at] * np.float32(2.0 ** -80)
    c.upload()
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == 0
    assert A.np64(o)[0, 2].any() and np.abs(A.np64(o)[0, 2]).max() < 1e-9
    keys, values, key_size, value_size = c.sequence(0)
    ref, ref_lse, spread = _q4.attention(A.np64(q)[0], keys, values, value_size, d ** -0.5)
    # all other weights of head 2 are below 2^-1000: what is left is one position's value
    assert (np.abs(A.np64(o)[0, 2] - ref[2]) <= 2.0 ** -7 * spread[2]).all()
    f = 2.0 ** -7 + 1e-3                                     # scores are of order one: e < 2^-11
    for h in (0, 1, 3):
        assert (np.abs(A.np64(o)[0, h] - ref[h]) <= f * spread[h]).all()


def test_offsets_past_32_bits(kda, cuda_device):
    """A cache whose codes pass 2^32 bytes, with the blocks at its far end in use."""
    dev, H_kv, bs, d = cuda_device, 8, 256, 128
    n_blocks = (1 << 33) // (H_kv * bs * d) + 9
    c = kda.q4_cache(n_blocks, H_kv, bs, d, dev)
    kv, n = [700, 300], 2
    table = _i32([[n_blocks - 1, 3, n_blocks - 7], [n_blocks // 2 + 9, n_blocks - 2, -1]], dev)
    k, v = A.randn(16, (1000, H_kv, d), BF, dev), A.randn(17, (1000, H_kv, d), BF, dev)
    slots = [int(table[s, j // bs]) * bs + j % bs for s in range(n) for j in range(kv[s])]
    kda.cache_append_q4(k, v, _i32(slots, dev), c)
    q = A.randn(18, (n, 16, d), BF, dev)
    o, lse = kda.attn_decode_q4(q, c, table, _i32(kv, dev), want_lse=True)
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, _q4.Packed(k, v, kv), d ** -0.5, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_lengths_groups_and_blocks_are_flagged(kda, cuda_device, dtype):
    own, d, dev = [24, 34, 17, 4], 64, cuda_device
    q = A.randn(20, (4, 4, d), dtype, dev)
    c = _q4.Paged(21, own, 2, d, 16, dtype, dev)
    c.kv_lens[1], c.kv_lens[3] = 16 * c.table.shape[1] + 1, -2
    o, lse = c.decode(kda, q)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    assert (o[[1, 3]] == 0).all() and (lse[[1, 3]] == float("-inf")).all()
    _q4.check(o, lse, q, c, d ** -0.5, dtype, only=(0, 2))
    for start, prefix in (([0, 4], [17]), ([0, 4], [-16]), ([0, 3], [16]), ([1, 4], [16]), ([0, 9], [16]), ([0, 4], [64])):
        g = _q4.Paged(21, own, 2, d, 16, dtype, dev, [(0, 4)], [16])
        g.group_start, g.prefix_lens = _i32(start, dev), _i32(prefix, dev)
        g.decode(kda, q)
        assert kda.kda_check_status() & kda.KDA_DEV_BAD_GROUP, (start, prefix)
    bad = _q4.Paged(21, own, 2, d, 16, dtype, dev)
    bad.table[2, 1] = bad.n_blocks
    o, lse = bad.decode(kda, q)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    _q4.check(o, lse, q, bad, d ** -0.5, dtype, only=(0, 1, 3))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_in_a_graph_on_another_stream(kda, cuda_device, dtype):
    """A serving step on a 4-bit cache (plan, norm and rotation in place, append, attention), captured once and replayed
    over changing lengths, against the reference on what the cache then holds."""
    dev, d, H, H_kv, bs, n = cuda_device, 64, 4, 2, 16, 5
    lens = [0, 15, 16, 40, 7]
    c = _q4.Paged(22, lens, H_kv, d, bs, dtype, dev, extra=40, stride=6)
    used = int((c.table_np >= 0).sum())
    free = torch.tensor([b for b in range(c.n_blocks) if b not in set(c.table_np[c.table_np >= 0].tolist())], dtype=torch.int32, device=dev)
    assert free.numel() == c.n_blocks - used
    cached, new = _i32(lens, dev), _i32([1] * n, dev)
    cur = [_i32([0], dev), _i32([0], dev)]
    qkv = torch.zeros((n, H + 2 * H_kv, d), dtype=dtype, device=dev)
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    turns = kda.rope_turns([10000.0 ** (-2 * i / d) for i in range(d // 2)], device=dev)
    w = 1 + A.randn(23, (d,), F32, dev, 0.2)
    o, lse = torch.zeros((n, H, d), dtype=dtype, device=dev), torch.zeros((n, H), device=dev)
    side = torch.cuda.Stream()

    def step(stream=None):
        p = kda.cache_plan(cached, new, c.table, free, cur[0], cur[1], block_size=bs, n_blocks=c.n_blocks, max_tokens=n, stream=stream)
        kda.qk_norm_rope(q, k, p.positions, turns, q_weight=w, k_weight=w, q_out=q, k_out=k, stream=stream)
        kda.cache_append_q4(k, v, p.slot_map, c.cache, stream=stream)
        kda.attn_decode_q4(q, c.cache, c.table, p.kv_lens, o=o, lse=lse, stream=stream)
        return p

    step(side)                                                  # loads the kernels before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p = step()
    for i in range(20):
        qkv.copy_(A.randn(30 + i, qkv.shape, dtype, dev))
        graph.replay()
        lens = [x + 1 for x in lens]
        assert p.kv_lens.tolist() == lens
        cached.copy_(p.kv_lens)
        cur[0].copy_(cur[1])
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    c.kv, c.table_np = lens, c.table.cpu().numpy()
    from oracle import cache_q4 as oq
    c.codes = np.stack([oq.unpacked(t.cpu().numpy()) for t in (c.cache.k_codes, c.cache.v_codes)])
    scales = np.stack([t.float().cpu().numpy() for t in (c.cache.k_scales, c.cache.v_scales)])
    c.s, c.m = scales[..., 0], scales[..., 1]
    _q4.check(o, lse, q, c, d ** -0.5, dtype)                   # q was rotated in place
