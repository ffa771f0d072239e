"""Decode attention over the paged cache, alone and behind shared prefixes, against the float64
reference.  The bounds are derived in ``_attention``."""
import numpy as np
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _decode(kda, q, c, groups=None, prefix=None, **kw):
    dev = q.device
    kw.setdefault("want_lse", True)
    o, lse = kda.attn_decode(q, c.k, c.v, c.table, c.kv_lens, group_start=None if groups is None else _i32(groups, dev),
                             prefix_lens=None if groups is None else _i32(prefix, dev), **kw)
    torch.cuda.synchronize()
    return o, lse


def _check(o, lse, q, c, scale, dtype):
    keys, values = c.keys_values()
    n = len(c.kv)
    A.check(o, lse, A.split(q, [1] * n), keys, values, [k - 1 for k in c.kv], scale, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 8, 2, 16), (64, 4, 4, 32), (64, 5, 1, 16), (128, 9, 1, 64), (128, 24, 1, 128),
                                         (64, 128, 1, 256), (64, 51, 3, 16)])
def test_plain_decode(kda, cuda_device, dtype, d, H, H_kv, bs):
    kv = [1, 15, 16, 17, 0, 63, 64, 65, 200, 333]
    c = A.Paged(1, kv, H_kv, d, bs, dtype, cuda_device)
    q = A.randn(2, (len(kv), H, d), dtype, cuda_device)
    o, lse = _decode(kda, q, c)
    assert kda.kda_check_status() == 0
    _check(o, lse, q, c, d ** -0.5, dtype)
    assert (o[4] == 0).all() and (lse[4] == float("-inf")).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 8, 2, 16), (64, 3, 3, 32), (128, 100, 1, 16), (64, 16, 8, 64)])
def test_shared_prefixes(kda, cuda_device, dtype, d, H, H_kv, bs):
    """Groups of many and of one, a prefix of zero, suffixes of zero and more; the result equals the
    unshared call's within the same bounds."""
    p = [2 * bs, 0, 5 * bs, bs]
    start = [0, 40, 42, 43, 50]
    rng = np.random.RandomState(3)
    kv = [p[g] + int(rng.randint(0, 70)) for g in range(4) for _ in range(start[g], start[g + 1])]
    kv[0], kv[45] = p[0], p[3]                                  # empty suffixes
    c = A.Paged(4, kv, H_kv, d, bs, dtype, cuda_device, groups=[(start[g], start[g + 1], p[g] // bs) for g in range(4)])
    q = A.randn(5, (50, H, d), dtype, cuda_device)
    o, lse = _decode(kda, q, c, start, p)
    assert kda.kda_check_status() == 0
    _check(o, lse, q, c, d ** -0.5, dtype)
    o2, lse2 = _decode(kda, q, c)
    _check(o2, lse2, q, c, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_prefix_and_long_suffix(kda, cuda_device, dtype):
    """Keys split over many thread blocks on both sides, against the formula in float64 on the GPU."""
    d, H, H_kv, bs, n, prefix = 128, 8, 2, 64, 3, 64 * 70
    kv = [prefix + 9001, prefix + 1, prefix + 3000]
    blocks = [-(-x // bs) for x in kv]
    shared = prefix // bs
    total = shared + sum(b - shared for b in blocks)
    k, v = (A.randn(s, (total, H_kv, bs, d), dtype, cuda_device) for s in (6, 7))
    table = torch.full((n, max(blocks)), -1, dtype=torch.int32)
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(8)).int()
    at = shared
    for s in range(n):
        table[s, :shared] = perm[:shared]
        table[s, shared:blocks[s]] = perm[at:at + blocks[s] - shared]
        at += blocks[s] - shared
    table = table.to(cuda_device)
    q = A.randn(9, (n, H, d), dtype, cuda_device, 2.0)
    o, lse = kda.attn_decode(q, k, v, table, _i32(kv, cuda_device), group_start=_i32([0, n], cuda_device),
                             prefix_lens=_i32([prefix], cuda_device), want_lse=True)
    assert kda.kda_check_status() == 0
    for s in range(n):
        ks, vs = (x[table[s, :blocks[s]].long()].transpose(1, 2).reshape(-1, H_kv, d)[:kv[s]].double() for x in (k, v))
        ks, vs = (x.repeat_interleave(H // H_kv, 1) for x in (ks, vs))
        x = torch.einsum("hd,khd->hk", q[s].double(), ks) * d ** -0.5
        w = torch.softmax(x, -1)
        ref, spread = torch.einsum("hk,khd->hd", w, vs), torch.einsum("hk,khd->hd", w, vs.abs())
        e, r = A.score_error(A.np64(q), A.np64(ks), d ** -0.5, d), A.half_step(dtype)
        f = 2 * e + 2.0 ** -20 + kv[s] * A.U + (r if dtype == BF else 0.0)
        assert ((o[s].double() - ref).abs() <= f * spread + r * ref.abs() * (1 + f)).all()
        z = torch.logsumexp(x, -1)
        assert ((lse[s].double() - z).abs() <= e + 2.0 ** -20 + kv[s] * A.U + 4 * A.U * z.abs()).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_hidden_slots_hold_anything(kda, cuda_device, dtype):
    """Unowned slots are NaN throughout (the fixture's fill); infinities there change nothing either."""
    kv, d = [5, 70, 129], 64
    c = A.Paged(10, kv, 2, d, 32, dtype, cuda_device)
    q = A.randn(11, (3, 4, d), dtype, cuda_device)
    a, la = _decode(kda, q, c)
    c.k[torch.isnan(c.k)] = float("inf")
    c.v[torch.isnan(c.v)] = float("-inf")
    b, lb = _decode(kda, q, c)
    assert torch.equal(a, b) and torch.equal(la, lb)
    _check(a, la, q, A.Paged(10, kv, 2, d, 32, dtype, cuda_device), d ** -0.5, dtype)


def test_offsets_past_32_bits(kda, cuda_device):
    """A cache of more than 2^32 elements, with the blocks at its far end in use."""
    H_kv, bs, d = 8, 256, 128
    n_blocks = (1 << 32) // (H_kv * bs * d) + 40
    k = torch.empty((n_blocks, H_kv, bs, d), dtype=BF, device=cuda_device)
    v = torch.empty_like(k)
    kv = [700, 300]
    table_np = np.array([[n_blocks - 1, 3, n_blocks - 7], [n_blocks // 2 + 9, n_blocks - 2, -1]], np.int32)
    new_k, new_v = A.randn(12, (1000, H_kv, d), BF, cuda_device), A.randn(13, (1000, H_kv, d), BF, cuda_device)
    slots = [int(table_np[s, j // bs]) * bs + j % bs for s, n in enumerate(kv) for j in range(n)]
    kda.kda_cache_append(new_k, new_v, _i32(slots, cuda_device), k, v)
    table = torch.from_numpy(table_np).to(cuda_device)
    q = A.randn(14, (2, 16, d), BF, cuda_device)
    o, lse = kda.attn_decode(q, k, v, table, _i32(kv, cuda_device), want_lse=True)
    qp = A.randn(15, (1000, 16, d), BF, cuda_device)
    op, _ = kda.attn_prefill_paged(qp, k, v, table, _i32(kv, cuda_device), A.cu_of(kv, cuda_device))
    want, _ = kda.attn_prefill(qp, new_k, new_v, A.cu_of(kv, cuda_device))
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    A.check(o, lse, A.split(q, [1, 1]), A.split(new_k, kv), A.split(new_v, kv), [n - 1 for n in kv], d ** -0.5, BF)
    assert torch.equal(op, want)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_bad_lengths_groups_and_blocks_are_flagged(kda, cuda_device, dtype):
    kv, d = [40, 50, 33, 20], 64
    q = A.randn(16, (4, 4, d), dtype, cuda_device)
    c = A.Paged(17, kv, 2, d, 16, dtype, cuda_device)
    c.kv_lens[1] = 16 * c.table.shape[1] + 1
    c.kv_lens[3] = -2
    o, lse = _decode(kda, q, c)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    assert (o[[1, 3]] == 0).all() and (lse[[1, 3]] == float("-inf")).all()
    good = A.Paged(17, kv, 2, d, 16, dtype, cuda_device)
    keys, values = good.keys_values()
    for s in (0, 2):
        A.check(o[s:s + 1], lse[s:s + 1], [A.np64(q[s:s + 1])], keys[s:s + 1], values[s:s + 1], [kv[s] - 1], d ** -0.5, dtype)
    for start, prefix in (([0, 4], [17]), ([0, 4], [-16]), ([0, 3], [16]), ([1, 4], [16]), ([0, 9], [16]), ([0, 4], [32])):
        _decode(kda, q, good, start, prefix)
        assert kda.kda_check_status() & kda.KDA_DEV_BAD_GROUP, (start, prefix)
    bad = A.Paged(17, kv, 2, d, 16, dtype, cuda_device)
    bad.table[2, 1] = bad.n_blocks
    o, lse = _decode(kda, q, bad)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    for s in (0, 1, 3):
        A.check(o[s:s + 1], lse[s:s + 1], [A.np64(q[s:s + 1])], keys[s:s + 1], values[s:s + 1], [kv[s] - 1], d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_in_a_graph_on_another_stream(kda, cuda_device, dtype):
    """plan, append and decode captured once and replayed over changing lengths."""
    dev, d, H, H_kv, bs, n = cuda_device, 64, 4, 2, 16, 5
    side = torch.cuda.Stream()
    cached, new = _i32([0, 15, 16, 40, 7], dev), _i32([1] * n, dev)
    table = torch.full((n, 6), -1, dtype=torch.int32)
    for s, c in enumerate([0, 15, 16, 40, 7]):
        table[s, :-(-c // bs)] = torch.arange(-(-c // bs)) + 6 * s
    table = table.to(dev)
    free = torch.arange(40, 80, dtype=torch.int32, device=dev)
    cur = [_i32([0], dev), _i32([0], dev)]
    kc, vc = (A.randn(s, (80, H_kv, bs, d), dtype, dev) for s in (20, 21))
    k, v = (torch.zeros((n, H_kv, d), dtype=dtype, device=dev) for _ in range(2))
    q = torch.zeros((n, H, d), dtype=dtype, device=dev)
    o, lse = torch.zeros_like(q), torch.zeros((n, H), device=dev)

    def step(stream=None):
        p = kda.cache_plan(cached, new, table, free, cur[0], cur[1], block_size=bs, n_blocks=80, max_tokens=n, stream=stream)
        kda.kda_cache_append(k, v, p.slot_map, kc, vc, stream=stream)
        kda.attn_decode(q, kc, vc, table, p.kv_lens, o=o, lse=lse, stream=stream)
        return p

    step()                                                      # loads the kernels before the capture
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        p = step()
    lens = [0, 15, 16, 40, 7]
    for i in range(20):
        k.copy_(A.randn(30 + i, k.shape, dtype, dev))
        v.copy_(A.randn(60 + i, v.shape, dtype, dev))
        q.copy_(A.randn(90 + i, q.shape, dtype, dev))
        graph.replay()
        lens = [x + 1 for x in lens]
        assert p.kv_lens.tolist() == lens
        cached.copy_(p.kv_lens)
        cur[0].copy_(cur[1])
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    from oracle import attention as oa
    kk, vv, tb = A.np64(kc), A.np64(vc), table.cpu().numpy()
    A.check(o, lse, A.split(q, [1] * n), [oa.gather(kk, tb[s], x) for s, x in enumerate(lens)],
            [oa.gather(vv, tb[s], x) for s, x in enumerate(lens)], [x - 1 for x in lens], d ** -0.5, dtype)
