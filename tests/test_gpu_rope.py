"""Norms and rotation of queries and keys on the GPU against the float64 reference.

Bound of one result, from the arithmetic (u = 2^-24, r = half a step of the type): the sum of d squares is off by at most
(d + 3) u of itself, its inverse root by half that and 3 u, the products with it and the weight by 2 u; the angle by 2^-32 of
a turn and 2^-25 of an eighth of one (0.5 u together), sine and cosine by 2 u; the two products and their sum by 2 u.  All of it relative to
|a| + |b| of the pair:  |y - ref| <= (d / 2 + 16) u (|a| + |b|) + r |ref|.
"""
import numpy as np
import pytest
import torch

import _attention as A
from oracle import rope as orope

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _turns(rng, n):
    """Frequencies of the usual range, and some that wrap around a turn at every position."""
    f = [int(2.0 ** 64 * 10000.0 ** (-i / n) / (2 * np.pi)) for i in range(n)]
    f[::5] = [int(x) for x in rng.randint(0, 1 << 62, len(f[::5])) * 4 + 3]
    return f


def _i64(turns, dev):
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in turns], dtype=torch.int64, device=dev)


def _positions(rng, T, hi=1 << 31):
    p = rng.randint(0, hi, T)
    p[: min(T, 3)] = [0, 1, hi - 1][: min(T, 3)]
    return p


def _check(got, x, weight, eps, pos, turns, interleaved, dtype):
    d = x.shape[-1]
    live = np.asarray(pos) >= 0
    ref, spread = orope.norm_rope(A.np64(x)[live], None if weight is None else A.np64(weight), eps, np.asarray(pos)[live], turns, interleaved)
    bound = (d / 2 + 16) * A.U * spread + A.half_step(dtype) * np.abs(ref) * (1 + 2.0 ** -8) + 1e-37
    off = np.abs(A.np64(got)[live] - ref)
    assert (off <= bound).all(), (float((off / bound).max()), np.argwhere(off > bound)[:4].tolist())


def _norms(seed, d, dev):
    return 1 + A.randn(seed, (d,), F32, dev, 0.3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,rot", [(128, 4, 1, 128), (64, 3, 2, 64), (128, 5, 5, 40), (64, 1, 1, 8), (128, 40, 8, 64),
                                          (64, 7, 3, 0), (128, 1, 130, 120)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(kda, cuda_device, dtype, d, H, H_kv, rot, interleaved, norm):
    dev, T = cuda_device, 9
    rng = np.random.RandomState(d + rot)
    x = A.randn(1, (T, H + 2 * H_kv, d), dtype, dev, 3.0)
    q, k = x[:, :H], x[:, H:H + H_kv]                       # views of a fused projection
    wq, wk = (_norms(2, d, dev), _norms(3, d, dev)) if norm else (None, None)
    pos, turns = _positions(rng, T), _turns(rng, rot // 2)
    pos[4] = -1
    q_out, k_out = torch.full((T, H, d), 7.0, dtype=dtype, device=dev), torch.full((T, H_kv + 1, d), 7.0, dtype=dtype, device=dev)
    a, b = kda.qk_norm_rope(q, k, torch.from_numpy(pos).int().to(dev), _i64(turns, dev), interleaved=interleaved, q_weight=wq,
                            k_weight=wk, eps=1e-5, q_out=q_out, k_out=k_out[:, 1:])
    assert kda.kda_check_status() == 0
    assert a is q_out and (q_out[4] == 7).all() and (k_out[4] == 7).all() and (k_out[:, 0] == 7).all()
    _check(a, q, wq, 1e-5, pos, turns, interleaved, dtype)
    _check(b, k, wk, 1e-5, pos, turns, interleaved, dtype)
    # in place, with outputs that are the views themselves
    before = x.clone()
    kda.qk_norm_rope(q, k, torch.from_numpy(pos).int().to(dev), _i64(turns, dev), interleaved=interleaved, q_weight=wq,
                     k_weight=wk, eps=1e-5, q_out=q, k_out=k)
    live = pos >= 0
    assert torch.equal(q[live], a[live]) and torch.equal(k[live], b[live])
    assert torch.equal(x[4], before[4]) and torch.equal(x[:, H + H_kv:], before[:, H + H_kv:])


@pytest.mark.parametrize("T", [1, 2, 63, 700, 6000])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_lengths(kda, cuda_device, T, dtype, d):
    """Rows spread over many warps for few tokens, and one warp for a token's rows for many."""
    dev, H, H_kv = cuda_device, 32, 8
    rng = np.random.RandomState(T)
    q, k = A.randn(4, (T, H, d), dtype, dev), A.randn(5, (T, H_kv, d), dtype, dev)
    pos, turns, w = _positions(rng, T), _turns(rng, d // 2), _norms(6, d, dev)
    a, b = kda.qk_norm_rope(q, k, torch.from_numpy(pos).int().to(dev), _i64(turns, dev), q_weight=w, k_weight=w)
    at = np.unique(np.concatenate([[0, T - 1], rng.randint(0, T, 40)]))
    _check(a[at], q[at], w, 1e-6, pos[at], turns, False, dtype)
    _check(b[at], k[at], w, 1e-6, pos[at], turns, False, dtype)


def test_one_norm_only_and_no_rotation(kda, cuda_device):
    dev = cuda_device
    q, k, w = A.randn(7, (5, 2, 64), F32, dev), A.randn(8, (5, 3, 64), F32, dev), _norms(9, 64, dev)
    pos = torch.zeros(5, dtype=torch.int32, device=dev)
    a, b = kda.qk_norm_rope(q, k, pos, q_weight=w)
    assert torch.equal(b, k)
    _check(a, q, w, 1e-6, [0] * 5, [], False, F32)


@pytest.mark.parametrize("dtype,bad", [(BF, float("nan")), (F32, float("inf"))])
def test_rows_are_apart(kda, cuda_device, dtype, bad):
    """A head that holds something not finite changes no other head, and zeros stay zeros under a norm."""
    dev, d = cuda_device, 64
    q, k, w = A.randn(10, (3, 4, d), dtype, dev), A.randn(11, (3, 2, d), dtype, dev), _norms(12, d, dev)
    pos, turns = torch.tensor([5, 6, 7], dtype=torch.int32, device=dev), _i64(_turns(np.random.RandomState(1), d // 2), dev)
    a, b = kda.qk_norm_rope(q, k, pos, turns, q_weight=w, k_weight=w)
    q[1, 2, 9] = bad
    k[2, 1] = 0
    a2, b2 = kda.qk_norm_rope(q, k, pos, turns, q_weight=w, k_weight=w)
    hit = torch.zeros(3, 4, dtype=torch.bool)
    hit[1, 2] = True
    assert torch.equal(a2[~hit], a[~hit]) and torch.isnan(a2[1, 2]).any()
    assert torch.equal(b2[:2], b[:2]) and torch.equal(b2[2, 0], b[2, 0]) and (b2[2, 1] == 0).all()


def test_bad_positions_are_flagged(kda, cuda_device):
    dev = cuda_device
    q, k = A.randn(13, (4, 2, 64), BF, dev), A.randn(14, (4, 1, 64), BF, dev)
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    kda.qk_norm_rope(q, k, torch.tensor([3, -2, -1, 4], dtype=torch.int32, device=dev), q_out=q_out, k_out=k_out)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_POSITION
    assert torch.equal(q_out[[0, 3]], q[[0, 3]]) and (q_out[1:3] == 0).all() and (k_out[1:3] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,bs,rot,interleaved,norm", [(128, 8, 2, 16, 128, False, True), (64, 0, 3, 64, 32, True, False),
                                                              (64, 5, 1, 256, 64, False, True), (128, 3, 9, 32, 0, False, True)])
@pytest.mark.parametrize("T", [1, 130])
def test_append(kda, cuda_device, dtype, d, H, H_kv, bs, rot, interleaved, norm, T):
    """What ``qk_norm_rope`` and ``kda_cache_append`` give in turn, bit for bit, with padded and skipped tokens."""
    dev = cuda_device
    rng = np.random.RandomState(T + d)
    x = A.randn(15, (T, H + 2 * H_kv, d), dtype, dev)
    q, k, v = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    n_blocks = -(-T // bs) + 3
    caches = [A.randn(16 + i, (n_blocks, H_kv, bs, d), dtype, dev) for i in range(2)]
    slots = rng.permutation(n_blocks * bs)[:T]
    slots[1::5] = -1                                       # no place in the cache, yet queries
    pos = _positions(rng, T)
    pos[2::7], slots[2::7] = -1, -1                        # padding
    pos, slots = (torch.from_numpy(a).int().to(dev) for a in (pos, slots))
    turns = _i64(_turns(rng, rot // 2), dev)
    w = dict(q_weight=_norms(18, d, dev) if H else None, k_weight=_norms(19, d, dev)) if norm else {}
    want = [c.clone() for c in caches]
    zq, zk = torch.zeros((T, max(H, 1), d), dtype=dtype, device=dev), torch.zeros((T, H_kv, d), dtype=dtype, device=dev)
    fill = dict(w)
    if not H:
        fill["q_weight"] = None
    wq, wk = kda.qk_norm_rope(q if H else k[:, :1], k, pos, turns, interleaved=interleaved, q_out=zq, k_out=zk, **fill)
    kda.kda_cache_append(wk, v, slots, *want)
    q_out = torch.zeros_like(zq) if H else None
    got = kda.cache_append_rope(k, v, pos, turns, slots, *caches, q=q if H else None, q_out=q_out, interleaved=interleaved, **w)
    assert kda.kda_check_status() == 0
    assert got is q_out and (not H or torch.equal(q_out, wq))
    assert torch.equal(caches[0], want[0]) and torch.equal(caches[1], want[1])
    bad = slots.clone()
    bad[0] = n_blocks * bs
    kda.cache_append_rope(k, v, pos, turns, bad, *caches, interleaved=interleaved, k_weight=w.get("k_weight"))
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    assert torch.equal(caches[0], want[0]) and torch.equal(caches[1], want[1])


def test_append_past_32_bits(kda, cuda_device):
    """A cache of more than 2^32 elements, with its last slots in use."""
    dev, H_kv, bs, d, T = cuda_device, 8, 256, 128, 40
    n_blocks = (1 << 32) // (H_kv * bs * d) + 2
    kc = torch.zeros((n_blocks, H_kv, bs, d), dtype=BF, device=dev)
    vc = torch.zeros_like(kc)
    k, v = A.randn(20, (T, H_kv, d), BF, dev), A.randn(21, (T, H_kv, d), BF, dev)
    slots = torch.arange(n_blocks * bs - T, n_blocks * bs, dtype=torch.int32, device=dev)
    pos, turns = torch.arange(T, dtype=torch.int32, device=dev), _i64(_turns(np.random.RandomState(2), 64), dev)
    kda.cache_append_rope(k, v, pos, turns, slots, kc, vc)
    _, want = kda.qk_norm_rope(k, k, pos, turns)
    assert kda.kda_check_status() == 0
    assert torch.equal(kc[-1, :, -T:].transpose(0, 1), want) and torch.equal(vc[-1, :, -T:].transpose(0, 1), v)
    assert not kc[:-1].any() and not kc[-1, :, :-T].any()


def test_step_in_a_graph_on_another_stream(kda, cuda_device):
    """One launch between projection and attention, captured once, replayed as positions and slots move on."""
    dev, n, H, H_kv, d, bs = cuda_device, 5, 4, 2, 64, 16
    qkv = torch.zeros((n, H + 2 * H_kv, d), dtype=BF, device=dev)
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    pos, slots = (torch.zeros(n, dtype=torch.int32, device=dev) for _ in range(2))
    kc, vc = (torch.zeros((n * 2, H_kv, bs, d), dtype=BF, device=dev) for _ in range(2))
    wkc, wvc = torch.zeros_like(kc), torch.zeros_like(vc)
    turns, w = _i64(_turns(np.random.RandomState(3), d // 2), dev), _norms(22, d, dev)
    side = torch.cuda.Stream()
    kda.cache_append_rope(k, v, pos, turns, slots - 1, kc, vc, q=q, q_weight=w, k_weight=w, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = kda.cache_append_rope(k, v, pos, turns, slots, kc, vc, q=q, q_weight=w, k_weight=w)
    for i in range(12):
        qkv.copy_(A.randn(30 + i, qkv.shape, BF, dev))
        pos.copy_(torch.arange(n, device=dev) + 3 + i)
        slots.copy_((torch.arange(n, device=dev) * 2 * bs) + i)
        graph.replay()
        a, b = kda.qk_norm_rope(q, k, pos, turns, q_weight=w, k_weight=w)
        kda.kda_cache_append(b, v, slots, wkc, wvc)
        assert torch.equal(out, a)
    assert kda.kda_check_status() == 0
    assert torch.equal(kc, wkc) and torch.equal(vc, wvc)
