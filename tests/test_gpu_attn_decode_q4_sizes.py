"""Decode attention over the 4-bit cache where sizes differ widely: value groups without width, values that shrink or grow
along a sequence while scores do the same, queries whose channels differ.  Against the float64 reference.

The bounds are ``_q4``'s.  What falls under fp16's range (half a step is 2^-25 there, the largest weight times step of a head
and group lies at 2^6 or more) is at most 2^-31 of that largest one a key: ``_check`` adds 8 K of these, for the codes' 8.
"""
import numpy as np
import pytest
import torch

import _attention as A
import _q4

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KEYS = 32                                                    # of a tile


def _each(c, i, x, t):
    """t [positions] for all of sequence i's slots of keys (x = 0) or values (1), beside c.s[x] and c.m[x]."""
    bs = c.codes.shape[3]
    out = np.zeros(c.s[x].shape, np.float32)
    for j in range(c.kv[i]):
        out[c.table_np[i, j // bs], :, j % bs] = t[j]
    return out


def _scale_values(c, i, t):
    """Multiply sequence i's values by t [positions], powers of two or 0 (nobody else owns a slot then)."""
    by = _each(c, i, 1, t)
    with np.errstate(invalid="ignore"):
        c.s[1], c.m[1] = c.s[1] * by, c.m[1] * by


def _check(kda, q, c, dtype, n):
    """n requests of the query q [H, d] on c's only sequence: as many as make pieces of whole sequences, or one cut into small
    pieces.  ``_q4.check`` for each, with the weights that fall under fp16's range."""
    scale = q.shape[1] ** -0.5
    o, lse = kda.attn_decode_q4(q.repeat(n, 1, 1), c.cache, c.table.repeat(n, 1), c.kv_lens.repeat(n), want_lse=True)
    assert kda.kda_check_status() == 0
    keys, values, key_size, value_size = c.sequence(0)
    qn, on = A.np64(q), A.np64(o)
    ref, ref_lse, spread = _q4.attention(qn, keys, values, value_size, scale)
    (H, d), (K, H_kv, _) = qn.shape, keys.shape
    assert np.isfinite(on).all()
    e = 2 * (d + 18) * 2 * A.U * abs(scale) * float(np.abs(qn).max(0) @ key_size.max((0, 1)))
    f = 2 * e + 2.0 ** -20 + 2 * K * A.U + (2.0 ** -11 if dtype == BF else 2.0 ** -21)
    bs = c.codes.shape[3]
    step = np.stack([c.s[1][c.table_np[0, j // bs], :, j % bs] for j in range(K)]).astype(np.float64)   # [K, H_kv, d / 64]
    low = np.zeros_like(ref)
    for h in range(H):
        x = scale * (keys[:, h // (H // H_kv)] @ qn[h])
        w = np.exp(x - x.max())
        low[h] = np.repeat(8 * K * 2.0 ** -31 * (w[:, None] * step[:, h // (H // H_kv)]).max(0) / w.sum(), 64)
    r = A.half_step(dtype)
    bound = (f * spread + low) * (1 + r) + r * np.abs(ref) + 2.0 ** -120
    off = np.abs(on - ref)
    assert (off <= bound).all(), (float((off / bound).max()), np.argwhere(off > bound)[:4].tolist())
    assert (np.abs(A.np64(lse) - ref_lse) <= e + 2.0 ** -20 + K * A.U + 4 * A.U * np.abs(ref_lse)).all()


HEADS = [(64, 4, 1), (128, 8, 2), (128, 16, 1)]
REQUESTS = [1, 3000]


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,H_kv", HEADS)
def test_weights_of_zero_meet_large_values(kda, cuda_device, dtype, n, d, H, H_kv):
    """Tiny values at the first positions, large ones at positions whose weights are zeros in fp32."""
    c = _stairs(kda, cuda_device, dtype, d, H, H_kv, [0, -200], [-90, 40])
    q = torch.ones((H, d), dtype=dtype, device=cuda_device)
    _check(kda, q, c, dtype, n)


def _stairs(kda, dev, dtype, d, H, H_kv, scores, sizes):
    """One sequence of a tile for each of the scores (log2, for a query of ones); the tile's values are N(0, 1) times 2^size."""
    c = _q4.Paged(31, [KEYS * len(scores)], H_kv, d, 32, dtype, dev)
    by_tile = lambda t: np.repeat(np.array(t, np.float64), KEYS)
    _scale_values(c, 0, 2.0 ** by_tile(sizes))
    c.s[0] = c.s[0] * 0                                      # keys of one value, whose product with ones is the score
    m = A.np64(_q4.bf16(by_tile(scores) * np.log(2) * d ** -0.5))
    c.m[0] = np.where(np.isnan(c.m[0]), np.nan, _each(c, 0, 0, m))
    c.upload()
    return c


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,H_kv", HEADS)
@pytest.mark.parametrize("size", [0, -7, -14, -20, -27, -60])
@pytest.mark.parametrize("empty", ["32", "64", "300", "each"])
def test_value_groups_without_width(kda, cuda_device, dtype, n, d, H, H_kv, size, empty):
    """Values of zero in the first positions, or in the first 96 of every 160 of many pieces; small ones behind them."""
    K = 2500 if empty == "each" else 700
    c = _q4.Paged(32, [K], H_kv, d, 32, dtype, cuda_device)
    j = np.arange(K)
    _scale_values(c, 0, np.where(j % 160 < 96 if empty == "each" else j < int(empty), 0.0, 2.0 ** size))
    c.upload()
    q = A.randn(33, (H, d), dtype, cuda_device)
    _check(kda, q, c, dtype, n)


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_group_without_width(kda, cuda_device, dtype, n):
    """Only one of a head's two groups has no width at first; positions of one value, not of zero, among them."""
    d, H, K = 128, 4, 200
    c = _q4.Paged(34, [K], 1, d, 16, dtype, cuda_device)
    for j in range(K):
        at = (1, c.table_np[0, j // 16], 0, j % 16, 1)
        if j < 40:
            c.s[at], c.m[at] = 0, (0, 2.0 ** -18)[j % 2]
        else:
            c.s[at], c.m[at] = c.s[at] * np.float32(2.0 ** -18), c.m[at] * np.float32(2.0 ** -18)
    c.upload()
    q = A.randn(35, (H, d), dtype, cuda_device)
    _check(kda, q, c, dtype, n)


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,H_kv", HEADS)
@pytest.mark.parametrize("first,score,size", [(90, 9, -40), (110, 30, -50), (60, 9, -10), (-60, 9, 20), (60, -9, -20), (-90, -3, 30), (100, 12, -25)])
def test_sizes_that_move_with_the_scores(kda, cuda_device, dtype, n, d, H, H_kv, first, score, size):
    """Tile by tile the scores rise or fall by `score` (log2) and the values by `size`.  Heads of half the scores, of their
    opposite and of none stand beside each other."""
    tiles = range(min(6, 1 + (first + 116) // -size) if size < 0 else 6)       # down to 2^-116
    c = _stairs(kda, cuda_device, dtype, d, H, H_kv, [score * i for i in tiles], [first + size * i for i in tiles])
    q = torch.ones((H, d), dtype=dtype, device=cuda_device)
    for h, x in enumerate((1, 0.5, -1, 0)):
        q[h::4] = x
    _check(kda, q, c, dtype, n)


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_very_different_sizes(kda, cuda_device, dtype, n, d):
    """Values in runs of 1 to 60 positions whose sizes are 2^-60 .. 2^60, in many orders, and scores of all kinds."""
    rng = np.random.RandomState(36)
    for std in (0.3, 3.0):
        runs = []
        while sum(n for n, _ in runs) < 900:
            runs.append((rng.randint(1, 60), rng.randint(-60, 61)))
        t = np.concatenate([np.full(n, 2.0 ** e) for n, e in runs])[:900]
        c = _q4.Paged(37, [900], 1, d, 16, dtype, cuda_device)
        _scale_values(c, 0, t)
        c.upload()
        q = A.randn(38, (8, d), dtype, cuda_device, std)
        _check(kda, q, c, dtype, n)


@pytest.mark.parametrize("n", REQUESTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [4, 16])
@pytest.mark.parametrize("size", [0, 15, 27, 30, 60])
@pytest.mark.parametrize("group", [0, 1])
def test_queries_of_different_sizes_in_the_two_groups(kda, cuda_device, dtype, n, H, size, group):
    """One group's channels of the queries are 2^size times as large, and its keys are zeros: the scores are the other's."""
    d, K = 128, 200
    c = _q4.Paged(39, [K], 1, d, 16, dtype, cuda_device)
    c.s[0][..., group], c.m[0][..., group] = c.s[0][..., group] * 0, c.m[0][..., group] * 0
    c.upload()
    q = A.randn(40, (H, d), dtype, cuda_device)
    q[..., 64 * group:64 * group + 64] *= 2.0 ** size
    _check(kda, q, c, dtype, n)                  # (the bound: keys of zero times any query are zero)
