"""The 4-bit cache's append and read-back on the GPU: the codes, scales and values are those of the definition, bit for bit."""
import numpy as np
import pytest
import torch

import _attention as A
import _q4
from oracle import cache_q4 as oq

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def _same(a, b):
    """Equal as numbers, NaN equal to itself."""
    a, b = a.double(), b.double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def _filled(kda, rng, n_blocks, H, bs, d, dev):
    c = kda.q4_cache(n_blocks, H, bs, d, dev)
    for i, t in enumerate(c):
        t.copy_(torch.from_numpy(rng.randint(0, 256, t.shape)).to(torch.uint8) if i % 2 == 0 else torch.from_numpy(rng.randn(*t.shape)))
    return c


def _expect(c, k, v, slots):
    """(the cache after the append, the values) of the definition, on the CPU."""
    out, values = [t.cpu().clone() for t in c], []
    bs = c.k_codes.shape[2]
    for i, x in enumerate((k, v)):
        codes, s, m = oq.quantize(x.float().cpu().numpy())
        values.append(torch.from_numpy(oq.values(codes, s, m)))
        for t, slot in enumerate(slots):
            if slot >= 0:
                out[2 * i][slot // bs, :, slot % bs] = torch.from_numpy(oq.packed(codes[t]))
                out[2 * i + 1][slot // bs, :, slot % bs] = _q4.bf16(np.stack([s[t], m[t]], -1))
    return out, values


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,bs", [(64, 1, 16), (128, 3, 32), (64, 8, 256), (128, 8, 16), (128, 1, 64), (64, 130, 16)])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_append(kda, cuda_device, dtype, d, H, bs, T):
    """Views of a fused projection; padded and out-of-range slots; every other slot untouched; values to views, or in place."""
    dev, rng = cuda_device, np.random.RandomState(T)
    n_blocks = -(-T // bs) + 3
    x = A.randn(T, (T, 4 * H, d), dtype, dev, 2.0) + 0.5
    k, v = x[:, H:2 * H], x[:, 3 * H:]
    c = _filled(kda, rng, n_blocks, H, bs, d, dev)
    slots = rng.permutation(n_blocks * bs)[:T]
    slots[::5] = -1
    want, values = _expect(c, k, v, slots)
    k_out = torch.full((T, H + 1, d), 7.0, dtype=dtype, device=dev)
    got, none = kda.cache_append_q4(k, v, _i32(slots, dev), c, k_out=k_out[:, 1:])
    assert kda.kda_check_status() == 0 and none is None
    assert all(_same(a.cpu(), b) for a, b in zip(c, want))
    live = slots >= 0
    assert torch.equal(got[live].cpu(), values[0][live].to(dtype)) and (k_out[~live] == 7).all() and (k_out[:, 0] == 7).all()
    bad = slots.copy()
    bad[0] = n_blocks * bs
    before = x.clone()
    kda.cache_append_q4(k, v, _i32(bad, dev), c, k_out=k, v_out=v)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    assert all(_same(a.cpu(), b) for a, b in zip(c, want))
    assert torch.equal(k[live].cpu(), values[0][live].to(dtype)) and torch.equal(v[live].cpu(), values[1][live].to(dtype))
    assert torch.equal(k[~live], before[~live, H:2 * H]) and torch.equal(x[:, :H], before[:, :H])


def _odd_groups():
    """Groups of 64 where the definition's corners are."""
    big = 3.0e38
    rows = [np.zeros(64), np.full(64, -0.0), np.full(64, 1.7), np.full(64, -3.3e-39), np.r_[np.zeros(63), 1e-40],
            np.r_[np.full(32, big), np.full(32, -big)], np.r_[np.full(63, 1.0), np.inf], np.r_[np.full(63, 1.0), -np.inf],
            np.r_[np.nan, np.ones(63)], np.full(64, np.nan), np.full(64, 3.4e38), np.full(64, -3.4e38),
            np.r_[np.full(63, -1e-3), 1e30], np.r_[np.full(63, 1.0), 1 + 2.0 ** -7], np.arange(64) / 4.2, -np.arange(64) * 1e-39,
            np.r_[0.0, 15.0, np.arange(62) % 15 + 0.5], np.r_[-8.0, 7.0, np.arange(62) % 15 - 7.5], np.r_[0, 30.0, np.arange(62) % 15 * 2 + 1.0],
            np.r_[np.full(63, 2.0 ** -126), 2.0 ** -133]]
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_corners(kda, cuda_device, dtype, d):
    dev, rows = cuda_device, torch.from_numpy(_odd_groups())
    T = rows.shape[0]
    k = rows.repeat(1, d // 64).view(T, 1, d).to(dtype).to(dev)
    v = rows.flip(0).repeat(1, d // 64).view(T, 1, d).to(dtype).to(dev)
    c = _filled(kda, np.random.RandomState(0), 3, 1, 16, d, dev)
    slots = np.arange(T) + 5
    want, values = _expect(c, k, v, slots)
    got = kda.cache_append_q4(k, v, _i32(slots, dev), c, want_values=True)
    assert kda.kda_check_status() == 0
    assert all(_same(a.cpu(), b) for a, b in zip(c, want))
    for a, b in zip(got, values):
        assert _same(a.cpu(), b.float().to(dtype))


@pytest.mark.parametrize("dtype,T,H,d", [(BF, 5000, 8, 128), (F32, 3001, 3, 64), (BF, 40000, 1, 64)])
def test_append_of_many(kda, cuda_device, dtype, T, H, d):
    """Whole batches, values of many magnitudes, against the definition: several tokens a thread block, ragged ends."""
    dev, bs = cuda_device, 64
    n_blocks = -(-T // bs) + 1
    g = torch.Generator().manual_seed(T)
    size = torch.exp(3 * torch.randn((T, H, 1), generator=g))
    k, v = ((torch.randn((T, H, d), generator=g) * size).to(dtype).to(dev) for _ in range(2))
    c = _filled(kda, np.random.RandomState(1), n_blocks, H, bs, d, dev)
    slots = torch.randperm(n_blocks * bs, generator=g)[:T].numpy()
    kda.cache_append_q4(k, v, _i32(slots, dev), c)
    assert kda.kda_check_status() == 0
    for i, x in enumerate((k, v)):
        codes, s, m = oq.quantize(x.float().cpu().numpy())
        assert np.array_equal(c[2 * i].cpu().numpy()[slots // bs, :, slots % bs], oq.packed(codes))
        assert _same(c[2 * i + 1].cpu()[slots // bs, :, slots % bs], _q4.bf16(np.stack([s, m], -1)))
        err = np.abs(oq.values(codes, s, m) - x.double().cpu().numpy()).reshape(T, H, -1, 64)
        assert (err <= 0.5 * s[..., None].astype(np.float64) * (1 + 2.0 ** -20)).all()


def _unpack_expect(c, out, to_np, first, dtype):
    bs = c.codes.shape[3]
    for x in range(2):
        v = torch.from_numpy(oq.values(c.codes[x], c.s[x], c.m[x])).to(dtype)
        for i, n in enumerate(c.kv):
            for j in range(first[i], n):
                out[x][to_np[i, j // bs], :, j % bs] = v[c.table_np[i, j // bs], :, j % bs]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,H,bs", [(64, 1, 16), (128, 3, 32), (64, 2, 256), (128, 8, 16), (64, 5, 64)])
@pytest.mark.parametrize("kv", [[1], [0, 0], [5, 0, 16, 17, 300, 31, 64], "many"])
def test_unpack(kda, cuda_device, dtype, d, H, bs, kv):
    """Positions from first on, to other blocks; nothing else of the full-width cache is written."""
    dev, rng = cuda_device, np.random.RandomState(d)
    if kv == "many":
        kv = (rng.randint(0, 30, 600) * rng.randint(0, 2, 600)).tolist()
    c = _q4.Paged(2, kv, H, d, bs, dtype, dev)
    need = [-(-n // bs) for n in kv]
    wide = sum(need) + 2
    perm, to_np, at = rng.permutation(wide), np.full((len(kv), max(need) + 2), -1, np.int32), 0
    for i, n in enumerate(need):
        to_np[i, :n] = perm[at:at + n]
        at += n
    for first in (None, [int(rng.randint(0, n + 3)) for n in kv]):
        caches = [A.randn(3 + i, (wide, H, bs, d), dtype, dev) for i in range(2)]
        want = [t.cpu().clone() for t in caches]
        _unpack_expect(c, want, to_np, first or [0] * len(kv), dtype)
        kda.cache_unpack_q4(c.cache, c.table, c.kv_lens, *caches, _i32(to_np, dev), first=None if first is None else _i32(first, dev))
        assert kda.kda_check_status() == 0
        assert torch.equal(caches[0].cpu(), want[0]) and torch.equal(caches[1].cpu(), want[1])


def test_unpack_flags_bad_lengths_and_blocks(kda, cuda_device):
    dev, bs, d, kv = cuda_device, 16, 64, [20, 20, 20, 20, 20]
    c = _q4.Paged(4, kv, 2, d, bs, BF, dev)
    to_np = np.arange(10, dtype=np.int32).reshape(5, 2)
    caches = [torch.zeros((10, 2, bs, d), dtype=BF, device=dev) for _ in range(2)]
    c.kv_lens[1] = 33
    kda.cache_unpack_q4(c.cache, c.table, c.kv_lens, *caches, _i32(to_np, dev), first=_i32([0, 0, -1, 0, 0], dev))
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    want = [t.cpu().clone().zero_() for t in caches]
    _unpack_expect(c, want, to_np, [0, 99, 99, 0, 0], BF)
    assert torch.equal(caches[0].cpu(), want[0]) and torch.equal(caches[1].cpu(), want[1])
    c.kv_lens.fill_(20)
    c.table[0, 1] = c.n_blocks
    to_np[3, 0] = 10
    caches = [torch.zeros_like(t) for t in caches]
    kda.cache_unpack_q4(c.cache, c.table, c.kv_lens, *caches, _i32(to_np, dev))
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    want = [t.zero_() for t in want]
    kv, c.kv = c.kv, [16, 20, 20, 0, 20]
    _unpack_expect(c, want, to_np, [0] * 5, BF)
    v = torch.from_numpy(oq.values(c.codes, c.s, c.m)).to(BF)
    for x in range(2):
        want[x][to_np[3, 1], :, :4] = v[x, c.table_np[3, 1], :, :4]
    assert torch.equal(caches[0].cpu(), want[0]) and torch.equal(caches[1].cpu(), want[1])


def test_past_32_bits(kda, cuda_device):
    """A cache whose elements and bytes pass 2^32, with its far end in use, written and read back."""
    dev, H, bs, d, T = cuda_device, 8, 256, 128, 300
    n_blocks = (1 << 33) // (H * bs * d) + 3
    c = kda.q4_cache(n_blocks, H, bs, d, dev)
    k, v = A.randn(5, (T, H, d), BF, dev), A.randn(6, (T, H, d), BF, dev)
    table = _i32([[n_blocks - 1, n_blocks - 3]], dev)
    slots = torch.cat([(n_blocks - 1) * bs + torch.arange(256), (n_blocks - 3) * bs + torch.arange(T - 256)]).int().to(dev)
    ko, vo = kda.cache_append_q4(k, v, slots, c, want_values=True)
    wide = (1 << 32) // (H * bs * d) + 3
    kc, vc = (torch.zeros((wide, H, bs, d), dtype=BF, device=dev) for _ in range(2))
    kda.cache_unpack_q4(c, table, _i32([T], dev), kc, vc, _i32([[wide - 1, 7]], dev))
    assert kda.kda_check_status() == 0
    codes, s, m = oq.quantize(k.float().cpu().numpy())
    want = torch.from_numpy(oq.values(codes, s, m)).to(BF)
    assert torch.equal(ko.cpu(), want)
    for cache, values in ((kc, ko), (vc, vo)):
        assert torch.equal(cache[wide - 1].transpose(0, 1), values[:256]) and torch.equal(cache[7, :, :T - 256].transpose(0, 1), values[256:])
        assert not cache[8:wide - 1].any()
