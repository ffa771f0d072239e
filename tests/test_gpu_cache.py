"""The paged cache's step plan and append on the GPU: integers and copies, so everything is exact."""
import numpy as np
import pytest
import torch

from oracle import attention as oa

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def _setup(seed, cached, new, bs, extra=4):
    rng = np.random.RandomState(seed)
    have = [-(-c // bs) for c in cached]
    need = [-(-(c + t) // bs) for c, t in zip(cached, new)]
    n_blocks = sum(need) + extra
    perm = rng.permutation(n_blocks)
    table = np.full((len(cached), max(need, default=0) + 2), -1)
    at = 0
    for s, h in enumerate(have):
        table[s, :h] = perm[at:at + h]
        at += h
    return table, np.concatenate([[-9, -9], perm[at:]]), n_blocks


def _plan(kda, dev, cached, new, table, free, begin, bs, n_blocks, max_tokens, **kw):
    tb, end = _i32(table, dev), _i32([-1], dev)
    p = kda.cache_plan(_i32(cached, dev), _i32(new, dev), tb, _i32(free, dev), _i32([begin], dev), end, block_size=bs,
                       n_blocks=n_blocks, max_tokens=max_tokens, **kw)
    torch.cuda.synchronize()
    return dict(table=tb.cpu().numpy(), cu_seqlens=p.cu_seqlens.tolist(), kv_lens=p.kv_lens.tolist(),
                slot_map=p.slot_map.tolist(), positions=p.positions.tolist(), free_end=int(end))


CASES = [([0], [1]), ([5], [0]), ([0, 0, 0], [0, 0, 0]), ([15, 16, 17, 0, 3], [1, 1, 1, 40, 0]), ([100, 0], [5000, 3])]


@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("cached,new", CASES + [("many", 700), ("many", 256), ("many", 2049)])
@pytest.mark.parametrize("pad", [0, 1, 777])
def test_plan_matches_the_definition(kda, cuda_device, bs, cached, new, pad):
    if cached == "many":
        rng = np.random.RandomState(new)
        cached, new = rng.randint(0, 300, new).tolist(), (rng.randint(0, 30, new) * rng.randint(0, 2, new)).tolist()
    table, free, n_blocks = _setup(1, cached, new, bs)
    T = sum(new) + pad
    got = _plan(kda, cuda_device, cached, new, table, free, 2, bs, n_blocks, T)
    assert kda.kda_check_status() == 0
    want = oa.plan(cached, new, table, free, 2, bs, T)
    for key in want:
        assert np.array_equal(got[key], want[key]), key


def test_plan_of_no_sequences(kda, cuda_device):
    got = _plan(kda, cuda_device, [], [], np.zeros((0, 3)), [4, 5], 1, 16, 8, 5)
    assert got["cu_seqlens"] == [0] and got["slot_map"] == [-1] * 5 and got["free_end"] == 1
    assert kda.kda_check_status() == 0


def test_plan_when_the_free_list_ends(kda, cuda_device):
    """The third sequence gets one of its two blocks, the fourth none; the second still fits in its own."""
    cached, new, bs = [0, 18, 30, 0], [20, 5, 20, 9], 16
    table = np.array([[-1, -1, -1, -1], [0, 1, -1, -1], [2, 3, -1, -1], [-1] * 4])
    got = _plan(kda, cuda_device, cached, new, table, [10, 11, 12], 0, bs, 20, 60)
    assert kda.kda_check_status() == kda.KDA_DEV_NO_BLOCKS
    assert got["kv_lens"] == [20, 23, 48, 0] and got["free_end"] == 3 and got["cu_seqlens"] == [0, 20, 25, 45, 54]
    assert got["table"][2].tolist() == [2, 3, 12, -1] and got["table"][3].tolist() == [-1] * 4
    want = [160 + i for i in range(16)] + [176 + i for i in range(4)] + [16 + i for i in range(2, 7)]
    want += [48 + 14, 48 + 15] + [192 + i for i in range(16)] + [-1, -1] + [-1] * 9 + [-1] * 6
    assert got["slot_map"] == want and got["positions"][43:54] == [48, 49] + list(range(9))


def test_plan_flags_bad_lengths_and_blocks(kda, cuda_device):
    bs, table = 16, np.array([[0, 1], [2, 3], [-1, -1], [-1, -1]])
    got = _plan(kda, cuda_device, [-4, 20, 0, 0], [3, 40, -2, 1], table, [5, 99, 7, 8], 0, bs, 20, 30)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS | kda.KDA_DEV_BAD_SLOT
    # -4 counts as 0 and takes block 5; 20 + 40 is cut to the row's 32; the last takes the bad entry
    assert got["kv_lens"] == [3, 32, 0, 1] and got["cu_seqlens"] == [0, 3, 15, 15, 16]
    assert got["slot_map"][:3] == [80, 81, 82] and got["slot_map"][15] == -1 and got["table"][3, 0] == -1
    got = _plan(kda, cuda_device, [0, 0], [20, 20], np.full((2, 2), -1), [1, 2, 3, 4], 0, bs, 20, 25)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    assert got["cu_seqlens"] == [0, 20, 25] and got["kv_lens"] == [20, 5] and got["free_end"] == 3
    for begin in (-1, 9):
        got = _plan(kda, cuda_device, [0], [3], [[-1]], [1, 2], begin, bs, 20, 4)
        assert kda.kda_check_status() == kda.KDA_DEV_NO_BLOCKS
        assert got["slot_map"] == [-1] * 4 and got["kv_lens"] == [0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,H,bs", [(64, 1, 16), (128, 3, 32), (64, 8, 256), (128, 8, 16)])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_append(kda, cuda_device, dtype, d, H, bs, T):
    """Views of a fused projection; padded and out-of-range slots; every other slot untouched."""
    dev = cuda_device
    n_blocks = -(-T // bs) + 3
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, 4 * H, d), generator=g).to(dtype).to(dev)
    k, v = x[:, H:2 * H], x[:, 3 * H:]
    kc, vc = (torch.randn((n_blocks, H, bs, d), generator=g).to(dtype).to(dev) for _ in range(2))
    slots = torch.randperm(n_blocks * bs, generator=g)[:T]
    slots[::5] = -1
    want = []
    for cache, new in ((kc, k), (vc, v)):
        flat = cache.clone().permute(0, 2, 1, 3).reshape(-1, H, d)
        for t in range(T):
            if slots[t] >= 0:
                flat[slots[t]] = new[t]
        want.append(flat.view(n_blocks, bs, H, d).permute(0, 2, 1, 3))
    kda.kda_cache_append(k, v, slots.int().to(dev), kc, vc)
    assert kda.kda_check_status() == 0
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    bad = slots.clone()
    bad[0] = n_blocks * bs
    kda.kda_cache_append(k, v, bad.int().to(dev), kc, vc)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
