"""Cases of the softmax-attention side of a hybrid stack: the paged key/value cache's step plan and append, causal
attention over packed prompts, and decode attention over the cache with prefixes that several requests share.

Shapes.  q [T, H, d]; k, v [T, H_kv, d] (H a multiple of H_kv: query head h reads key/value head h // (H / H_kv));
caches [n_blocks, H_kv, block_size, d]; slot = block * block_size + offset inside the block.  Sequence s owns the packed
tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1, and they are the last ones of its kv_lens[s] positions.

Lengths come from the case itself (`lens_seed`), values from the seed.
"""
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 512 requests: every request appends one token
        dict(name="plan_step_512", kind="plan", n=512, new_lo=1, new_hi=1, cached_lo=1, cached_hi=16384, block_size=16,
             lens_seed=11),
        # the mixed prompt batch: 64 prompts of 1 to 16384 tokens, half of them behind a cached prefix
        dict(name="plan_prompts_64", kind="plan", n=64, new_lo=1, new_hi=16384, cached_lo=0, cached_hi=4096,
             block_size=16, lens_seed=12),
        # the decode step's keys and values into the cache
        dict(name="append_step_512", kind="append", tokens=512, pad=0, H_kv=8, d=128, block_size=16, dtype="bf16",
             fused=True),
        # a whole prompt batch's keys and values, straight out of the fused projection, with padded tokens at the end
        dict(name="append_prompt_32k", kind="append", tokens=32768, pad=200, H_kv=8, d=128, block_size=16,
             dtype="bf16", fused=True),
        # the smallest prompt: one sequence of 512 tokens, 2 heads, fp32
        dict(name="prefill_tiny_fp32", kind="prefill", n=1, lo=512, hi=512, H=2, H_kv=2, d=64, dtype="fp32",
             fused=False, lens_seed=1),
        # the bench's prompt batch, 4 x 8192 tokens, 32 heads
        dict(name="prefill_4x8k", kind="prefill", n=4, lo=8192, hi=8192, H=32, H_kv=8, d=128, dtype="bf16",
             fused=True, lens_seed=2),
        # ragged prompts of one to 2500 tokens
        dict(name="prefill_ragged_37", kind="prefill", n=37, lo=1, hi=2500, H=16, H_kv=2, d=64, dtype="bf16",
             fused=True, lens_seed=3),
        # prompts resumed behind a cached prefix: keys and values from the paged cache
        dict(name="resume_8", kind="resume", n=8, lo=1, hi=1024, cached_lo=256, cached_hi=4096, H=32, H_kv=8, d=128,
             block_size=16, dtype="bf16", lens_seed=4),
        # a few short requests: latency
        dict(name="decode_small_7", kind="decode", n=7, groups=0, prefix=0, lo=1, hi=700, H=32, H_kv=8, d=128,
             block_size=16, dtype="bf16", lens_seed=5),
        # the decode batch of 512 requests in 8 groups, each behind its own 4096-token prefix
        dict(name="decode_shared_512", kind="decode", n=512, groups=8, prefix=4096, lo=1, hi=2048, H=32, H_kv=8, d=128,
             block_size=16, dtype="bf16", lens_seed=6),
        # one request of 2^20 tokens, 8 heads
        dict(name="decode_long_1m", kind="decode", n=1, groups=0, prefix=0, lo=1048576, hi=1048576, H=8, H_kv=8,
             d=128, block_size=64, dtype="bf16", lens_seed=7),
        # an odd fp32 batch with a short shared prefix
        dict(name="decode_fp32_33", kind="decode", n=33, groups=3, prefix=768, lo=1, hi=900, H=12, H_kv=4, d=64,
             block_size=32, dtype="fp32", lens_seed=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["plan", "append", "prefill", "prefill", "resume", "decode", "decode"])
    c = dict(kind=kind, lens_seed=rng.randrange(1 << 20))
    bs = rng.choice([16, 16, 32, 64, 128, 256])
    if kind == "plan":
        n = _log(rng, 1, 2000)
        c |= dict(n=n, new_lo=0, new_hi=_log(rng, 1, max(1, 400000 // n)), cached_lo=0, cached_hi=_log(rng, 1, 16384),
                  block_size=bs)
        return c
    H_kv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    c |= dict(d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
    small = c["dtype"] == "fp32"
    if kind == "append":
        c |= dict(tokens=_log(rng, 1, 32768), pad=rng.choice([0, rng.randrange(300)]), H_kv=H_kv, block_size=bs,
                  fused=rng.random() < 0.5)
        c.pop("lens_seed")
        return c
    c |= dict(H=H_kv * G, H_kv=H_kv)
    if kind == "prefill":
        n = _log(rng, 1, 40)
        most = min(6000, 24000 // n, int((8e9 / (n * H_kv * G)) ** 0.5)) if not small else min(1500, 8000 // n)
        c |= dict(n=n, lo=1, hi=_log(rng, 1, most), fused=rng.random() < 0.5)
    elif kind == "resume":
        n = _log(rng, 1, 16)
        c |= dict(n=n, lo=1, hi=_log(rng, 1, 700 if not small else 200), cached_lo=0, cached_hi=_log(rng, 256, 4000),
                  block_size=bs)
    else:
        n = _log(rng, 1, 300)
        groups = rng.choice([0, 1, min(n, rng.randrange(1, 9))])
        c |= dict(n=n, groups=groups, prefix=0 if not groups else bs * _log(rng, 1, max(1, 6000 // bs)), lo=0,
                  hi=_log(rng, 1, min(8000, 400000 // n)), block_size=bs)
    return c


# ------------------------------------------------------------------------------------------------ lengths

def _lens(rng, n, lo, hi):
    return [rng.randint(lo, hi) for _ in range(n)]


def _lengths(case):
    """Host lengths of a case: (new or suffix lengths, cached or prefix lengths)."""
    rng = random.Random(case["lens_seed"])
    if case["kind"] == "plan":
        new = _lens(rng, case["n"], case["new_lo"], case["new_hi"])
        return new, _lens(rng, case["n"], case["cached_lo"], case["cached_hi"])
    if case["kind"] == "prefill":
        return _lens(rng, case["n"], case["lo"], case["hi"]), [0] * case["n"]
    if case["kind"] == "resume":
        new = _lens(rng, case["n"], case["lo"], case["hi"])
        return new, [c // 256 * 256 for c in _lens(rng, case["n"], case["cached_lo"], case["cached_hi"])]
    suffix = _lens(rng, case["n"], case["lo"], case["hi"])
    return suffix, [case["prefix"] if case["groups"] else 0] * case["n"]


def _group_start(case):
    """Contiguous groups of nearly equal size."""
    n, g = case["n"], case["groups"]
    return [n * i // g for i in range(g + 1)] if g else []


def _esize(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    if case["kind"] == "plan":
        new, cached = _lengths(case)
        bs, total = case["block_size"], sum(new)
        blocks = sum(-(-(c + t) // bs) - -(-c // bs) for c, t in zip(cached, new))
        return {"bytes": 4 * (2 * case["n"] + 2 * case["n"] + 2 * blocks + 2 * total), "flops": 0}
    if case["kind"] == "append":
        return {"bytes": 4 * case["tokens"] * case["H_kv"] * case["d"] * _esize(case) + 4 * (case["tokens"] + case["pad"]),
                "flops": 0}
    new, old = _lengths(case)
    H, H_kv, d, e = case["H"], case["H_kv"], case["d"], _esize(case)
    if case["kind"] == "decode":
        groups = case["groups"]
        keys = sum(new) + groups * case["prefix"]
        pairs = sum(a + b for a, b in zip(new, old))
        rows, table = case["n"], 4 * sum(-(-(a + b) // case["block_size"]) for a, b in zip(new, old))
    else:
        keys = sum(new) + sum(old)
        pairs = sum(t * c + t * (t + 1) // 2 for t, c in zip(new, old))
        rows = sum(new)
        table = 0 if case["kind"] == "prefill" else 4 * sum(-(-(a + b) // case["block_size"]) for a, b in zip(new, old))
    return {"bytes": 2 * rows * H * d * e + 4 * rows * H + 2 * keys * H_kv * d * e + table, "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _cu(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])


def _qkv(g, T, H, H_kv, d, dtype, fused):
    """q, k, v of a layer: dense tensors, or views of the fused projection's output."""
    if fused:
        x = _randn(g, (T, H + 2 * H_kv, d), dtype)
        x[:, :H] *= 2
        return x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    return _randn(g, (T, H, d), dtype, 2.0), _randn(g, (T, H_kv, d), dtype), _randn(g, (T, H_kv, d), dtype)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    kind = case["kind"]
    s = dict(kind=kind, bs=case.get("block_size"))
    if kind == "plan":
        new, cached = _lengths(case)
        bs, n = case["block_size"], case["n"]
        have = [-(-c // bs) for c in cached]
        need = [-(-(c + t) // bs) for c, t in zip(cached, new)]
        n_blocks = sum(need) + 8
        perm = rng.permutation(n_blocks).astype(np.int32)
        table = np.full((n, max(1, max(need))), -1, dtype=np.int32)
        at = 0
        for i in range(n):
            table[i, :have[i]] = perm[at:at + have[i]]
            at += have[i]
        begin = 3
        free = np.concatenate([np.full(begin, -1, np.int32), perm[at:]])
        s |= dict(cached=_i32(cached, dev), new=_i32(new, dev), table=torch.from_numpy(table).to(dev),
                  free=torch.from_numpy(free).to(dev), begin=_i32([begin], dev), end=_i32([0], dev),
                  n_blocks=n_blocks, max_tokens=sum(new) + 16)
        return s
    d, H_kv, dtype = case["d"], case["H_kv"], _dtype(case)
    if kind == "append":
        bs, T = case["block_size"], case["tokens"]
        n_blocks = -(-T // bs) + 64
        _, k, v = _qkv(g, T + case["pad"], 4 * H_kv if case["fused"] else 1, H_kv, d, dtype, case["fused"])
        # a batch fills most of a few blocks: whole blocks in a random order, padded tokens marked -1
        slots = (rng.permutation(n_blocks)[:, None].astype(np.int64) * bs + np.arange(bs)).reshape(-1)[7:7 + T]
        slots = np.concatenate([slots, np.full(case["pad"], -1, np.int64)]).astype(np.int32)
        s |= dict(k=k, v=v, slots=torch.from_numpy(slots).to(dev),
                  k_cache=_randn(g, (n_blocks, H_kv, bs, d), dtype), v_cache=_randn(g, (n_blocks, H_kv, bs, d), dtype))
        return s
    new, old = _lengths(case)
    H = case["H"]
    s["scale"] = d ** -0.5
    s["kv_max"] = max(1, max(a + b for a, b in zip(new, old)))
    if kind == "prefill":
        q, k, v = _qkv(g, sum(new), H, H_kv, d, dtype, case["fused"])
        s |= dict(q=q, k=k, v=v, cu=_i32(_cu(new).tolist(), dev), q_max=max(new))
        return s
    bs = case["block_size"]
    need = [-(-(a + b) // bs) for a, b in zip(new, old)]
    starts = _group_start(case) if kind == "decode" else []
    shared = case["prefix"] // bs if starts else 0
    n_blocks = sum(need) - shared * (case["n"] - len(starts[1:])) + 3
    perm = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((case["n"], max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for a, b in zip(starts[:-1], starts[1:]):
        table[a:b, :shared] = perm[at:at + shared]
        at += shared
    for i in range(case["n"]):
        table[i, shared:need[i]] = perm[at:at + need[i] - shared]
        at += need[i] - shared
    s |= dict(k_cache=_randn(g, (n_blocks, H_kv, bs, d), dtype), v_cache=_randn(g, (n_blocks, H_kv, bs, d), dtype),
              table=torch.from_numpy(table).to(dev), kv_lens=_i32([a + b for a, b in zip(new, old)], dev))
    if kind == "resume":
        s |= dict(q=_randn(g, (sum(new), H, d), dtype, 2.0), cu=_i32(_cu(new).tolist(), dev), q_max=max(new))
    else:
        s |= dict(q=_randn(g, (case["n"], H, d), dtype, 2.0),
                  group_start=_i32(starts, dev) if starts else None,
                  prefix_lens=_i32([case["prefix"]] * case["groups"], dev) if starts else None)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_plan(s):
    bs, T = s["bs"], s["max_tokens"]
    cached, new = s["cached"].long(), s["new"].long()
    kv = cached + new
    have, need = (cached + bs - 1) // bs, (kv + bs - 1) // bs
    taken = need - have
    first = s["begin"].long() + taken.cumsum(0) - taken
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    j = torch.arange(s["table"].shape[1], device=kv.device)
    fresh = (j >= have[:, None]) & (j < need[:, None])
    ids = s["free"][(first[:, None] + j - have[:, None]).clamp(0, s["free"].numel() - 1)]
    s["table"].copy_(torch.where(fresh, ids, s["table"]))
    t = torch.arange(T, device=kv.device)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=kv.numel() - 1)
    pos = cached[seq] + t - cu[seq]
    live = t < cu[-1]
    block = s["table"][seq, (pos // bs).clamp(max=s["table"].shape[1] - 1)].long()
    slot = torch.where(live, block * bs + pos % bs, torch.full_like(pos, -1))
    return dict(block_table=s["table"], kv_lens=kv.int(), cu_seqlens=cu.int(), slot_map=slot.int(),
                positions=torch.where(live, pos, torch.full_like(pos, -1)).int(),
                free_end=(s["begin"].long() + taken.sum()).int())


def _plain_append(s):
    live = s["slots"] >= 0
    slot = torch.where(live, s["slots"], torch.zeros_like(s["slots"])).long()
    block, off = slot // s["bs"], slot % s["bs"]
    last = s["slots"][0].long()                       # padded tokens rewrite token 0's row with itself
    block = torch.where(live, block, last // s["bs"])
    off = torch.where(live, off, last % s["bs"])
    for new, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        cache[block, :, off] = torch.where(live[:, None, None], new, new[:1])
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attention(q, k, v, first, kv_lens, scale):
    """q [n, L, H, d], k, v [n, H_kv, K, d] in fp32; query i of sequence s sees the keys j <= first[s] + i, j < kv_lens[s].
    Returns o [n, L, H, d] and lse [n, L, H] in fp32; a row that sees nothing gives zeros and -inf."""
    n, L, H, d = q.shape
    H_kv, K = k.shape[1], k.shape[2]
    G = H // H_kv
    qg = (q * scale).reshape(n, L, H_kv, G, d).permute(0, 2, 3, 1, 4).reshape(n, H_kv, G * L, d)
    x = (qg @ k.transpose(2, 3)).view(n, H_kv, G, L, K)
    j = torch.arange(K, device=q.device)
    last = first[:, None] + torch.arange(L, device=q.device)
    seen = (j <= last[:, :, None]) & (j < kv_lens[:, None, None])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(n, H_kv, G * L, K) @ v).view(n, H_kv, G, L, d) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + total.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(n, L, H, d), lse.permute(0, 3, 1, 2).reshape(n, L, H)


def _paged(cache, table, bs, K):
    """[n, H_kv, K, d] in fp32 from the cache."""
    blocks = table[:, :-(-K // bs)].clamp(min=0).long()
    x = cache[blocks].transpose(1, 2)                  # [n, H_kv, blocks, bs, d]
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :K].float()


def _plain_prompt(s, k, v, kv_lens):
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.arange(s["q_max"], device=cu.device)).clamp(max=s["q"].shape[0] - 1)
    kv_lens = lens if kv_lens is None else kv_lens.long()
    if k is None:
        k, v = (x[at].transpose(1, 2).float() for x in (s["k"], s["v"]))
    o, lse = _plain_attention(s["q"][at].float(), k, v, kv_lens - lens, kv_lens, s["scale"])
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return dict(o=o[seq, t - cu[seq]].to(s["q"].dtype), lse=lse[seq, t - cu[seq]])


def _run_plain(s):
    kind = s["kind"]
    if kind == "plan":
        return _plain_plan(s)
    if kind == "append":
        return _plain_append(s)
    if kind == "prefill":
        return _plain_prompt(s, None, None, None)
    k, v = (_paged(c, s["table"], s["bs"], s["kv_max"]) for c in (s["k_cache"], s["v_cache"]))
    if kind == "resume":
        return _plain_prompt(s, k, v, s["kv_lens"])
    kv = s["kv_lens"].long()
    o, lse = _plain_attention(s["q"][:, None].float(), k, v, kv - 1, kv, s["scale"])
    return dict(o=o[:, 0].to(s["q"].dtype), lse=lse[:, 0])


def run(s):
    if not own:
        return _run_plain(s)
    import hybrid_linear_attention_kda_gb300 as kda
    kind = s["kind"]
    if kind == "plan":
        p = kda.cache_plan(s["cached"], s["new"], s["table"], s["free"], s["begin"], s["end"], block_size=s["bs"],
                           n_blocks=s["n_blocks"], max_tokens=s["max_tokens"])
        return dict(block_table=s["table"], kv_lens=p.kv_lens, cu_seqlens=p.cu_seqlens, slot_map=p.slot_map,
                    positions=p.positions, free_end=s["end"])
    if kind == "append":
        kda.kda_cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if kind == "prefill":
        o, lse = kda.attn_prefill(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], want_lse=True)
    elif kind == "resume":
        o, lse = kda.attn_prefill_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu"],
                                        scale=s["scale"], want_lse=True)
    else:
        o, lse = kda.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                                 group_start=s["group_start"], prefix_lens=s["prefix_lens"], scale=s["scale"],
                                 want_lse=True)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_rows(q, keys, values, scale, first):
    """Softmax attention of one sequence in float64.  q [L, H, d], keys, values [K, H_kv, d]; row i sees keys
    0 .. first + i.  Walks the queries in blocks, each against the keys that its last row sees."""
    L, H, d = q.shape
    H_kv = keys.shape[1]
    o = torch.zeros((L, H, d), dtype=torch.float64, device=q.device)
    lse = torch.full((L, H), float("-inf"), dtype=torch.float64, device=q.device)
    step = max(1, min(1024, (1 << 29) // max(1, keys.shape[0] * H)))
    for a in range(0, L, step):
        b = min(L, a + step)
        K = min(keys.shape[0], first + b)
        if K <= 0:
            continue
        for h in range(H_kv):
            heads = slice(h * (H // H_kv), (h + 1) * (H // H_kv))
            x = torch.einsum("lgd,kd->glk", q[a:b, heads].double(), keys[:K, h].double()) * scale
            hidden = torch.arange(K, device=q.device)[None] > first + torch.arange(a, b, device=q.device)[:, None]
            x[:, hidden] = float("-inf")
            z = torch.logsumexp(x, -1)
            lse[a:b, heads] = z.T
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[a:b, heads] = torch.einsum("glk,kd->lgd", p, values[:K, h].double())
    return o, lse


def _exact_plan(s):
    bs = s["bs"]
    cached, new = s["cached"].cpu().tolist(), s["new"].cpu().tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    take = int(s["begin"].cpu()[0])
    cu, slots, positions = [0], [], []
    for i, (c, t) in enumerate(zip(cached, new)):
        for j in range(-(-c // bs), -(-(c + t) // bs)):
            table[i, j] = free[take]
            take += 1
        pos = np.arange(c, c + t)
        positions.append(pos)
        slots.append(table[i, pos // bs].astype(np.int64) * bs + pos % bs)
        cu.append(cu[-1] + t)
    rest = np.full(s["max_tokens"] - cu[-1], -1)
    return dict(block_table=table, kv_lens=np.array([c + t for c, t in zip(cached, new)], np.int32),
                cu_seqlens=np.array(cu, np.int32), slot_map=np.concatenate(slots + [rest]).astype(np.int32),
                positions=np.concatenate(positions + [rest]).astype(np.int32), free_end=np.array([take], np.int32))


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "plan":
        return _exact_plan(s)
    if kind == "append":
        slots = s["slots"].cpu().numpy()
        at = torch.from_numpy(np.nonzero(slots >= 0)[0]).to(s["k"].device)
        slot = s["slots"][at].long()
        out = {}
        for name, new in (("k_cache", s["k"]), ("v_cache", s["v"])):
            n_blocks, H_kv, bs, d = s[name].shape
            flat = s[name].double().permute(0, 2, 1, 3).reshape(n_blocks * bs, H_kv, d)
            flat[slot] = new[at].double()
            out[name] = flat.view(n_blocks, bs, H_kv, d).permute(0, 2, 1, 3).contiguous()
        return out
    new, old = _lengths(case)
    if kind == "decode":
        cu, lens = list(range(case["n"] + 1)), [a + b for a, b in zip(new, old)]
    else:
        cu, lens = _cu(new).tolist(), [a + b for a, b in zip(new, old)]
    o, lse = [], []
    for i, K in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        if kind == "prefill":
            keys, values = s["k"][a:b], s["v"][a:b]
        else:
            blocks = s["table"][i, :-(-K // s["bs"])].long()
            keys, values = (c[blocks].permute(0, 2, 1, 3).reshape(-1, c.shape[1], c.shape[3])[:K]
                            for c in (s["k_cache"], s["v_cache"]))
        x, z = _exact_rows(s["q"][a:b], keys, values, s["scale"], K - (b - a))
        o.append(x)
        lse.append(z)
    return dict(o=torch.cat(o), lse=torch.cat(lse))
