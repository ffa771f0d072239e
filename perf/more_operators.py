"""Cases of the operators around the softmax-attention cache: norms of queries and keys for each head with the position
rotation in the same pass, the same on the way into the paged cache, and a cache held in 4 bits: its append, its read-back
into a full-width cache, and decode attention over it, behind full-width prefixes that several requests share.

Shapes.  q [T, H, d]; k, v [T, H_kv, d]; caches [n_blocks, H_kv, block_size, d]; slot = block * block_size + offset inside
the block.  The 4-bit cache has two tensors each for keys and values: codes uint8 [n_blocks, H_kv, block_size, d / 2]
(channel 2 i in the low half of byte i) and scales bf16 [n_blocks, H_kv, block_size, d / 64, 2], (s, m) for each group of 64
channels, so that a channel's value is m + code * s.

Lengths come from the case itself (`lens_seed`), values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 512 requests, out of the fused projection: norms and rotation before the attention
        dict(name="norm_rope_step_512", kind="norm_rope", tokens=512, pad=0, H=32, H_kv=8, d=128, rot=128,
             interleaved=False, norm=True, fused=True, dtype="bf16", pos_hi=16384, lens_seed=31),
        # a whole prompt batch, at positions up to a million
        dict(name="norm_rope_prompt_32k", kind="norm_rope", tokens=32768, pad=200, H=32, H_kv=8, d=128, rot=128,
             interleaved=False, norm=True, fused=True, dtype="bf16", pos_hi=1 << 20, lens_seed=32),
        # the decode step's queries, keys and values in one pass: rotated, and into the cache
        dict(name="append_rope_step_512", kind="append_rope", tokens=512, pad=0, H=32, H_kv=8, d=128, rot=128,
             interleaved=False, norm=True, fused=True, dtype="bf16", pos_hi=16384, block_size=16, lens_seed=33),
        # a prompt batch in fp32 whose heads are rotated in half of their channels, adjacent pairs, without norms
        dict(name="append_rope_prompt_fp32", kind="append_rope", tokens=7001, pad=37, H=16, H_kv=2, d=64, rot=32,
             interleaved=True, norm=False, fused=False, dtype="fp32", pos_hi=8192, block_size=64, lens_seed=34),
        # the decode step's keys and values into the 4-bit cache
        dict(name="append_q4_step_512", kind="append_q4", tokens=512, pad=0, H_kv=8, d=128, block_size=16, dtype="bf16",
             fused=True, lens_seed=35),
        # a prompt batch's, with the values that the cache now stands for, which its own attention then sees
        dict(name="append_q4_prompt_32k", kind="append_q4", tokens=32768, pad=200, H_kv=8, d=128, block_size=16,
             dtype="bf16", fused=True, lens_seed=36),
        # a few short fp32 requests read back before their next prompt
        dict(name="unpack_q4_5_fp32", kind="unpack_q4", n=5, first_hi=40, lo=1, hi=300, H_kv=2, d=64, block_size=16,
             dtype="fp32", lens_seed=37),
        # 24 conversations of up to 16384 tokens read back before their next prompts
        dict(name="unpack_q4_24x16k", kind="unpack_q4", n=24, first_hi=0, lo=1, hi=16384, H_kv=8, d=128, block_size=64,
             dtype="bf16", lens_seed=38),
        # a handful of short requests, no sharing: latency
        dict(name="decode_q4_7_short", kind="decode_q4", n=7, groups=0, prefix=0, lo=1, hi=700, H=32, H_kv=8, d=128,
             block_size=16, dtype="bf16", lens_seed=39),
        # 512 requests behind 8 shared system prompts of 4096 tokens, own tokens up to 2048 in 4 bits
        dict(name="decode_q4_512_prefix", kind="decode_q4", n=512, groups=8, prefix=4096, lo=1, hi=2048, H=32, H_kv=8,
             d=128, block_size=64, dtype="bf16", lens_seed=40),
        # one request a million tokens long
        dict(name="decode_q4_one_million", kind="decode_q4", n=1, groups=0, prefix=0, lo=1 << 20, hi=1 << 20, H=32,
             H_kv=8, d=128, block_size=64, dtype="bf16", lens_seed=41),
        # a small model in fp32 behind three shared prompts
        dict(name="decode_q4_33_fp32", kind="decode_q4", n=33, groups=3, prefix=768, lo=0, hi=2000, H=12, H_kv=4, d=64,
             block_size=32, dtype="fp32", lens_seed=42),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["norm_rope", "append_rope", "append_q4", "unpack_q4", "decode_q4", "decode_q4", "decode_q4"])
    d, H_kv = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8])
    H = H_kv * rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    c = dict(kind=kind, d=d, H_kv=H_kv, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]), lens_seed=rng.randrange(1 << 20))
    bs = rng.choice([16, 16, 32, 64, 128, 256])
    if kind != "norm_rope":
        c |= dict(block_size=bs)
    if kind in ("norm_rope", "append_rope"):
        c |= dict(tokens=_log(rng, 1, min(32768, int(1.5e8) // ((H + 2 * H_kv) * d))), pad=rng.choice([0, rng.randrange(300)]),
                  H=H, rot=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                  fused=rng.random() < 0.6, pos_hi=_log(rng, 100, 1 << 21))
    elif kind == "append_q4":
        c |= dict(tokens=_log(rng, 1, 32768), pad=rng.choice([0, rng.randrange(300)]), fused=rng.random() < 0.6)
    elif kind == "unpack_q4":
        n = _log(rng, 1, 200)
        c |= dict(n=n, first_hi=rng.choice([0, 0, 500]), lo=0, hi=_log(rng, 1, min(16384, 300000 // n)))
    else:
        n = _log(rng, 1, 300)
        groups = rng.choice([0, 0, 1, min(n, rng.randrange(1, 9))])
        c |= dict(n=n, groups=groups, prefix=0 if not groups else bs * _log(rng, 1, max(1, 6000 // bs)), lo=0, H=H,
                  hi=_log(rng, 1, min(30000, 400000 // n)))
    return c


def _lengths(case):
    """Host lengths of a case: (own or read positions, first read position or shared prefix)."""
    rng = random.Random(case["lens_seed"])
    own_lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    if case["kind"] == "unpack_q4":
        return own_lens, [rng.randint(0, case["first_hi"]) for _ in range(case["n"])]
    return own_lens, [case["prefix"] if case["groups"] else 0] * case["n"]


def _group_start(case):
    """Contiguous groups of nearly equal size."""
    n, g = case["n"], case["groups"]
    return [n * i // g for i in range(g + 1)] if g else []


def _esize(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    kind, H_kv, d, e = case["kind"], case["H_kv"], case["d"], _esize(case)
    q4 = d // 2 + d // GROUP * 4                       # bytes of a head's vector in the 4-bit cache
    if kind in ("norm_rope", "append_rope"):
        T, rows = case["tokens"], case["H"] + (1 if kind == "norm_rope" else 2) * H_kv
        turned = case["H"] + H_kv
        return {"bytes": 2 * T * rows * d * e + (4 if kind == "norm_rope" else 8) * (T + case["pad"]),
                "flops": T * turned * ((4 * d if case["norm"] else 0) + 3 * case["rot"])}
    if kind == "append_q4":
        T = case["tokens"]
        return {"bytes": 2 * T * H_kv * (2 * d * e + q4) + 4 * (T + case["pad"]), "flops": 6 * 2 * T * H_kv * d}
    own_lens, other = _lengths(case)
    if kind == "unpack_q4":
        K = sum(max(0, a - b) for a, b in zip(own_lens, other))
        return {"bytes": 2 * K * H_kv * (q4 + d * e) + 8 * case["n"], "flops": 2 * 2 * K * H_kv * d}
    pairs = sum(a + b for a, b in zip(own_lens, other))
    table = 4 * sum(-(-(a + b) // case["block_size"]) for a, b in zip(own_lens, other))
    return {"bytes": 2 * case["n"] * case["H"] * d * e + 4 * case["n"] * case["H"] + table
            + 2 * H_kv * (sum(own_lens) * q4 + case["groups"] * case["prefix"] * d * e), "flops": 4 * d * case["H"] * pairs}


# ------------------------------------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def _i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def _qkv(g, T, H, H_kv, d, dtype, fused):
    """q, k, v of a layer: dense tensors, or views of the fused projection's output."""
    if fused:
        x = _randn(g, (T, H + 2 * H_kv, d), dtype)
        return x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    return _randn(g, (T, H, d), dtype), _randn(g, (T, H_kv, d), dtype), _randn(g, (T, H_kv, d), dtype)


def _slots(rng, T, pad, bs):
    """A batch's slots: most of a few blocks, whole blocks in a random order; padded tokens are -1."""
    n_blocks = -(-T // bs) + 64
    slots = (rng.permutation(n_blocks)[:, None].astype(np.int64) * bs + np.arange(bs)).reshape(-1)[7:7 + T]
    return np.concatenate([slots, np.full(pad, -1)]).astype(np.int32), n_blocks


def _bits_toward(x, up):
    """x (fp32) rounded to bf16 towards +inf or -inf."""
    i = x.contiguous().view(torch.int32)
    away = (x > 0) if up else (x < 0)                  # magnitudes grow in this direction
    return (torch.where(away, i + 0xFFFF, i) & -0x10000).view(torch.float32)


def _quantize(x):
    """(codes uint8 [..., d / 2], scales bf16 [..., d / 64, 2]) of x [..., d]: fp32 arithmetic, each step rounded to nearest
    but for m (down) and s (up) to bf16.  A group that is not finite, or as wide as fp32, has s = 0 and m = NaN."""
    y = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    m = _bits_toward(lo, False)
    s = _bits_toward((hi - m) / torch.full_like(m, 15), True)      # by a tensor: by a number it is a product on the GPU
    fine = torch.isfinite(y).all(-1, keepdim=True) & torch.isfinite(m) & torch.isfinite(hi - m) & torch.isfinite(s)
    code = torch.round((y - m) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15)
    code = torch.where(fine & (s > 0), code, torch.zeros_like(code)).to(torch.uint8).flatten(-2)
    m, s = torch.where(fine, m, torch.full_like(m, float("nan"))), torch.where(fine, s, torch.zeros_like(s))
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([s, m], -1).to(torch.bfloat16)


def _values(codes, scales):
    """The fp32 values of codes [..., d / 2] and scales [..., d / 64, 2]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    s = scales.float()
    return n.mul_(s[..., :1]).add_(s[..., 1:]).flatten(-2)


def _q4_cache(g, shape):
    """Codes and scales of normally distributed keys or values of this shape."""
    n, H_kv, bs, d = shape
    codes = torch.empty((n, H_kv, bs, d // 2), dtype=torch.uint8, device=g.device)
    scales = torch.empty((n, H_kv, bs, d // GROUP, 2), dtype=torch.bfloat16, device=g.device)
    step = max(1, (1 << 26) // (H_kv * bs * d))
    for a in range(0, n, step):
        codes[a:a + step], scales[a:a + step] = _quantize(_randn(g, (min(step, n - a), H_kv, bs, d), torch.bfloat16))
    return codes, scales


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    kind, d, H_kv, dtype = case["kind"], case["d"], case["H_kv"], _dtype(case)
    s = dict(kind=kind, bs=case.get("block_size"))
    if kind in ("norm_rope", "append_rope"):
        T, pad, H, R = case["tokens"], case["pad"], case["H"], case["rot"]
        q, k, v = _qkv(g, T + pad, H, H_kv, d, dtype, case["fused"])
        freq = [10000.0 ** (-2 * i / R) for i in range(R // 2)]
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) for f in freq]
        pos = np.concatenate([rng.randint(0, case["pos_hi"], T), np.full(pad, -1)])
        s |= dict(q=q, k=k, positions=_i32(pos, dev), inv_freq=torch.tensor(freq, dtype=torch.float64, device=dev),
                  turns=torch.tensor(turns, dtype=torch.int64, device=dev), interleaved=case["interleaved"], eps=1e-6,
                  q_out=torch.zeros((T + pad, H, d), dtype=dtype, device=dev))
        s |= dict(q_weight=1 + _randn(g, (d,), torch.float32, 0.1) if case["norm"] else None,
                  k_weight=1 + _randn(g, (d,), torch.float32, 0.1) if case["norm"] else None)
        if kind == "norm_rope":
            s |= dict(k_out=torch.zeros((T + pad, H_kv, d), dtype=dtype, device=dev))
            return s
        slots, n_blocks = _slots(rng, T, pad, case["block_size"])
        s |= dict(v=v, slots=_i32(slots, dev), k_cache=_randn(g, (n_blocks, H_kv, case["block_size"], d), dtype),
                  v_cache=_randn(g, (n_blocks, H_kv, case["block_size"], d), dtype))
        return s
    bs = case["block_size"]
    if kind == "append_q4":
        T, pad = case["tokens"], case["pad"]
        _, k, v = _qkv(g, T + pad, 4 * H_kv if case["fused"] else 1, H_kv, d, dtype, case["fused"])
        slots, n_blocks = _slots(rng, T, pad, bs)
        kc, vc = (_q4_cache(g, (n_blocks, H_kv, bs, d)) for _ in range(2))
        s |= dict(k=k, v=v, slots=_i32(slots, dev), k_codes=kc[0], k_scales=kc[1], v_codes=vc[0], v_scales=vc[1],
                  k_out=torch.zeros((T + pad, H_kv, d), dtype=dtype, device=dev),
                  v_out=torch.zeros((T + pad, H_kv, d), dtype=dtype, device=dev))
        return s
    own_lens, other = _lengths(case)
    total = own_lens if kind == "unpack_q4" else [a + b for a, b in zip(own_lens, other)]
    need = [-(-t // bs) for t in total]
    starts = _group_start(case) if kind == "decode_q4" else []
    shared = case["prefix"] // bs if starts else 0
    n_blocks = sum(need) - shared * case["n"] + 3
    perm = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((case["n"], max(1, max(need))), -1, dtype=np.int32)
    order = rng.permutation(shared * len(starts[1:]) + 1).astype(np.int32)      # blocks of the full-width prefixes
    for i, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        table[a:b, :shared] = order[i * shared:(i + 1) * shared]
    at = 0
    for i in range(case["n"]):
        table[i, shared:need[i]] = perm[at:at + need[i] - shared]
        at += need[i] - shared
    kc, vc = (_q4_cache(g, (n_blocks, H_kv, bs, d)) for _ in range(2))
    s |= dict(k_codes=kc[0], k_scales=kc[1], v_codes=vc[0], v_scales=vc[1], table=torch.from_numpy(table).to(dev),
              kv_lens=_i32(total, dev), longest=max(total))
    if kind == "unpack_q4":
        wide = sum(need) + 5
        to = np.full_like(table, -1)
        order, at = rng.permutation(wide).astype(np.int32), 0
        for i in range(case["n"]):
            to[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
        s |= dict(to_table=torch.from_numpy(to).to(dev), first=_i32(other, dev) if case["first_hi"] else None,
                  k_cache=_randn(g, (wide, H_kv, bs, d), dtype), v_cache=_randn(g, (wide, H_kv, bs, d), dtype))
        return s
    s |= dict(q=_randn(g, (case["n"], case["H"], d), dtype, 2.0), scale=d ** -0.5, prefix=shared * bs,
              group_start=_i32(starts, dev) if starts else None,
              prefix_lens=_i32([case["prefix"]] * case["groups"], dev) if starts else None,
              k_prefix=_randn(g, (len(order), H_kv, bs, d), dtype) if starts else None,
              v_prefix=_randn(g, (len(order), H_kv, bs, d), dtype) if starts else None)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _angles(s):
    """cos and sin [T, 1, R / 2] in fp32, of angles formed in fp64: positions are large."""
    x = s["positions"].double()[:, None, None] * s["inv_freq"]
    return x.cos().float(), x.sin().float()


def _turned(x, weight, cos, sin, eps, interleaved):
    """x [T, heads, d], normed and rotated in fp32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if interleaved else -2).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _scatter(cache, slots, bs, new):
    """cache[slots] = new [T, H_kv, ...] where the slot is not -1, without a copy to the host: a padded token writes the
    first token's row again."""
    slot = torch.where(slots >= 0, slots, slots[0]).long()
    live = (slots >= 0).view(-1, *[1] * (new.dim() - 1))
    cache[slot // bs, :, slot % bs] = torch.where(live, new, new[:1]).to(cache.dtype)


def _plain_norm_rope(s):
    cos, sin = _angles(s)
    live = (s["positions"] >= 0)[:, None, None]
    q = _turned(s["q"], s["q_weight"], cos, sin, s["eps"], s["interleaved"]).to(s["q"].dtype)
    k = _turned(s["k"], s["k_weight"], cos, sin, s["eps"], s["interleaved"]).to(s["k"].dtype)
    s["q_out"].copy_(torch.where(live, q, s["q_out"]))
    if s["kind"] == "norm_rope":
        s["k_out"].copy_(torch.where(live, k, s["k_out"]))
        return dict(q=s["q_out"], k=s["k_out"])
    _scatter(s["k_cache"], s["slots"], s["bs"], k)
    _scatter(s["v_cache"], s["slots"], s["bs"], s["v"])
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_append_q4(s):
    live = (s["slots"] >= 0)[:, None, None]
    out = {}
    for x in ("k", "v"):
        codes, scales = _quantize(s[x])
        _scatter(s[x + "_codes"], s["slots"], s["bs"], codes)
        _scatter(s[x + "_scales"], s["slots"], s["bs"], scales)
        s[x + "_out"].copy_(torch.where(live, _values(codes, scales).to(s[x].dtype), s[x + "_out"]))
        out |= {x: s[x + "_out"], x + "_codes": s[x + "_codes"], x + "_scales": s[x + "_scales"]}
    return out


def _plain_unpack_q4(s):
    bs = s["bs"]
    p = torch.arange(s["table"].shape[1] * bs, device=s["table"].device)
    seen = p < s["kv_lens"][:, None]
    if s["first"] is not None:
        seen = seen & (p >= s["first"][:, None])
    seq, pos = seen.nonzero(as_tuple=True)
    off = pos % bs
    block, to = s["table"][seq, pos // bs].long(), s["to_table"][seq, pos // bs].long()
    for x in ("k", "v"):
        s[x + "_cache"][to, :, off] = _values(s[x + "_codes"][block, :, off], s[x + "_scales"][block, :, off]).to(s[x + "_cache"].dtype)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _paged(s, x):
    """[n, H_kv, K, d] in fp32: the shared prefix out of the full-width cache, the rest out of the 4-bit one."""
    shared = s["prefix"] // s["bs"]
    blocks = s["table"].clamp(min=0).long()
    parts = [s[x + "_prefix"][blocks[:, :shared]].float()] if shared else []
    if blocks.shape[1] > shared:
        parts.append(_values(s[x + "_codes"][blocks[:, shared:]], s[x + "_scales"][blocks[:, shared:]]))
    y = torch.cat(parts, 1).transpose(1, 2)            # [n, H_kv, blocks, bs, d]
    return y.reshape(y.shape[0], y.shape[1], -1, y.shape[-1])[:, :, :max(1, s["longest"])]


def _plain_decode_q4(s):
    n, H, d = s["q"].shape
    k = _paged(s, "k")
    H_kv, K = k.shape[1], k.shape[2]
    x = (s["q"].float() * s["scale"]).view(n, H_kv, H // H_kv, d) @ k.transpose(2, 3)
    x.masked_fill_((torch.arange(K, device=x.device) >= s["kv_lens"][:, None])[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ _paged(s, "v")) / torch.where(total == 0, torch.ones_like(total), total)
    return dict(o=o.view(n, H, d).to(s["q"].dtype), lse=(m + total.log()).view(n, H))


def run(s):
    kind = s["kind"]
    if not own:
        return (_plain_norm_rope(s) if kind in ("norm_rope", "append_rope") else _plain_append_q4(s) if kind == "append_q4"
                else _plain_unpack_q4(s) if kind == "unpack_q4" else _plain_decode_q4(s))
    import hybrid_linear_attention_kda_gb300 as kda
    if kind == "norm_rope":
        q, k = kda.qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], interleaved=s["interleaved"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], q_out=s["q_out"],
                                k_out=s["k_out"])
        return dict(q=q, k=k)
    if kind == "append_rope":
        q = kda.cache_append_rope(s["k"], s["v"], s["positions"], s["turns"], s["slots"], s["k_cache"], s["v_cache"],
                                  q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"], q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], eps=s["eps"])
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    cache = kda.Q4Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    if kind == "append_q4":
        k, v = kda.cache_append_q4(s["k"], s["v"], s["slots"], cache, k_out=s["k_out"], v_out=s["v_out"])
        return dict(k=k, v=v, k_codes=cache.k_codes, k_scales=cache.k_scales, v_codes=cache.v_codes, v_scales=cache.v_scales)
    if kind == "unpack_q4":
        kda.cache_unpack_q4(cache, s["table"], s["kv_lens"], s["k_cache"], s["v_cache"], s["to_table"], first=s["first"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    o, lse = kda.attn_decode_q4(s["q"], cache, s["table"], s["kv_lens"], k_prefix=s["k_prefix"], v_prefix=s["v_prefix"],
                                group_start=s["group_start"], prefix_lens=s["prefix_lens"], scale=s["scale"], want_lse=True)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_turned(x, weight, pos, freq, eps, interleaved):
    """Norm, then each pair as one complex number times e^(i angle)."""
    T, heads, d = x.shape
    R = 2 * freq.numel()
    y = torch.empty((T, heads, d), dtype=torch.float64, device=x.device)
    for a in range(0, T, 4096):
        part = x[a:a + 4096].double()
        if weight is not None:
            part = part / torch.sqrt(part.square().sum(-1, keepdim=True) / d + eps) * weight.double()
        pair = part[..., :R].reshape(-1, heads, R // 2, 2) if interleaved else part[..., :R].reshape(-1, heads, 2, R // 2).transpose(-1, -2)
        angle = pos[a:a + 4096].double()[:, None, None] * freq
        z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle)
        z = torch.view_as_real(z)
        part[..., :R] = (z if interleaved else z.transpose(-1, -2)).reshape(-1, heads, R)
        y[a:a + 4096] = part
    return y


def _exact_rows(s, x):
    """Codes, scales and values of the 4-bit append of the tokens x, in numpy; the roundings that the definition names are
    made with numpy's fp32."""
    f = np.float32
    rows = x.float().cpu().numpy().astype(f)
    T, H, d = rows.shape
    y = rows.reshape(T, H, d // GROUP, GROUP)
    lo, hi = y.min(-1), y.max(-1)

    def coarse(v, up):                                 # to bf16 along the real line, by its neighbours
        near = torch.from_numpy(np.ascontiguousarray(v)).to(torch.bfloat16)
        i = near.view(torch.int16).numpy().astype(np.int64)
        w = near.float().numpy()
        over = (w < v) if up else (w > v)
        step = np.where((i >= 0) == up, 1, -1)         # the next one in that direction, by its bits
        i = np.where(over, i + step, i).astype(np.int16)
        return torch.from_numpy(i).view(torch.bfloat16).float().numpy()

    m = coarse(lo, False)
    s_ = coarse(((hi - m).astype(f) / f(15)).astype(f), True)
    div = np.where(s_ > 0, s_, f(1))[..., None]
    code = np.clip(np.rint(((y - m[..., None]).astype(f) / div).astype(f)), 0, 15) * (s_ > 0)[..., None]
    value = code.astype(np.float64) * s_[..., None].astype(np.float64) + m[..., None].astype(np.float64)
    flat = code.reshape(T, H, d).astype(np.uint8)
    return flat[..., 0::2] + 16 * flat[..., 1::2], np.stack([s_, m], -1).astype(np.float64), value.reshape(T, H, d)


def _written(cache, slots, bs, rows):
    """The cache [n_blocks, H_kv, bs, ...] in float64 (or whole numbers) after rows have gone to their slots."""
    flat = cache.transpose(1, 2).reshape(-1, cache.shape[1], *cache.shape[3:])
    flat = flat.double() if cache.is_floating_point() else flat.clone()
    at = (slots >= 0).nonzero()[:, 0]
    flat[slots[at].long()] = rows[at].to(flat.dtype)
    return flat.view(cache.shape[0], bs, *flat.shape[1:]).transpose(1, 2).contiguous()


def _exact_values(codes, scales):
    n = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=codes.device)
    n[..., 0::2], n[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    s = scales.double().repeat_interleave(GROUP, -2)
    return s[..., 1] + n * s[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    kind, bs = s["kind"], s["bs"]
    if kind in ("norm_rope", "append_rope"):
        how = (s["positions"], s["inv_freq"], s["eps"], s["interleaved"])
        q, k = (_exact_turned(s[x], s[x + "_weight"], *how) for x in ("q", "k"))
        live = (s["positions"] >= 0)[:, None, None]
        q = q * live
        if kind == "norm_rope":
            return dict(q=q, k=k * live)
        return dict(q=q, k_cache=_written(s["k_cache"], s["slots"], bs, k), v_cache=_written(s["v_cache"], s["slots"], bs, s["v"]))
    if kind == "append_q4":
        out, dev = {}, s["k"].device
        live = (s["slots"] >= 0)[:, None, None]
        for x in ("k", "v"):
            codes, scales, values = (torch.from_numpy(a).to(dev) for a in _exact_rows(s, s[x]))
            out |= {x: values * live, x + "_codes": _written(s[x + "_codes"], s["slots"], bs, codes),
                    x + "_scales": _written(s[x + "_scales"], s["slots"], bs, scales)}
        return out
    table, lens = s["table"].cpu().tolist(), s["kv_lens"].cpu().tolist()
    if kind == "unpack_q4":
        first = s["first"].cpu().tolist() if s["first"] is not None else [0] * case["n"]
        to, out = s["to_table"].cpu().tolist(), {}
        for x in ("k", "v"):
            wide = s[x + "_cache"].double()
            for i in range(case["n"]):
                for j in range(first[i] // bs, -(-lens[i] // bs)):
                    a, b = max(0, first[i] - j * bs), min(bs, lens[i] - j * bs)
                    if a < b:
                        wide[to[i][j], :, a:b] = _exact_values(s[x + "_codes"][table[i][j], :, a:b], s[x + "_scales"][table[i][j], :, a:b])
            out[x + "_cache"] = wide
        return out
    n, H, d = s["q"].shape
    H_kv = s["k_codes"].shape[1]
    o = torch.zeros((n, H, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((n, H), float("-inf"), dtype=torch.float64, device=s["q"].device)
    for i in range(n):
        K, shared = lens[i], s["prefix"] // bs
        if K == 0:
            continue
        blocks = s["table"][i, :-(-K // bs)].long()
        kv = []
        for x in ("k", "v"):
            y = _exact_values(s[x + "_codes"][blocks[shared:]], s[x + "_scales"][blocks[shared:]])
            y = torch.cat([s[x + "_prefix"][blocks[:shared]].double(), y]) if shared else y
            kv.append(y.transpose(1, 2).reshape(-1, H_kv, d)[:K])
        q = s["q"][i].double().view(H_kv, H // H_kv, d)
        x = torch.einsum("hgd,khd->hgk", q, kv[0]) * s["scale"]
        z = torch.logsumexp(x, -1)
        lse[i] = z.reshape(H)
        o[i] = torch.einsum("hgk,khd->hgd", torch.exp(x - z[..., None]), kv[1]).reshape(H, d)
    return dict(o=o, lse=lse)
