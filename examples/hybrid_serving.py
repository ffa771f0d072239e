"""A small hybrid stack served with the library: KDA layers with a fixed-size state per
request, interleaved with softmax-attention layers over a paged cache, for requests that
share one system prompt.

The system prompt runs once; its cache blocks and its KDA state are what the requests start
from.  Their prompts run as one packed batch behind it.  Then one decode step is captured in
a CUDA graph and replayed per token: the plan, the appends, the attention with the shared
prefix read once, and the KDA updates, with the lengths and the free list advancing on the
device.  ``--check`` recomputes every request from its first token, without cache, states or
sharing, and compares the hidden states.

    python examples/hybrid_serving.py --requests 16 --steps 32 --check
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_linear_attention_kda_gb300 as kda  # noqa: E402

UNIT = 256          # a KDA prefill resumes at a multiple of this many tokens


class HybridStack:
    """``pattern`` gives each layer's kind: "k" is KDA, "a" softmax attention, with norms of its
    queries and keys and a position rotation if ``rope``.  Random weights; the projections are
    plain matrix products, and there are no feed-forward layers."""

    def __init__(self, pattern="kkka", heads=8, kv_heads=2, d=128, dtype=torch.bfloat16, device="cuda", seed=0, rope=False):
        gen = torch.Generator(device).manual_seed(seed)
        self.pattern, self.H, self.H_kv, self.d, self.dtype, self.device = pattern, heads, kv_heads, d, dtype, device
        self.width = heads * d
        self.turns = kda.rope_turns([10000.0 ** (-2 * i / d) for i in range(d // 2)], device) if rope else None

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device=device) * rows ** -0.5).to(dtype)

        self.layers = []
        for kind in pattern:
            w = {"out": weight(self.width, self.width)}
            if kind == "k":
                w["qkv"], w["alpha"], w["beta"] = weight(self.width, 3 * self.width), weight(self.width, self.width), \
                    weight(self.width, heads)
            else:
                w["qkv"] = weight(self.width, (heads + 2 * kv_heads) * d)
                if rope:
                    w["q_weight"], w["k_weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device=device) for _ in range(2))
            self.layers.append(w)

    def turned(self, i, q, k, positions):
        """Layer i's queries and keys, normed and rotated in place."""
        if self.turns is not None:
            kda.qk_norm_rope(q, k, positions, self.turns, q_weight=self.layers[i]["q_weight"],
                             k_weight=self.layers[i]["k_weight"], q_out=q, k_out=k)
        return q, k

    def forward(self, x, kda_layer, attn_layer):
        """x [T, width] through the stack.  kda_layer(i, q, k, v, alpha, beta) and attn_layer(i,
        q, k, v) give the outputs [T, H, d] of layer i; q, k and v of an attention layer are
        views of one projection."""
        T, H, H_kv, d = x.shape[0], self.H, self.H_kv, self.d
        for i, (kind, w) in enumerate(zip(self.pattern, self.layers)):
            h = torch.nn.functional.rms_norm(x.float(), (self.width,)).to(self.dtype)
            qkv = h @ w["qkv"]
            if kind == "k":
                q, k, v = qkv.view(T, 3, H, d).unbind(1)
                q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(self.dtype) for t in (q, k))
                alpha = torch.sigmoid((h @ w["alpha"]).float() + 4).view(T, H, d)
                beta = torch.sigmoid((h @ w["beta"]).float())
                y = kda_layer(i, q, k, v.contiguous(), alpha, beta)
            else:
                y = attn_layer(i, *qkv.view(T, H + 2 * H_kv, d).split((H, H_kv, H_kv), 1))
            x = x + (y.reshape(T, self.width) @ w["out"])
        return x


class Server:
    """The requests' caches and states: per attention layer one pair of paged caches, per KDA
    layer one state pool (slot s for request s, the last slot for the shared prompt), and one
    block table and free list for all layers.

    With ``four_bit`` the pair of caches holds the shared prompt, in its first ``shared_blocks``
    blocks, and behind them, while prompts run, the values of the 4-bit cache's blocks."""

    def __init__(self, net, n, capacity, block_size=64, four_bit=False, prefix=0):
        self.net, self.n, self.block_size, self.four_bit = net, n, block_size, four_bit
        stride = -(-capacity // block_size)
        self.n_blocks = (n + 1) * stride
        self.shared_blocks = prefix // block_size if four_bit else 0
        dev = net.device
        self.q4 = {i: kda.q4_cache(self.n_blocks, net.H_kv, block_size, net.d, dev)
                   for i, kind in enumerate(net.pattern) if kind == "a" and four_bit}
        shape = (self.shared_blocks + self.n_blocks, net.H_kv, block_size, net.d)
        self.caches = {i: (torch.empty(shape, dtype=net.dtype, device=dev), torch.empty(shape, dtype=net.dtype, device=dev))
                       for i, kind in enumerate(net.pattern) if kind == "a"}
        self.pools = {i: torch.zeros(n + 1, net.H, net.d, net.d, device=dev)
                      for i, kind in enumerate(net.pattern) if kind == "k"}
        self.free = torch.randperm(self.n_blocks, device=dev, dtype=torch.int32)
        self.free_begin, self.free_end = (torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(2))
        self.table = torch.full((n, stride), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(n, dtype=torch.int32, device=dev)
        self.slots = torch.arange(n, dtype=torch.int32, device=dev)
        self.group_start = torch.tensor([0, n], dtype=torch.int32, device=dev)
        self.prefix_lens = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ones = torch.ones(n, dtype=torch.int32, device=dev)
        self.prefix = 0

    def plan(self, table, lens, new_lens, max_tokens):
        """Blocks and slots for the step's new tokens; the free list moves on."""
        plan = kda.cache_plan(lens, new_lens, table, self.free, self.free_begin, self.free_end,
                              block_size=self.block_size, n_blocks=self.n_blocks, max_tokens=max_tokens)
        self.free_begin.copy_(self.free_end)
        return plan

    def start(self, x):
        """The shared prompt, x [a multiple of UNIT, width]."""
        T = x.shape[0]
        table, zero = self.table[:1].clone(), torch.zeros(1, dtype=torch.int32, device=x.device)
        if self.four_bit:                                  # the prompt has blocks of its own
            blocks = torch.arange(self.shared_blocks, dtype=torch.int32, device=x.device)
            plan = kda.cache_plan(zero, zero + T, table, blocks, zero.clone(), zero.clone(), block_size=self.block_size,
                                  n_blocks=self.shared_blocks, max_tokens=T)
        else:
            plan = self.plan(table, zero, zero + T, T)

        def kda_layer(i, q, k, v, alpha, beta):
            o, self.pools[i][self.n:] = kda.prefill(q, k, v, alpha, beta, plan.cu_seqlens, T)
            return o

        def attn_layer(i, q, k, v):
            q, k = self.net.turned(i, q, k, plan.positions)
            kda.kda_cache_append(k, v, plan.slot_map, *self.caches[i])
            return kda.attn_prefill(q, k, v, plan.cu_seqlens)[0]

        y = self.net.forward(x, kda_layer, attn_layer)
        self.table[:, :T // self.block_size] = table[:, :T // self.block_size]
        self.lens.fill_(T)
        self.prefix_lens.fill_(T)
        self.prefix = T
        return y

    def prompts(self, x, new_lens):
        """The requests' own prompts, packed: x [sum of new_lens, width], new_lens int32 [n]."""
        T = x.shape[0]
        plan = self.plan(self.table, self.lens, new_lens, T)
        start = torch.full_like(self.slots, self.prefix)
        shared = torch.full_like(self.slots, self.n)

        def kda_layer(i, q, k, v, alpha, beta):
            o, self.pools[i][:self.n] = kda.prefill(q, k, v, alpha, beta, plan.cu_seqlens, T, start_pos=start,
                                                    init_slot=shared, pool=self.pools[i])
            return o

        table, slots = self.table, plan.slot_map
        if self.four_bit:                                  # the wide caches' own numbers, behind the prompt's blocks
            own = torch.arange(table.shape[1], device=x.device) >= self.shared_blocks
            table = torch.where(own & (table >= 0), table + self.shared_blocks, table)
            slots = torch.where(slots >= 0, slots + self.shared_blocks * self.block_size, slots)

        def attn_layer(i, q, k, v):
            q, k = self.net.turned(i, q, k, plan.positions)
            if self.four_bit:
                k, v = kda.cache_append_q4(k, v, plan.slot_map, self.q4[i], k_out=k, v_out=v)
            kda.kda_cache_append(k, v, slots, *self.caches[i])
            return kda.attn_prefill_paged(q, *self.caches[i], table, plan.kv_lens, plan.cu_seqlens)[0]

        y = self.net.forward(x, kda_layer, attn_layer)
        self.lens.copy_(plan.kv_lens)
        return y

    def more_prompts(self, x, new_lens):
        """Further turns: more tokens for the requests, behind what they hold.  With ``four_bit``, what
        their attention has to see of that is read back into the wide caches first."""
        if "k" in self.net.pattern:
            raise ValueError(f"a KDA layer resumes at multiples of {UNIT} tokens only")
        if self.four_bit:
            own = torch.arange(self.table.shape[1], device=x.device) >= self.shared_blocks
            wide = torch.where(own & (self.table >= 0), self.table + self.shared_blocks, self.table)
            first = torch.full_like(self.lens, self.prefix)
            for i, cache in self.q4.items():
                kda.cache_unpack_q4(cache, self.table, self.lens, *self.caches[i], wide, first=first)
        return self.prompts(x, new_lens)

    def step(self, x):
        """One new token per request, x [n, width].  Only device work of fixed sizes, so that it
        can be captured."""
        plan = self.plan(self.table, self.lens, self.ones, self.n)

        def kda_layer(i, q, k, v, alpha, beta):
            o = torch.empty_like(v)
            kda.kda_decode_step(q, k, v, alpha, beta, self.pools[i], self.slots, o)
            return o

        def attn_layer(i, q, k, v):
            shared = dict(group_start=self.group_start, prefix_lens=self.prefix_lens)
            if self.four_bit:
                q, k = self.net.turned(i, q, k, plan.positions)
                kda.cache_append_q4(k, v, plan.slot_map, self.q4[i])
                k_prefix, v_prefix = (c[:self.shared_blocks] for c in self.caches[i])
                return kda.attn_decode_q4(q, self.q4[i], self.table, plan.kv_lens, k_prefix=k_prefix, v_prefix=v_prefix, **shared)[0]
            if self.net.turns is not None:
                w = self.net.layers[i]
                q = kda.cache_append_rope(k, v, plan.positions, self.net.turns, plan.slot_map, *self.caches[i], q=q,
                                          q_weight=w["q_weight"], k_weight=w["k_weight"])
            else:
                kda.kda_cache_append(k, v, plan.slot_map, *self.caches[i])
            return kda.attn_decode(q, *self.caches[i], self.table, plan.kv_lens, **shared)[0]

        y = self.net.forward(x, kda_layer, attn_layer)
        self.lens.copy_(plan.kv_lens)
        return y

    def capture(self, x):
        """A graph of ``step`` on the buffer x; returns (graph, its output)."""
        saved = [t.clone() for t in self._advancing()]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):                    # first calls outside the capture
            self.step(x)
        torch.cuda.current_stream().wait_stream(stream)
        for t, was in zip(self._advancing(), saved):
            t.copy_(was)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x)
        return graph, y

    def _advancing(self):
        return [self.lens, self.free_begin, self.free_end, self.table, *self.pools.values()]


def recompute(net, x, cu_seqlens, prefix=0, four_bit=False):
    """The stack over whole packed sequences, from their first tokens; with ``four_bit``, tokens
    behind the first ``prefix`` of each have the keys and values that a 4-bit cache stands for."""
    T = x.shape[0]
    at = torch.arange(T, dtype=torch.int32, device=x.device)
    positions = at - cu_seqlens[torch.searchsorted(cu_seqlens, at, right=True) - 1]
    if four_bit:
        cache = kda.q4_cache(-(-T // 256), net.H_kv, 256, net.d, x.device)
        slots = torch.where(positions >= prefix, at, -1)

    def attn_layer(i, q, k, v):
        q, k = net.turned(i, q, k, positions)
        if four_bit:
            kda.cache_append_q4(k, v, slots, cache, k_out=k, v_out=v)
        return kda.attn_prefill(q, k, v, cu_seqlens)[0]

    return net.forward(x, lambda i, q, k, v, a, b: kda.prefill(q, k, v, a, b, cu_seqlens, T, want_final=False)[0], attn_layer)


def serve(net, n=8, prefix=2 * UNIT, longest=300, steps=16, block_size=64, seed=1, four_bit=False):
    """Serve ``n`` requests.  The input of a decode step is the last output, normalised, as a
    stand-in for sampling and embedding.  Returns (all inputs, all outputs, cu_seqlens) of the
    requests' full sequences, packed, and the milliseconds of one decode step."""
    gen = torch.Generator(net.device).manual_seed(seed)
    lens = torch.randint(1, longest + 1, (n,), generator=gen, device=net.device, dtype=torch.int32)
    own = torch.randn(int(lens.sum()), net.width, generator=gen, device=net.device).to(net.dtype)
    system = torch.randn(prefix, net.width, generator=gen, device=net.device).to(net.dtype)
    server = Server(net, n, prefix + longest + steps, block_size, four_bit, prefix)
    shared = server.start(system)
    hidden = server.prompts(own, lens)
    ends = lens.cumsum(0)
    last = hidden[ends - 1]
    x = torch.empty_like(last)
    graph, y = server.capture(x)
    fed, got = [], []
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(steps):
        x.copy_(torch.nn.functional.rms_norm(last.float(), (net.width,)))
        graph.replay()
        last = y.clone()
        fed.append(x.clone())
        got.append(last)
    end.record()
    assert kda.kda_check_status() == 0
    fed, got = torch.stack(fed, 1), torch.stack(got, 1)
    inputs, outputs = [], []
    for s, stop in enumerate(ends.tolist()):
        mine = slice(stop - int(lens[s]), stop)
        inputs += [system, own[mine], fed[s]]
        outputs += [shared, hidden[mine], got[s]]
    cu = torch.zeros(n + 1, dtype=torch.int32, device=net.device)
    cu[1:] = (lens + prefix + steps).cumsum(0)
    return torch.cat(inputs), torch.cat(outputs), cu, begin.elapsed_time(end) / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--pattern", default="kkka")
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--dtype", choices=("bf16", "fp32"), default="bf16")
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prefix", type=int, default=2 * UNIT, help=f"tokens of the system prompt, a multiple of {UNIT}")
    ap.add_argument("--longest", type=int, default=300, help="longest prompt of a request")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--rope", action="store_true", help="norms of queries and keys, and a position rotation")
    ap.add_argument("--cache", choices=("full", "4bit"), default="full", help="the requests' own tokens in the attention layers")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    with torch.no_grad():
        net = HybridStack(a.pattern, a.heads, a.kv_heads, dtype=dtype, rope=a.rope)
        four_bit = a.cache == "4bit"
        x, y, cu, ms = serve(net, a.requests, a.prefix, a.longest, a.steps, four_bit=four_bit)
        print(f"{a.requests} requests behind {a.prefix} shared tokens, layers {a.pattern}: {ms:.3f} ms a decode step, "
              f"{a.requests / ms * 1e3:.0f} tokens/s")
        if a.check:
            want = recompute(net, x, cu, a.prefix, four_bit)
            err = (y.double() - want.double()).norm() / want.double().norm()
            print(f"relative distance to the recomputed hidden states: {err:.2e}")


if __name__ == "__main__":
    main()
