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
    """``pattern`` gives each layer's kind: "k" is KDA, "a" softmax attention.  Random weights;
    the projections are plain matrix products, and there are no feed-forward layers."""

    def __init__(self, pattern="kkka", heads=8, kv_heads=2, d=128, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        self.pattern, self.H, self.H_kv, self.d, self.dtype, self.device = pattern, heads, kv_heads, d, dtype, device
        self.width = heads * d

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
            self.layers.append(w)

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
    block table and free list for all layers."""

    def __init__(self, net, n, capacity, block_size=64):
        self.net, self.n, self.block_size = net, n, block_size
        stride = -(-capacity // block_size)
        self.n_blocks = (n + 1) * stride
        dev = net.device
        shape = (self.n_blocks, net.H_kv, block_size, net.d)
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
        plan = self.plan(table, zero, zero + T, T)

        def kda_layer(i, q, k, v, alpha, beta):
            o, self.pools[i][self.n:] = kda.prefill(q, k, v, alpha, beta, plan.cu_seqlens, T)
            return o

        def attn_layer(i, q, k, v):
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

        def attn_layer(i, q, k, v):
            kda.kda_cache_append(k, v, plan.slot_map, *self.caches[i])
            return kda.attn_prefill_paged(q, *self.caches[i], self.table, plan.kv_lens, plan.cu_seqlens)[0]

        y = self.net.forward(x, kda_layer, attn_layer)
        self.lens.copy_(plan.kv_lens)
        return y

    def step(self, x):
        """One new token per request, x [n, width].  Only device work of fixed sizes, so that it
        can be captured."""
        plan = self.plan(self.table, self.lens, self.ones, self.n)

        def kda_layer(i, q, k, v, alpha, beta):
            o = torch.empty_like(v)
            kda.kda_decode_step(q, k, v, alpha, beta, self.pools[i], self.slots, o)
            return o

        def attn_layer(i, q, k, v):
            kda.kda_cache_append(k, v, plan.slot_map, *self.caches[i])
            return kda.attn_decode(q, *self.caches[i], self.table, plan.kv_lens, group_start=self.group_start,
                                   prefix_lens=self.prefix_lens)[0]

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


def recompute(net, x, cu_seqlens):
    """The stack over whole packed sequences, from their first tokens."""
    return net.forward(x, lambda i, q, k, v, a, b: kda.prefill(q, k, v, a, b, cu_seqlens, x.shape[0], want_final=False)[0],
                       lambda i, q, k, v: kda.attn_prefill(q, k, v, cu_seqlens)[0])


def serve(net, n=8, prefix=2 * UNIT, longest=300, steps=16, block_size=64, seed=1):
    """Serve ``n`` requests.  The input of a decode step is the last output, normalised, as a
    stand-in for sampling and embedding.  Returns (all inputs, all outputs, cu_seqlens) of the
    requests' full sequences, packed, and the milliseconds of one decode step."""
    gen = torch.Generator(net.device).manual_seed(seed)
    lens = torch.randint(1, longest + 1, (n,), generator=gen, device=net.device, dtype=torch.int32)
    own = torch.randn(int(lens.sum()), net.width, generator=gen, device=net.device).to(net.dtype)
    system = torch.randn(prefix, net.width, generator=gen, device=net.device).to(net.dtype)
    server = Server(net, n, prefix + longest + steps, block_size)
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
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    with torch.no_grad():
        net = HybridStack(a.pattern, a.heads, a.kv_heads, dtype=dtype)
        x, y, cu, ms = serve(net, a.requests, a.prefix, a.longest, a.steps)
        print(f"{a.requests} requests behind {a.prefix} shared tokens, layers {a.pattern}: {ms:.3f} ms a decode step, "
              f"{a.requests / ms * 1e3:.0f} tokens/s")
        if a.check:
            want = recompute(net, x, cu)
            err = (y.double() - want.double()).norm() / want.double().norm()
            print(f"relative distance to the recomputed hidden states: {err:.2e}")


if __name__ == "__main__":
    main()
