"""The hybrid-stack example with norms, rotation and a 4-bit cache: served requests equal the recomputed sequences, and a
further turn behind what is read back from the 4-bit cache equals them too.

Distances are norm-wise.  Without the 4-bit cache they are those of ``test_gpu_hybrid_example``: e1 = 8 layers K 2^-24 for fp32
(sums of at most K terms), 2 sqrt(12 layers) 2^-8 for bf16.  The 4-bit cache passes on a distance e of its inputs as follows: a
value near the middle of two codes moves by a whole step s where its input moves by t, with probability t / s, so that the
expected square is t s.  A group of 64 is at most about 15 / 4 of its standard deviation to each side, and s a fifteenth of
the width, so s <= sigma / 2 (3 sigma / 5 with outliers) and the distance behind the cache is sqrt(e s / sigma) <= sqrt(0.6 e).
It enters the stack again at each attention layer's output; a layer passes on at most twice what it gets, as in that test.
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_serving", os.path.join(ROOT, "examples", "hybrid_serving.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _tolerance(dtype, pattern, longest_sum, four_bit):
    e = 8 * len(pattern) * longest_sum * 2.0 ** -24 if dtype == torch.float32 else 2 * (12 * len(pattern)) ** 0.5 * 2.0 ** -8
    return e + 2 * pattern.count("a") * (0.6 * e) ** 0.5 if four_bit else e


def _compare(got, want, cu, tolerance):
    assert torch.isfinite(got).all()
    got, want = got.double(), want.double()
    for a, b in zip(cu.tolist()[:-1], cu.tolist()[1:]):
        err = float((got[a:b] - want[a:b]).norm() / want[a:b].norm())
        assert err <= tolerance, (a, err, tolerance)


@pytest.mark.gpu
@pytest.mark.parametrize("four_bit", [False, True])
@pytest.mark.parametrize("pattern,heads,kv_heads,d,dtype,n,prefix,longest,steps,block_size", [
    ("kkka", 4, 2, 128, torch.float32, 3, 256, 40, 5, 64),
    ("aka", 4, 1, 64, torch.float32, 5, 512, 130, 20, 16),
    ("kkka", 8, 2, 128, torch.bfloat16, 7, 512, 300, 12, 64),
])
def test_served_equals_recomputed(cuda_device, kda, pattern, heads, kv_heads, d, dtype, n, prefix, longest, steps, block_size, four_bit):
    ex = _example()
    with torch.no_grad():
        net = ex.HybridStack(pattern, heads, kv_heads, d, dtype=dtype, device=cuda_device, rope=True)
        x, y, cu, _ = ex.serve(net, n, prefix, longest, steps, block_size, four_bit=four_bit)
        want = ex.recompute(net, x, cu, prefix, four_bit)
    assert kda.kda_check_status() == 0
    _compare(y, want, cu, _tolerance(dtype, pattern, max(net.width, prefix + longest + steps), four_bit))


@pytest.mark.gpu
@pytest.mark.parametrize("four_bit", [False, True])
def test_further_turns(cuda_device, kda, four_bit):
    """Two turns of several requests behind a shared prompt, in a stack of attention layers."""
    ex = _example()
    dev, prefix, turns = cuda_device, 256, [[30, 1, 70, 16], [5, 64, 3, 17]]
    gen = torch.Generator(dev).manual_seed(3)
    with torch.no_grad():
        net = ex.HybridStack("aa", 4, 2, 64, dtype=torch.float32, device=dev, rope=True)
        server = ex.Server(net, 4, prefix + 200, 16, four_bit, prefix)
        system = torch.randn(prefix, net.width, generator=gen, device=dev)
        shared = server.start(system)
        inputs, outputs = [[system] for _ in range(4)], [[shared] for _ in range(4)]
        for turn, lens in enumerate(turns):
            x = torch.randn(sum(lens), net.width, generator=gen, device=dev)
            new = torch.tensor(lens, dtype=torch.int32, device=dev)
            y = (server.more_prompts if turn else server.prompts)(x, new)
            for s, (a, b) in enumerate(zip(x.split(lens), y.split(lens))):
                inputs[s].append(a)
                outputs[s].append(b)
        lens = [prefix + sum(t) for t in zip(*turns)]
        cu = torch.tensor([sum(lens[:i]) for i in range(5)], dtype=torch.int32, device=dev)
        want = ex.recompute(net, torch.cat(sum(inputs, [])), cu, prefix, four_bit)
    assert kda.kda_check_status() == 0 and server.lens.tolist() == lens
    _compare(torch.cat(sum(outputs, [])), want, cu, _tolerance(torch.float32, "aa", max(net.width, max(lens)), four_bit))
    with pytest.raises(ValueError, match="KDA layer"):
        ex.Server(ex.HybridStack("ka", 4, 2, 64, device=dev), 1, 300).more_prompts(system[:1], new[:1])
