"""The hybrid-stack example: prompts behind a shared, cached prefix and graph-replayed decode
steps give what the same stack gives over whole sequences, recomputed without a cache."""
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


def _tolerance(dtype, layers, longest_sum):
    """Norm-wise distance of two ways through the stack.  fp32: each of the about 8 sums of a
    layer has at most ``longest_sum`` terms and is off by at most longest_sum * 2^-24 of its
    terms' norm.  bf16: 6 tensors are rounded per layer (2^-8 each), independently in the two
    ways, so that their squares add; a layer passes on at most twice the distance it gets."""
    if dtype == torch.float32:
        return 8 * layers * longest_sum * 2.0 ** -24
    return 2 * (2 * 6 * layers) ** 0.5 * 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("pattern,heads,kv_heads,dtype,n,prefix,longest,steps,block_size", [
    ("kkka", 4, 2, torch.float32, 3, 256, 40, 5, 64),
    ("aka", 4, 1, torch.float32, 5, 512, 130, 20, 16),
    ("kkka", 8, 2, torch.bfloat16, 7, 512, 300, 12, 64),
    ("akka", 4, 4, torch.bfloat16, 1, 256, 1, 3, 256),
])
def test_served_equals_recomputed(cuda_device, kda, pattern, heads, kv_heads, dtype, n, prefix, longest, steps, block_size):
    ex = _example()
    with torch.no_grad():
        net = ex.HybridStack(pattern, heads, kv_heads, dtype=dtype, device=cuda_device)
        x, y, cu, _ = ex.serve(net, n, prefix, longest, steps, block_size)
        want = ex.recompute(net, x, cu)
    assert kda.kda_check_status() == 0
    assert torch.isfinite(y).all()
    longest_sum = max(net.width, prefix + longest + steps)
    got, want = y.double(), want.double()
    for s in range(n):
        mine = slice(int(cu[s]), int(cu[s + 1]))
        err = float((got[mine] - want[mine]).norm() / want[mine].norm())
        assert err <= _tolerance(dtype, len(pattern), longest_sum), (s, err)
