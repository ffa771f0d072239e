"""The library and the host-side prefix index work in a process that has no torch."""
import os
import subprocess
import sys

from hybrid_linear_attention_kda_gb300 import build as kbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None                       # importing it raises
import numpy as np
import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300.prefix_cache import PrefixCache
kda.load()
assert kda.kda_abi_version() > 0
index = PrefixCache(slot_base=0, n_slots=8)
plan = index.plan_request(np.arange(600, dtype=np.int32))
assert plan["start_pos"] == 0
assert kda.CachePlanArgs().n_seqs == 0 and kda.KDA_DEV_NO_BLOCKS == 0x40
"""


def test_load_without_torch():
    kbuild.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
