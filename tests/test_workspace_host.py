"""Which workspaces the calls accept (no GPU): the part that moe_forward_few
alone uses is asked for by it alone."""
import os
import subprocess
import sys

import pytest

from mixture_experts_layer_41_b200 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process that sees no GPU a call whose arguments pass fails at its first
# CUDA call, and one whose workspace is too small before it.
CODE = """
import sys, ctypes as C
sys.path.insert(0, %r)
from mixture_experts_layer_41_b200 import _lib as L, api
A = 1 << 20
weights = L.moe_weights(A, A, A, %s)
stats = L.moe_stats(A, A, A, A)
cfg = lambda T: api.make_config(num_tokens=T, hidden=2048, intermediate=768, num_experts=8, top_k=1, weight_dtype=%r)
small, larger = cfg(16), cfg(17)
n = api.moe_workspace_size(larger)
assert api.moe_workspace_size(small) > n
lib = L.lib()
c, w, s = C.byref(small), C.byref(weights), C.byref(stats)
print(lib.moe_permute(c, A, A, A, A, A, A, A, A, s, A, n, None),
      lib.moe_grouped_ffn(c, A, A, w, A, A, n, None),
      lib.moe_forward(c, A, A, None, w, A, None, None, None, A, n, None),
      lib.moe_forward_few(c, A, A, None, w, A, None, None, None, A, n, None),
      lib.moe_grouped_ffn(c, A, A, w, A, A, 4096, None))
"""


@pytest.mark.parametrize("weights,slots", [
    ("bf16", "None, None, None, None, None, None, None, None, None"),
    ("i8_channel", "A, A, A, None, None, None, None, None, None"),
    ("q4_affine_g64", "A, A, A, A, A, A, None, None, None"),
])
def test_workspace_of_a_larger_batch_serves_few_rows(weights, slots):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", CODE % (ROOT, slots, weights)], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in r.stdout.split()]
    assert got == [L.MOE_ERR_CUDA] * 3 + [L.MOE_ERR_WORKSPACE] * 2
