"""GPU test of first calls that host threads make at the same time."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

# eight threads, each on its own stream, all at their first call of the library; then the same calls in turn
CHILD = """
import threading
import torch
from long_context_prefill_dhsa_b200 import binding
binding._load_marshal()
g = torch.Generator(device="cuda").manual_seed(1)
bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
n = 8
f = torch.rand(64, dtype=torch.float64, device="cuda", generator=g)
lengths = torch.tensor([900, 313], dtype=torch.int32, device="cuda")
sets = [(bf(2, 8, t, 128), bf(2, 1, 1000, 128), bf(2, 1, 1000, 128)) for t in (1, 40, 9, 20, 1, 40, 9, 20)]
weight, pos = torch.rand(2, 1, 1000, device="cuda", generator=g), torch.zeros(2, 1, 1000, dtype=torch.int32, device="cuda")

def calls(Q, K, V):
    q, _, _ = binding.rotary_qkv(Q, None, f)
    w = weight.clone()
    o = binding.tree_attn(q, K, V, lengths, weight=w)
    k, v, p = K.clone(), V.clone(), pos.clone()
    m = binding.cache_evict(k, v, w, p, lengths, 300)
    return q, o, k, v, w, m

got, failed, gate = [None] * n, [], threading.Barrier(n)

def work(i):
    try:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            gate.wait(60)
            got[i] = calls(*sets[i])
            s.synchronize()
    except BaseException as e:
        failed.append(repr(e))

torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join(120) for t in threads]
assert not failed and all(x is not None for x in got), failed
torch.cuda.synchronize()
for x, y in zip(got, [calls(*s) for s in sets]):
    assert all(torch.equal(a, b) for a, b in zip(x, y))
assert binding.check_device_status() == 0
print("same")
"""


@needs_gpu
def test_first_calls_of_several_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
