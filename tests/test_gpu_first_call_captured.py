"""The first call of a process made inside a graph capture: nothing the serving
operators do on their first call (attributes of kernels, how many clusters the
device runs) breaks a capture, and the replay gives what a plain call gives."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys
sys.path.insert(0, {root!r})
import torch
import speculative_decoding_verification_vocab_gb300 as sv
g = torch.Generator(device="cuda").manual_seed(1)
B, Hq, Hkv, D, page, n = 2, 8, 2, 64, 16, {n}
per = -(-n // page)
kv = torch.randn(1, 2, B * per, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
probs = torch.softmax(torch.randn(B, 3, 40000, generator=g, device="cuda"), -1)
d = torch.randint(0, 40000, (B, 2), generator=g, device="cuda", dtype=torch.int32)
u, us = torch.rand(B, 2, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
sums = torch.zeros(1, B, Hkv, per * page, device="cuda")
start = kv.clone()

def run():
    out = sv.paged_attention(q, kv[0], table, lens, weight_sum=sums[0])
    kept, new, _ = sv.kv_evict(kv, table, lens, sums, n // 2, 2, 8)
    r = sv.verify_chain_probs(probs, probs[:, :2], d, u, us)
    return out, kept, new, r["tokens"]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
got, after = [t.clone() for t in got], kv.clone()
kv.copy_(start)
sums.zero_()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert torch.equal(after, kv)
print("same")
"""


@pytest.mark.parametrize("n", [300, 12000])
def test_first_call_inside_a_capture(n):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT, n=n)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
